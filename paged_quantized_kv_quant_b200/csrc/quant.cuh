// Quantisation of fp16 K/V rows to the cache formats, shared by the KV write
// kernel and the decode kernel's appending form (which writes the step's new
// tokens itself).
//
// Source: "ReVolta" PyPI page, "Weight and KV formats" ("E4M3 KV": static
// calibrated scales; "INT8 KV": scales per token and head computed at run
// time); "1Cat-LLM" README ("FP8 E4M3 / E5M2 KV storage").
//
// Codes without a division per element.  A code is the format's rounding of
// the correctly rounded fp32 quotient RN(x / s).  With r = RN(1 / s),
// r_lo = RN(r (1 - 2^-20)) and r_hi = RN(r (1 + 2^-20)), the products
// RN(x r_lo) and RN(x r_hi) lie strictly below and above RN(x / s) in
// magnitude (each factor is off by at most 2^-24 relatively, far less than
// the 2^-20 margin), and rounding to a code is monotonic: when both products
// give the same code, so does the quotient.  Otherwise -- a quotient within
// about 2^-20 of a rounding boundary, a few in a million -- the thread
// divides.  Products below the fp32 normal range round to a zero code on
// both sides, as does the quotient; scales whose reciprocal leaves the
// normal range always divide.
#pragma once

#include "common.cuh"
#include "internal.h"

#include <cuda_fp8.h>

namespace pkvq {

// fp32 quotient -> E4M3 / E5M2 with round-to-nearest-even and saturation to
// the largest finite value (the hardware conversion with .satfinite).
template <int KVT>
__device__ __forceinline__ uint32_t quant_fp8x2(float a, float b)
{
    __nv_fp8x2_storage_t p = __nv_cvt_float2_to_fp8x2(
        make_float2(a, b), __NV_SATFINITE, KVT == kKvE5m2 ? __NV_E5M2 : __NV_E4M3);
    return (uint32_t)p;
}

// fp16 NaN -> the format's all-ones NaN (S.1111.111 / S.11111.11) with the
// input's own sign.  Decided on the fp16 bits: fp32 arithmetic on the GPU does
// not keep the sign of a NaN.
__device__ __forceinline__ uint32_t fix_nan(uint32_t code, uint16_t hbits)
{
    if ((hbits & 0x7c00u) == 0x7c00u && (hbits & 0x03ffu))
        return ((hbits >> 8) & 0x80u) | 0x7fu;
    return code;
}

// True if one of the 8 fp16 values is a NaN (exponent all ones, mantissa
// non-zero): ((h & 0x7fff) + 0x3ff) carries into bit 15 exactly then.
__device__ __forceinline__ bool any_nan8(const uint4 &x)
{
    const uint32_t m = 0x7fff7fffu, k = 0x03ff03ffu;
    const uint32_t t = ((x.x & m) + k) | ((x.y & m) + k) | ((x.z & m) + k) | ((x.w & m) + k);
    return (t & 0x80008000u) != 0u;
}

// Reciprocal brackets of a positive scale (see the file comment); false if
// the products cannot be trusted (the reciprocal is not a normal number with
// room to spare), in which case the caller divides.
__device__ __forceinline__ bool recip_bracket(float s, float &r_lo, float &r_hi)
{
    const float r = __frcp_rn(s);
    r_lo = __fmul_rn(r, 1.0f - 0x1p-20f);
    r_hi = __fmul_rn(r, 1.0f + 0x1p-20f);
    return s > 0x1p-120f && s < 0x1p120f;
}

// 8 fp16 values -> 8 FP8 codes of x / scale (scale == 0 -> codes 0).
template <int KVT>
__device__ __forceinline__ uint2 quant_fp8_8(const uint4 &x, float scale, float r_lo, float r_hi,
                                             bool fast)
{
    if (scale == 0.0f)
        return make_uint2(0u, 0u);
    const __half2 *h = reinterpret_cast<const __half2 *>(&x);
    uint32_t c[4];
    bool same = fast;
    if (fast) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(h[i]);
            const uint32_t lo = quant_fp8x2<KVT>(__fmul_rn(f.x, r_lo), __fmul_rn(f.y, r_lo));
            const uint32_t hi = quant_fp8x2<KVT>(__fmul_rn(f.x, r_hi), __fmul_rn(f.y, r_hi));
            same &= lo == hi;
            c[i] = lo;
        }
    }
    if (!same) {   // a quotient next to a rounding boundary (or no brackets)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(h[i]);
            c[i] = quant_fp8x2<KVT>(__fdiv_rn(f.x, scale), __fdiv_rn(f.y, scale));
        }
    }
    if (any_nan8(x)) {
        const uint16_t *hb = reinterpret_cast<const uint16_t *>(&x);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            c[i] = fix_nan(c[i] & 0xffu, hb[2 * i]) | (fix_nan((c[i] >> 8) & 0xffu, hb[2 * i + 1]) << 8);
    }
    return make_uint2((c[0] & 0xffffu) | (c[1] << 16), (c[2] & 0xffffu) | (c[3] << 16));
}

__device__ __forceinline__ float absmax8(const uint4 &x)
{
    const __half2 *h = reinterpret_cast<const __half2 *>(&x);
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 f = __half22float2(h[i]);
        m = fmaxf(m, fmaxf(fabsf(f.x), fabsf(f.y)));
    }
    return m;
}

// Row scale s = fp16_rn(absmax / 127) over the 16-thread group (lanes of one
// half-warp); returns s as fp16 bits.
__device__ __forceinline__ uint16_t int8_row_scale(float local_absmax)
{
    float m = local_absmax;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    return __half_as_ushort(__float2half_rn(__fdiv_rn(m, 127.0f)));
}

// rint(q) for |q| < 2^22 as the bits of RN(q + 1.5 * 2^23): the integer sits
// in the low mantissa bits (ties to even, as rint).
__device__ __forceinline__ uint32_t rint_bits(float q)
{
    return __float_as_uint(__fadd_rn(q, 12582912.0f));
}

__device__ __forceinline__ uint32_t int8_code(uint32_t rbits)
{
    const int v = (int)rbits - (int)0x4B400000;   // bits of 1.5 * 2^23
    return (uint32_t)(max(-127, min(127, v)) & 0xff);
}

// 8 fp16 values -> 8 INT8 codes clamp(rint(x / s), -127, 127) (s == 0 ->
// codes 0).  |x / s| stays near 127 at most, far inside rint_bits' range; s is
// an fp16 value or absmax / 127 of fp16 values, whose reciprocal is normal.
__device__ __forceinline__ uint2 quant_int8_8(const uint4 &x, float s)
{
    if (s == 0.0f)
        return make_uint2(0u, 0u);
    float r_lo, r_hi;
    recip_bracket(s, r_lo, r_hi);
    const __half2 *h = reinterpret_cast<const __half2 *>(&x);
    uint32_t w[2] = {0u, 0u};
    bool same = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(h[i]);
        const uint32_t la = rint_bits(__fmul_rn(f.x, r_lo)), ha = rint_bits(__fmul_rn(f.x, r_hi));
        const uint32_t lb = rint_bits(__fmul_rn(f.y, r_lo)), hb = rint_bits(__fmul_rn(f.y, r_hi));
        same &= (la == ha) & (lb == hb);
        w[i >> 1] |= (int8_code(la) | (int8_code(lb) << 8)) << (16 * (i & 1));
    }
    if (!same) {   // a quotient next to a half-integer: divide
        w[0] = w[1] = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(h[i]);
            const uint32_t a = int8_code(rint_bits(__fdiv_rn(f.x, s)));
            const uint32_t b = int8_code(rint_bits(__fdiv_rn(f.y, s)));
            w[i >> 1] |= (a | (b << 8)) << (16 * (i & 1));
        }
    }
    return make_uint2(w[0], w[1]);
}

// --- block-scaled formats: one fp32 scale per (block, KV head) ---

// Largest code magnitude: a block's scale is absmax / this.
template <int KVT>
__device__ __forceinline__ constexpr float block_code_max()
{
    return KVT == kKvInt8Blk ? 127.0f : 448.0f;
}

// +-inf -> +-65504 and NaN -> 0, so that one such input neither voids a
// block's scale nor reaches the codes (a half is one of them iff its exponent
// is all ones: adding 0x0400 to the magnitude then carries into bit 15).
__device__ __forceinline__ uint4 finite8(uint4 x)
{
    const uint32_t m = 0x7fff7fffu, k = 0x04000400u;
    const uint32_t t = ((x.x & m) + k) | ((x.y & m) + k) | ((x.z & m) + k) | ((x.w & m) + k);
    if (t & 0x80008000u) {
        uint16_t *h = reinterpret_cast<uint16_t *>(&x);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if ((h[i] & 0x7c00u) == 0x7c00u)
                h[i] = (h[i] & 0x03ffu) ? 0u : (uint16_t)((h[i] & 0x8000u) | 0x7bffu);
    }
    return x;
}

// 8 finite fp16 values -> 8 codes of x / s by division, for the rare pieces
// whose bracketing products disagree.  Not inlined: 16 copies of 8 divisions
// per thread kept the write kernel waiting for its instructions (53 us instead
// of 39 us for 18K tokens x 8 heads, then with one warp for both K and V).
template <int KVT>
__device__ __noinline__ uint2 quant_block_divide(uint4 x, float s)
{
    const __half2 *h = reinterpret_cast<const __half2 *>(&x);
    uint32_t w[2] = {0u, 0u};
    if (s == 0.0f)
        return make_uint2(0u, 0u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(h[i]);
        const float a = __fdiv_rn(f.x, s), b = __fdiv_rn(f.y, s);
        const uint32_t c = KVT == kKvInt8Blk
                               ? int8_code(rint_bits(a)) | (int8_code(rint_bits(b)) << 8)
                               : quant_fp8x2<kKvFp8>(a, b) & 0xffffu;
        w[i >> 1] |= c << (16 * (i & 1));
    }
    return make_uint2(w[0], w[1]);
}

// Brackets of a block's scale: products with them round to one code iff the
// quotient does.
struct BlockScale {
    float s;
    float2 lo, hi;
    __device__ __forceinline__ explicit BlockScale(float scale) : s(scale)
    {
        float l = 0.0f, u = 0.0f;
        if (scale != 0.0f)
            recip_bracket(scale, l, u);   // absmax / 127 or / 448 of fp16 values: normal
        lo = make_float2(l, l);
        hi = make_float2(u, u);
    }
};

// 8 finite fp16 values -> 8 codes of x / s (s == 0 -> codes 0).
template <int KVT>
__device__ __forceinline__ uint2 quant_block_8(const uint4 &x, const BlockScale &b)
{
    const __half2 *h = reinterpret_cast<const __half2 *>(&x);
    uint32_t w[2], d[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 f0 = __half22float2(h[2 * i]), f1 = __half22float2(h[2 * i + 1]);
        const float2 l0 = __fmul2_rn(f0, b.lo), l1 = __fmul2_rn(f1, b.lo);
        const float2 u0 = __fmul2_rn(f0, b.hi), u1 = __fmul2_rn(f1, b.hi);
        if constexpr (KVT == kKvInt8Blk) {
            // |x / s| <= 127 (1 + 2^-20): the codes need no clamp
            const float2 k = make_float2(12582912.0f, 12582912.0f);   // 1.5 * 2^23: rint_bits
            const float2 a0 = __fadd2_rn(l0, k), a1 = __fadd2_rn(l1, k);
            const float2 c0 = __fadd2_rn(u0, k), c1 = __fadd2_rn(u1, k);
            auto low4 = [](float2 p, float2 q) {
                return __byte_perm(__byte_perm(__float_as_uint(p.x), __float_as_uint(p.y), 0x0040),
                                   __byte_perm(__float_as_uint(q.x), __float_as_uint(q.y), 0x0040),
                                   0x5410);
            };
            w[i] = low4(a0, a1);
            d[i] = low4(c0, c1);
        } else {
            w[i] = __byte_perm(quant_fp8x2<kKvFp8>(l0.x, l0.y), quant_fp8x2<kKvFp8>(l1.x, l1.y), 0x5410);
            d[i] = __byte_perm(quant_fp8x2<kKvFp8>(u0.x, u0.y), quant_fp8x2<kKvFp8>(u1.x, u1.y), 0x5410);
        }
    }
    // a quotient next to a rounding boundary; or scale 0, where -0 would keep its sign
    if ((w[0] != d[0]) | (w[1] != d[1]) | (b.s == 0.0f))
        return quant_block_divide<KVT>(x, b.s);
    return make_uint2(w[0], w[1]);
}

// 4 codes of a block whose scale grew: the codes of RN(value * ratio), ratio =
// RN(old scale / new scale) < 1.
template <int KVT>
__device__ __forceinline__ uint32_t requant_block_4(uint32_t codes, float ratio)
{
    if constexpr (KVT == kKvInt8Blk) {
        uint32_t r = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float v = (float)(int8_t)(codes >> (8 * i));
            r |= int8_code(rint_bits(__fmul_rn(v, ratio))) << (8 * i);
        }
        return r;
    } else {
        uint32_t lo, hi;
        e4m3x4_to_half2x2(codes, lo, hi);
        const float2 a = __half22float2(*reinterpret_cast<__half2 *>(&lo));
        const float2 b = __half22float2(*reinterpret_cast<__half2 *>(&hi));
        return quant_fp8x2<kKvFp8>(__fmul_rn(a.x, ratio), __fmul_rn(a.y, ratio)) |
               (quant_fp8x2<kKvFp8>(__fmul_rn(b.x, ratio), __fmul_rn(b.y, ratio)) << 16);
    }
}

// One thread's 8 elements (16-byte piece `sub` of 16) of a (token, KV head)
// row of K or V: the codes go to element offset drow * 128 + 8 sub of
// `cache` and, for INT8, the row scale to scale_tok[drow] (by piece 0).
// FP8 formats divide by head_scale (a per-head or per-layer value).  All 16
// threads of the row (one half-warp) take part, `write` or not: the INT8 row
// scale is a half-warp reduction.
template <int KVT>
__device__ __forceinline__ void quant_store_piece(uint8_t *cache, uint16_t *scale_tok,
                                                  float head_scale, size_t drow, int sub,
                                                  const uint4 &x, bool write)
{
    const size_t dst = drow * 128 + (size_t)sub * 8;
    if constexpr (KVT == kKvFp16) {
        if (write)
            *reinterpret_cast<uint4 *>(cache + dst * 2) = x;
    } else {
        uint2 c;
        if constexpr (kv_has_head_scale(KVT)) {
            const float sc = write ? head_scale : 0.0f;
            float lo, hi;
            const bool fast = recip_bracket(sc, lo, hi);
            c = quant_fp8_8<KVT>(x, sc, lo, hi, fast);
        } else {
            const uint16_t sb = int8_row_scale(absmax8(x));
            c = quant_int8_8(x, __half2float(__ushort_as_half(sb)));
            if (write && sub == 0)
                scale_tok[drow] = sb;
        }
        if (write)
            *reinterpret_cast<uint2 *>(cache + dst) = c;
    }
}

}  // namespace pkvq
