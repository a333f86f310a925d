// KV write + quantise into the block-scaled formats: INT8 or E4M3 codes with
// one fp32 scale per (block, KV head) for K and one for V.
//
// Mathematics.  The new tokens of a sequence are its last positions.  Per
// touched block, KV head and for K and V each, with Q the largest code
// magnitude (127 or 448) and A the largest magnitude among the new tokens'
// elements in the block:
//   s = RN(A / Q), or max(that, the stored scale) if the block already holds
//   older tokens; code = round(RN(x / s)).
// Where an older block's scale grows, its older codes are rounded again:
// code' = round(RN(value * RN(s_old / s))).  A scale never shrinks while its
// block holds tokens, so a code is rounded again only when it must be.
//
// 16 rows of K or of V of a (sequence, touched block, KV head) belong to one
// warp, whose 32 lanes hold them as 8 16-byte pieces each: all loads are in
// flight at once, the absmax is a warp reduction (blocks of 32 or 64 tokens: 2
// or 4 warps and one exchange through shared memory), the rows stay in
// registers between the reduction and the encoding, and each element is read
// and written once; no atomics.  Consecutive units take consecutive heads, whose
// rows are adjacent in memory.
//
// The floor is memory: 512 bytes read and 256 written per token and KV head, 17.5
// us for 18.4K tokens x 8 heads (E4M3).  Measured 30.9 us, 3.7 TB/s, so no unit is
// at its limit: 67 % of the issue slots are taken, most by the exact conversion
// (two bracketing products and two conversions per element), and 64 registers leave
// half of the SM's warps to hide the loads.  With the division inlined, one CTA per block and one warp for K
// and V of 16 rows both took 53 us; that warp with the division out of line 39 us,
// a warp each for K and V (this form) 31 us.  Not kept: a grid without index
// divisions, 32.7 us.
#include "common.cuh"
#include "internal.h"
#include "quant.cuh"

namespace pkvq {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kPieces = 8;   // 16-byte pieces of K (and of V) per lane: 16 rows x 16 / 32

// Largest magnitude of 8 fp16 values, twice over (a NaN stays one).
__device__ __forceinline__ __half2 absmax2(const uint4 &x)
{
    const __half2 *h = reinterpret_cast<const __half2 *>(&x);
    return __hmax2_nan(__hmax2_nan(__habs2(h[0]), __habs2(h[1])),
                       __hmax2_nan(__habs2(h[2]), __habs2(h[3])));
}

// A warp's largest |x| over its pieces; infinities and NaN (found once per
// warp, on the maximum) are replaced first.
__device__ __forceinline__ float warp_absmax(uint4 (&x)[kPieces])
{
    float m;
    for (int pass = 0;; ++pass) {
        __half2 a = absmax2(x[0]);
#pragma unroll
        for (int q = 1; q < kPieces; ++q)
            a = __hmax2_nan(a, absmax2(x[q]));
        const __half top = __hmax_nan(__low2half(a), __high2half(a));
        m = __half2float(top);
        if (pass == 1 || !__any_sync(0xffffffffu, !(m <= 65504.0f)))
            break;
#pragma unroll
        for (int q = 0; q < kPieces; ++q)
            x[q] = finite8(x[q]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}

// Warp w of the launch: K (even) or V (odd) of the 16-row part of a unit, the
// units being (sequence, touched block, KV head), heads fastest.
template <int KVT, int BS>
__global__ void __launch_bounds__(kThreads, 4)
kv_write_block_kernel(const KvWriteBlockParams p, const int max_touched)
{
    constexpr int WPU = BS / 16;   // parts per unit
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool isv = warp & 1;
    const long long unit = ((long long)blockIdx.x * (kWarps / 2) + (warp >> 1)) / WPU;
    const int part = (warp >> 1) % WPU;
    const int h = (int)(unit % p.num_kv_heads);
    const long long bi = unit / p.num_kv_heads;
    const int b = (int)(bi / max_touched), i = (int)(bi % max_touched);
    const int sub = lane & 15;

    // (no warp returns before the exchange of the reductions)
    bool act = b < p.batch;
    int ctx = 0, tok0 = 0, n = 0;
    if (act) {
        ctx = __ldg(p.context_lens + b);
        tok0 = b * p.q_len;
        n = p.q_len;
        if (p.cu_seqlens_new) {
            tok0 = __ldg(p.cu_seqlens_new + b);
            n = __ldg(p.cu_seqlens_new + b + 1) - tok0;
        }
        act = tok0 >= 0 && tok0 + (long long)n <= p.num_tokens;   // rows that there are
    }
    const int start = ctx - n;          // position of the first new token (< 0: skipped)
    const int lo = max(start, 0);
    const int blk = lo / BS + i;
    act = act && n > 0 && blk < p.max_blocks_per_seq && blk < (ctx + BS - 1) / BS;
    int phys = act ? __ldg(p.block_table + (size_t)b * p.max_blocks_per_seq + blk) : 0;
#ifdef PKVQ_BOUNDS_CHECK
    if (act && (phys < 0 || phys >= p.num_blocks)) {
        if (lane == 0)
            atomicOr(p.status, kStatusBadBlock);
        act = false;
        phys = 0;
    }
#endif
    // the first position of this lane's piece q is pos0 + 2 q
    const int pos0 = act ? blk * BS + 16 * part + (lane >> 4) : 0;
    uint4 x[kPieces];
    const __half *src = (isv ? p.v : p.k) +
                        ((size_t)(act ? tok0 + (pos0 - start) : 0) * p.num_kv_heads + h) * kHeadDim +
                        sub * 8;
    const size_t step = (size_t)2 * p.num_kv_heads * kHeadDim;
#pragma unroll
    for (int q = 0; q < kPieces; ++q) {
        const int pos = pos0 + 2 * q;
        x[q] = make_uint4(0u, 0u, 0u, 0u);
        if (act && pos >= lo && pos < ctx)
            x[q] = __ldcs(reinterpret_cast<const uint4 *>(src + q * step));
    }
    const size_t cu = (size_t)phys * p.num_kv_heads + h;
    float *scale = (isv ? p.v_scale_blk : p.k_scale_blk) + cu;
    const bool has_old = act && blk * BS < lo;
    const float s_old = has_old ? *scale : 0.0f;
    float top = warp_absmax(x);
    if constexpr (WPU > 1) {
        __shared__ float parts[kWarps];
        if (lane == 0)
            parts[warp] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WPU; ++w)
            top = fmaxf(top, parts[warp - 2 * part + 2 * w]);
    }
    if (!act)
        return;
    const float s = fmaxf(__fdiv_rn(top, block_code_max<KVT>()), s_old);
    const BlockScale sb(s);
    uint8_t *dst = (isv ? p.v_cache : p.k_cache) +
                   (cu * BS + 16 * part + (lane >> 4)) * kHeadDim + sub * 8;
#pragma unroll
    for (int q = 0; q < kPieces; ++q) {
        const int pos = pos0 + 2 * q;
        if (pos >= lo && pos < ctx)
            *reinterpret_cast<uint2 *>(dst + 256 * q) = quant_block_8<KVT>(x[q], sb);
    }
    if (has_old && s > s_old) {
        // older tokens of this block: its scale grew
        const float ratio = __fdiv_rn(s_old, s);
#pragma unroll 1
        for (int q = 0; q < kPieces && pos0 + 2 * q < lo; ++q) {
            uint2 *c = reinterpret_cast<uint2 *>(dst + 256 * q);
            const uint2 o = *c;
            *c = make_uint2(requant_block_4<KVT>(o.x, ratio), requant_block_4<KVT>(o.y, ratio));
        }
    }
    if (part == 0 && lane == 0)
        *scale = s;
}

template <int KVT>
cudaError_t launch_bs(const KvWriteBlockParams &p, cudaStream_t stream)
{
    // blocks that max_new_len consecutive positions can touch
    const int touched = (int)(((long long)p.max_new_len + p.block_size - 2) / p.block_size + 1);
    const long long warps = (long long)touched * p.batch * p.num_kv_heads * (p.block_size / 16) * 2;
    const long long grid = (warps + kWarps - 1) / kWarps;
    if (grid >= (1LL << 31))
        return cudaErrorInvalidValue;
    switch (p.block_size) {
    case 16: kv_write_block_kernel<KVT, 16><<<(unsigned)grid, kThreads, 0, stream>>>(p, touched); break;
    case 32: kv_write_block_kernel<KVT, 32><<<(unsigned)grid, kThreads, 0, stream>>>(p, touched); break;
    case 64: kv_write_block_kernel<KVT, 64><<<(unsigned)grid, kThreads, 0, stream>>>(p, touched); break;
    default: return cudaErrorInvalidValue;
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_write_block(const KvWriteBlockParams &p, int kv_dtype, cudaStream_t stream)
{
    if (p.batch == 0 || p.max_new_len == 0)
        return cudaSuccess;
    return kv_dtype == kKvInt8Blk ? launch_bs<kKvInt8Blk>(p, stream)
                                  : launch_bs<kKvE4m3Blk>(p, stream);
}

}  // namespace pkvq
