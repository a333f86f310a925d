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
// A CTA owns one (sequence, touched block, KV head): the block's absmax needs
// no atomics and no second pass, the rows stay in registers between the
// reduction and the encoding, and each element is read and written once.
// Bound by memory: 512 bytes read and 256 written per token and KV head.
#include "common.cuh"
#include "internal.h"
#include "quant.cuh"

namespace pkvq {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerPass = kThreads / 16;   // 16 threads x 8 elements per row

// Grid: x = (sequence, touched block), y = KV head.
template <int KVT, int BS>
__global__ void __launch_bounds__(kThreads) kv_write_block_kernel(const KvWriteBlockParams p,
                                                                  const int max_touched)
{
    constexpr int RP = BS / kRowsPerPass;   // rows per thread
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int b = blockIdx.x / max_touched, i = blockIdx.x % max_touched;
    const int h = blockIdx.y;
    const int sub = threadIdx.x & 15, r0 = threadIdx.x >> 4;

    const int ctx = __ldg(p.context_lens + b);
    int tok0 = b * p.q_len, n = p.q_len;
    if (p.cu_seqlens_new) {
        tok0 = __ldg(p.cu_seqlens_new + b);
        n = __ldg(p.cu_seqlens_new + b + 1) - tok0;
    }
    const int start = ctx - n;          // position of the first new token (< 0: skipped)
    const int lo = max(start, 0);
    const int blk = lo / BS + i;
    if (n <= 0 || blk * BS >= ctx || blk >= p.max_blocks_per_seq)
        return;
    const int phys = __ldg(p.block_table + (size_t)b * p.max_blocks_per_seq + blk);
#ifdef PKVQ_BOUNDS_CHECK
    if (phys < 0 || phys >= p.num_blocks) {
        if (threadIdx.x == 0)
            atomicOr(p.status, kStatusBadBlock);
        return;
    }
#endif
    const size_t unit = (size_t)phys * p.num_kv_heads + h;
    const bool has_old = blk * BS < lo;
    const float ks_old = has_old ? p.k_scale_blk[unit] : 0.0f;
    const float vs_old = has_old ? p.v_scale_blk[unit] : 0.0f;

    uint4 kx[RP], vx[RP];
    float ka = 0.0f, va = 0.0f;
#pragma unroll
    for (int q = 0; q < RP; ++q) {
        const int pos = blk * BS + q * kRowsPerPass + r0;
        kx[q] = vx[q] = make_uint4(0u, 0u, 0u, 0u);
        if (pos >= lo && pos < ctx) {
            const size_t src =
                ((size_t)(tok0 + (pos - start)) * p.num_kv_heads + h) * kHeadDim + sub * 8;
            kx[q] = __ldcs(reinterpret_cast<const uint4 *>(p.k + src));
            vx[q] = __ldcs(reinterpret_cast<const uint4 *>(p.v + src));
        }
    }
#pragma unroll
    for (int q = 0; q < RP; ++q) {
        kx[q] = finite8(kx[q]);
        vx[q] = finite8(vx[q]);
        ka = fmaxf(ka, absmax8(kx[q]));
        va = fmaxf(va, absmax8(vx[q]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        ka = fmaxf(ka, __shfl_xor_sync(0xffffffffu, ka, o));
        va = fmaxf(va, __shfl_xor_sync(0xffffffffu, va, o));
    }
    __shared__ float2 part[kThreads / 32];
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = make_float2(ka, va);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        ka = fmaxf(ka, part[w].x);
        va = fmaxf(va, part[w].y);
    }
    const float ks = fmaxf(__fdiv_rn(ka, block_code_max<KVT>()), ks_old);
    const float vs = fmaxf(__fdiv_rn(va, block_code_max<KVT>()), vs_old);
    const bool kgrew = has_old && ks > ks_old, vgrew = has_old && vs > vs_old;
    const float kratio = kgrew ? __fdiv_rn(ks_old, ks) : 1.0f;
    const float vratio = vgrew ? __fdiv_rn(vs_old, vs) : 1.0f;

#pragma unroll
    for (int q = 0; q < RP; ++q) {
        const int r = q * kRowsPerPass + r0, pos = blk * BS + r;
        uint2 *kd = reinterpret_cast<uint2 *>(p.k_cache + (unit * BS + r) * kHeadDim + sub * 8);
        uint2 *vd = reinterpret_cast<uint2 *>(p.v_cache + (unit * BS + r) * kHeadDim + sub * 8);
        if (pos >= lo && pos < ctx) {
            *kd = quant_block_8<KVT>(kx[q], ks);
            *vd = quant_block_8<KVT>(vx[q], vs);
        } else if (pos < lo) {   // an older token of this block
            if (kgrew) {
                const uint2 c = *kd;
                *kd = make_uint2(requant_block_4<KVT>(c.x, kratio), requant_block_4<KVT>(c.y, kratio));
            }
            if (vgrew) {
                const uint2 c = *vd;
                *vd = make_uint2(requant_block_4<KVT>(c.x, vratio), requant_block_4<KVT>(c.y, vratio));
            }
        }
    }
    if (threadIdx.x == 0) {
        p.k_scale_blk[unit] = ks;
        p.v_scale_blk[unit] = vs;
    }
}

template <int KVT>
cudaError_t launch_bs(const KvWriteBlockParams &p, cudaStream_t stream)
{
    // blocks that max_new_len consecutive positions can touch
    const int touched = (int)(((long long)p.max_new_len + p.block_size - 2) / p.block_size + 1);
    const long long x = (long long)touched * p.batch;
    if (x >= (1LL << 31) || p.num_kv_heads > 65535)
        return cudaErrorInvalidValue;
    const dim3 grid((unsigned)x, (unsigned)p.num_kv_heads);
    switch (p.block_size) {
    case 16: kv_write_block_kernel<KVT, 16><<<grid, kThreads, 0, stream>>>(p, touched); break;
    case 32: kv_write_block_kernel<KVT, 32><<<grid, kThreads, 0, stream>>>(p, touched); break;
    case 64: kv_write_block_kernel<KVT, 64><<<grid, kThreads, 0, stream>>>(p, touched); break;
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
