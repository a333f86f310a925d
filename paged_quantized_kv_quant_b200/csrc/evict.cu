// Eviction from a paged cache by accumulated attention weight: every
// (sequence, KV head) keeps its first tokens (attention sinks), its most
// recent ones and the heaviest of the others, moved in order to new blocks.
//
// Mathematics.  n = context length, m = min(n, budget).  If n <= budget all
// tokens stay.  Otherwise the kept set is {j < sink} + {j >= n - recent} + the
// budget - sink - recent positions of [sink, n - recent) with the largest
// weight, equal weights by the lowest position; NaN ranks below everything.
// Token keep[r], ascending, becomes token r.
//
// Selection: fp32 weights map to unsigned keys of the same order, and four
// passes over the row count 8-bit digits of the keys that share the prefix
// found so far (radix selection), which gives the key T of the last kept
// position and how many positions of that key stay.  One more pass ranks the
// positions: rank = kept before = (definite before) + min(equal before, ties).
//
// Block-scaled formats: a new block's scale is the largest of its tokens'
// source scales, and the codes from blocks with a smaller one are rounded again
// (code' = round(RN(value * RN(s_src / s_dst)))); tokens from a block with that
// scale keep their codes.
#include "common.cuh"
#include "internal.h"
#include "quant.cuh"

namespace pkvq {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kPer = 4;   // positions per thread and round of the ranking pass

// fp32 -> unsigned key of the same order; -0 equals +0, NaN is the lowest.
__device__ __forceinline__ uint32_t order_key(float w)
{
    if (w != w)
        return 0u;
    const uint32_t u = __float_as_uint(w + 0.0f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// Tokens of sequence b; never more than its weights or its table row hold.
__device__ __forceinline__ int evict_tokens(const EvictParams &p, int b)
{
    const long long most = min(p.weight_stride, (long long)p.max_blocks_per_seq * p.block_size);
    return (int)max(0LL, min((long long)__ldg(p.context_lens + b), most));
}

// Grid: x = KV head, y = sequence.
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ uint32_t hist[256];
    __shared__ uint32_t sel[2];          // digit, positions of larger digits
    __shared__ uint32_t wtot[kSelThreads / 32];
    const int h = blockIdx.x, b = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const size_t row = (size_t)b * p.num_kv_heads + h;
    const float *w = p.weights + row * p.weight_stride;
    float *wout = p.weights_out ? p.weights_out + row * p.weight_out_stride : nullptr;
    int32_t *keep = p.keep + row * p.budget;
    const int n = evict_tokens(p, b);
    const int m = min(n, p.budget);
    if (h == 0 && tid == 0)
        p.new_context_lens[b] = m;

    const bool all = n <= p.budget;
    const int c0 = all ? n : p.sink, c1 = all ? n : n - p.recent;   // candidates [c0, c1)
    uint32_t prefix = 0, need = all ? 0 : (uint32_t)(p.budget - p.sink - p.recent);
    if (!all && need > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += kSelThreads)
                hist[i] = 0u;
            __syncthreads();
            const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
            for (int j = c0 + tid; j < c1; j += kSelThreads) {
                const uint32_t k = order_key(__ldg(w + j));
                if ((k & mask) == prefix)
                    atomicAdd(&hist[(k >> shift) & 255u], 1u);
            }
            __syncthreads();
            if (warp == 0) {
                // lane l counts digits 255 - 8 l .. 248 - 8 l, from the largest down
                uint32_t c[8], t = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    c[i] = hist[255 - 8 * lane - i];
                    t += c[i];
                }
                uint32_t before = t;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t x = __shfl_up_sync(0xffffffffu, before, o);
                    if (lane >= o)
                        before += x;
                }
                before -= t;   // positions with digits above this lane's
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (before < need && before + c[i] >= need) {
                        sel[0] = 255 - 8 * lane - i;
                        sel[1] = before;
                    }
                    before += c[i];
                }
            }
            __syncthreads();
            prefix |= sel[0] << shift;
            need -= sel[1];
            // (the next pass's first barrier orders these reads before its writes)
        }
    }
    // all of key T's positions up to the need-th stay
    const uint32_t T = prefix, ties = need;
    const bool none = !all && p.budget == p.sink + p.recent;
    uint32_t def_base = 0, eq_base = 0;
    for (int j0 = 0; j0 < n; j0 += kSelThreads * kPer) {
        bool def[kPer], eq[kPer];
        float x[kPer];
        uint32_t cnt = 0;   // definite << 16 | equal
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int j = j0 + tid * kPer + i;
            def[i] = eq[i] = false;
            x[i] = 0.0f;
            if (j < n) {
                x[i] = __ldg(w + j);
                if (j < c0 || j >= c1) {
                    def[i] = true;
                } else if (!none) {
                    const uint32_t k = order_key(x[i]);
                    def[i] = k > T;
                    eq[i] = k == T;
                }
            }
            cnt += (def[i] ? 0x10000u : 0u) + (eq[i] ? 1u : 0u);
        }
        uint32_t inc = cnt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o)
                inc += y;
        }
        __syncthreads();   // the previous round's totals have been read
        if (lane == 31)
            wtot[warp] = inc;
        __syncthreads();
        uint32_t t = wtot[lane], s = t;   // 32 warps
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o)
                s += y;
        }
        const uint32_t total = __shfl_sync(0xffffffffu, s, 31);
        const uint32_t wbase = __shfl_sync(0xffffffffu, s - t, warp);
        const uint32_t before = wbase + inc - cnt;
        uint32_t d = def_base + (before >> 16), e = eq_base + (before & 0xffffu);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (def[i] || (eq[i] && e < ties)) {
                const uint32_t r = d + min(e, ties);
                keep[r] = j0 + tid * kPer + i;
                if (wout)
                    wout[r] = x[i];
            }
            d += def[i] ? 1u : 0u;
            e += eq[i] ? 1u : 0u;
        }
        def_base += total >> 16;
        eq_base += total & 0xffffu;
    }
    for (int r = m + tid; r < p.budget; r += kSelThreads)
        keep[r] = -1;
    if (wout)
        for (long long r = m + tid; r < p.weight_out_stride; r += kSelThreads)
            wout[r] = 0.0f;
}

// Moves the kept tokens of one new block and KV head.  Grid: x = block of the
// sequence's new table, y = KV head, z = sequence.  8 threads per row and
// 128-byte half; each thread moves 16 bytes of K and of V.
template <int KVT, int BS>
__global__ void __launch_bounds__(BS * 8) evict_move_kernel(const EvictParams p)
{
    constexpr bool kBlk = kv_has_block_scale(KVT);
    constexpr int kHalves = kv_elem_bytes(KVT);
    __shared__ float sk[BS], sv[BS];
    const int i = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    const int m = min(evict_tokens(p, b), p.budget);
    if (i * BS >= m)
        return;
    const int dst = __ldg(p.dst_block_table + (size_t)b * p.dst_max_blocks + i);
    // the list of kept positions comes from the kernel before
    asm volatile("griddepcontrol.wait;" ::: "memory");
#ifdef PKVQ_BOUNDS_CHECK
    if (dst < 0 || dst >= p.num_blocks) {
        if (threadIdx.x == 0)
            atomicOr(p.status, kStatusBadBlock);
        return;
    }
#endif
    const int r = threadIdx.x >> 3, c = threadIdx.x & 7;
    bool live = i * BS + r < m;
    int src = 0, off = 0;
    if (live) {
        const int j = p.keep[((size_t)b * p.num_kv_heads + h) * p.budget + i * BS + r];
        src = __ldg(p.block_table + (size_t)b * p.max_blocks_per_seq + j / BS);
        off = j % BS;
#ifdef PKVQ_BOUNDS_CHECK
        if (src < 0 || src >= p.num_blocks) {
            if (c == 0)
                atomicOr(p.status, kStatusBadBlock);
            live = false;
            src = 0;
        }
#endif
    }
    const size_t su = (size_t)src * p.num_kv_heads + h, du = (size_t)dst * p.num_kv_heads + h;
    uint4 kx[kHalves], vx[kHalves];
#pragma unroll
    for (int q = 0; q < kHalves; ++q) {
        kx[q] = vx[q] = make_uint4(0u, 0u, 0u, 0u);
        if (live) {
            const size_t o = ((su * BS + off) * kHalves + q) * 128 + c * 16;
            kx[q] = *reinterpret_cast<const uint4 *>(p.k_cache + o);
            vx[q] = *reinterpret_cast<const uint4 *>(p.v_cache + o);
        }
    }
    if constexpr (KVT == kKvInt8) {
        if (live && c == 0) {
            p.k_scale_tok[du * BS + r] = p.k_scale_tok[su * BS + off];
            p.v_scale_tok[du * BS + r] = p.v_scale_tok[su * BS + off];
        }
    }
    if constexpr (kBlk) {
        const float ks = live ? p.k_scale_blk[su] : 0.0f, vs = live ? p.v_scale_blk[su] : 0.0f;
        if (c == 0)
            sk[r] = ks, sv[r] = vs;
        __syncthreads();
        float km = 0.0f, vm = 0.0f;
#pragma unroll
        for (int q = 0; q < BS; ++q) {
            km = fmaxf(km, sk[q]);
            vm = fmaxf(vm, sv[q]);
        }
        if (ks < km) {
            const float f = __fdiv_rn(ks, km);
            kx[0] = make_uint4(requant_block_4<KVT>(kx[0].x, f), requant_block_4<KVT>(kx[0].y, f),
                               requant_block_4<KVT>(kx[0].z, f), requant_block_4<KVT>(kx[0].w, f));
        }
        if (vs < vm) {
            const float f = __fdiv_rn(vs, vm);
            vx[0] = make_uint4(requant_block_4<KVT>(vx[0].x, f), requant_block_4<KVT>(vx[0].y, f),
                               requant_block_4<KVT>(vx[0].z, f), requant_block_4<KVT>(vx[0].w, f));
        }
        if (threadIdx.x == 0) {
            p.k_scale_blk[du] = km;
            p.v_scale_blk[du] = vm;
        }
    }
#pragma unroll
    for (int q = 0; q < kHalves; ++q)
        if (live) {
            const size_t o = ((du * BS + r) * kHalves + q) * 128 + c * 16;
            *reinterpret_cast<uint4 *>(p.k_cache + o) = kx[q];
            *reinterpret_cast<uint4 *>(p.v_cache + o) = vx[q];
        }
}

template <int KVT, int BS>
cudaError_t launch_move(const EvictParams &p, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.budget + BS - 1) / BS), (unsigned)p.num_kv_heads,
                       (unsigned)p.batch);
    cfg.blockDim = dim3(BS * 8);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, evict_move_kernel<KVT, BS>, p);
}

}  // namespace

cudaError_t launch_evict(const EvictParams &p, int kv_dtype, int block_size, cudaStream_t stream)
{
    evict_select_kernel<<<dim3((unsigned)p.num_kv_heads, (unsigned)p.batch), kSelThreads, 0,
                          stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    // E4M3 and E5M2 rows move as bytes: their scales belong to the head
    const int t = kv_dtype == kKvE5m2 ? kKvFp8 : kv_dtype;
    switch (t * 100 + block_size) {
#define PKVQ_EVICT_CASE(T, B) \
    case T * 100 + B: return launch_move<T, B>(p, stream);
        PKVQ_EVICT_CASE(kKvFp8, 16) PKVQ_EVICT_CASE(kKvFp8, 32) PKVQ_EVICT_CASE(kKvFp8, 64)
        PKVQ_EVICT_CASE(kKvInt8, 16) PKVQ_EVICT_CASE(kKvInt8, 32) PKVQ_EVICT_CASE(kKvInt8, 64)
        PKVQ_EVICT_CASE(kKvFp16, 16) PKVQ_EVICT_CASE(kKvFp16, 32) PKVQ_EVICT_CASE(kKvFp16, 64)
        PKVQ_EVICT_CASE(kKvInt8Blk, 16) PKVQ_EVICT_CASE(kKvInt8Blk, 32)
        PKVQ_EVICT_CASE(kKvInt8Blk, 64)
        PKVQ_EVICT_CASE(kKvE4m3Blk, 16) PKVQ_EVICT_CASE(kKvE4m3Blk, 32)
        PKVQ_EVICT_CASE(kKvE4m3Blk, 64)
#undef PKVQ_EVICT_CASE
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace pkvq
