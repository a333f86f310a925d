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
// Selection: fp32 weights map to unsigned keys of the same order, and up to four
// passes count the 8-bit digits of the keys that share the prefix found so far
// (radix selection), which gives the key T of the last kept position and how
// many positions of that key stay; they end early when all keys of a prefix
// stay.  Then every position is ranked: rank = kept before = (definite before) +
// min(equal before, ties).  A cluster of up to 8 CTAs shares a row: each keeps
// its slice's keys in shared memory (one read of the weights), counts into its
// own histogram (four copies by lane: neighbours' weights share digits) and adds
// the non-zero counts to every CTA's totals over distributed shared memory.  Its
// time goes to the passes one after the other, not to bytes: about 1.8 us each, of
// which the cluster barrier takes 0.7 (32 rows of 32K: 17.6 us in all; with 8,192
// positions per CTA 18.5 us); each pass walks the whole slice, although after the
// first digit few keys still matter.  Measured and not kept: one CTA for a row of 32K (38 us);
// 11-bit digits, in two or three passes (reading 8 x 8 KB of other CTAs'
// histograms: 28.6 us; adding the non-zero counts: a microsecond more than this).
//
// Block-scaled formats: a new block's scale is the largest of its tokens'
// source scales, and the codes from blocks with a smaller one are rounded again
// (code' = round(RN(value * RN(s_src / s_dst)))); tokens from a block with that
// scale keep their codes.
#include "common.cuh"
#include "internal.h"
#include "quant.cuh"

#include <cooperative_groups.h>

namespace pkvq {
namespace {

constexpr int kSelThreads = 512;
constexpr int kMaxCluster = 8;
constexpr int kSliceTarget = 4096;     // positions per CTA before a larger cluster is taken
constexpr int kSelSmemMax = 160 * 1024;
constexpr int kCopies = 4;             // of a CTA's histogram, by lane

// fp32 -> unsigned key of the same order; -0 equals +0, NaN is the lowest.
__device__ __forceinline__ uint32_t order_key(float w)
{
    if (w != w)
        return 0u;
    const uint32_t u = __float_as_uint(w + 0.0f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// The weight of a key; NaN and zeros, whose bits a key does not hold, are read
// again from `src`.
__device__ __forceinline__ float key_weight(uint32_t k, const float *src)
{
    if (k == 0u || k == 0x80000000u)
        return __ldg(src);
    return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

// Tokens of sequence b; never more than its weights or its table row hold.
__device__ __forceinline__ int evict_tokens(const EvictParams &p, int b)
{
    const long long most = min(p.weight_stride, (long long)p.max_blocks_per_seq * p.block_size);
    return (int)max(0LL, min((long long)__ldg(p.context_lens + b), most));
}

// Grid: x = rank in the cluster (the whole cluster: one row), y = KV head, z =
// sequence.  kSmem: a slice's keys fit shared memory; otherwise every pass reads
// the weights again.
template <bool kSmem>
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p)
{
    namespace cg = cooperative_groups;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ uint4 keys4[];
    uint32_t *keys = reinterpret_cast<uint32_t *>(keys4);
    __shared__ uint32_t hist[256 * kCopies];
    __shared__ uint32_t total[4][256];       // each pass's counts of the whole row
    __shared__ uint32_t sel[3];              // digit, positions of larger digits, of this digit
    __shared__ uint2 slices[kMaxCluster];    // every slice's definite and equal positions
    __shared__ uint2 wtot[kSelThreads / 32];
    const cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), C = (int)cl.num_blocks();
    const int h = blockIdx.y, b = blockIdx.z;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const size_t row = (size_t)b * p.num_kv_heads + h;
    const float *w = p.weights + row * p.weight_stride;
    float *wout = p.weights_out ? p.weights_out + row * p.weight_out_stride : nullptr;
    int32_t *keep = p.keep + row * p.budget;
    const int n = evict_tokens(p, b);
    const int m = min(n, p.budget);
    const bool all = n <= p.budget;   // (for the whole cluster)

    const int per = ((n + C - 1) / C + 3) / 4 * 4;   // this CTA's slice: [s0, s1)
    const int s0 = min(n, rank * per), s1 = min(n, s0 + per);
    const int c0 = p.sink, c1 = n - p.recent;        // candidates
    uint32_t prefix = 0, need = all ? 0u : (uint32_t)(p.budget - p.sink - p.recent);
    const bool none = need == 0;
    if (!all) {
        for (int i = tid; i < 4 * 256; i += kSelThreads)
            total[i >> 8][i & 255] = 0u;
        for (int i = tid; i < 256 * kCopies; i += kSelThreads)
            hist[i] = 0u;
        cl.barrier_arrive();   // totals are clear: others may add to them
        if constexpr (kSmem) {
            // (8 loads in flight per thread)
            for (int j0 = s0; j0 < s1; j0 += 8 * kSelThreads) {
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int j = j0 + i * kSelThreads + tid;
                    x[i] = j < s1 ? __ldg(w + j) : 0.0f;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int j = j0 + i * kSelThreads + tid;
                    if (j < s1)
                        keys[j - s0] = order_key(x[i]);
                }
            }
        }
    }
    // what needs no selection, while the other CTAs get here
    if (h == 0 && rank == 0 && tid == 0)
        p.new_context_lens[b] = m;
    for (int r = m + rank * kSelThreads + tid; r < p.budget; r += C * kSelThreads)
        keep[r] = -1;
    if (wout)
        for (long long r = m + rank * kSelThreads + tid; r < p.weight_out_stride;
             r += C * kSelThreads)
            wout[r] = 0.0f;
    if (all) {
        for (int j = rank * kSelThreads + tid; j < n; j += C * kSelThreads) {
            keep[j] = j;
            if (wout)
                wout[j] = w[j];
        }
        return;
    }
    __syncthreads();
    cl.barrier_wait();

    // keys of positions j .. j + 3 (j - s0 a multiple of 4; those behind s1 are
    // not to be used)
    auto keys_at = [&](int j, uint32_t (&k)[4]) {
        if constexpr (kSmem) {
            const uint4 x = keys4[(j - s0) >> 2];
            k[0] = x.x, k[1] = x.y, k[2] = x.z, k[3] = x.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                k[i] = j + i < s1 ? order_key(__ldg(w + j + i)) : 0u;
        }
    };
    bool whole = false;
    uint32_t nd = 0, ne = 0;   // thread t: of this slice's digit t, definite and equal so far
    const int j1 = min(s1, c1);
    for (int pass = 0; !none && pass < 4 && !whole; ++pass) {
        const int shift = 24 - 8 * pass;
        const uint32_t mask = pass == 0 ? 0u : 0xffffffffu << (shift + 8);
        for (int j = s0 + tid * 4; j < j1; j += kSelThreads * 4) {
            uint32_t k[4];
            keys_at(j, k);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if ((k[i] & mask) == prefix && j + i >= c0 && j + i < j1)
                    atomicAdd(&hist[((k[i] >> shift) & 255u) * kCopies + (lane & (kCopies - 1))],
                              1u);
        }
        __syncthreads();
        // every CTA adds its counts to every CTA's totals, and clears its own
        uint32_t mine = 0;
        if (tid < 256) {
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
                mine += hist[tid * kCopies + i];
                hist[tid * kCopies + i] = 0u;
            }
            if (mine)
                for (int r = 0; r < C; ++r)
                    atomicAdd(&cl.map_shared_rank(total[pass], r)[tid], mine);
        }
        cl.sync();
        if (warp == 0) {
            // lane l takes digits 255 - 8 l .. 248 - 8 l, from the largest down
            uint32_t c[8], t = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                c[i] = total[pass][255 - 8 * lane - i];
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
                    sel[2] = c[i];
                }
                before += c[i];
            }
        }
        __syncthreads();
        const uint32_t digit = sel[0];
        prefix |= digit << shift;
        need -= sel[1];
        // all keys with this prefix stay: no digit is left to find
        whole = sel[2] == need;
        // this slice's share: larger digits stay; the last digit's positions are
        // the equal ones
        nd += tid < 256 && (uint32_t)tid > digit ? mine : 0u;
        ne = (uint32_t)tid == digit ? mine : 0u;
        // (the next pass's barriers order the reads of sel before its writes)
    }
    if (whole)
        nd += ne, ne = 0;
    // All positions above T (or from it on) stay, and the first `ties` of key T.
    const uint32_t T = prefix, ties = need;
    // definite and equal positions of every slice, told to every CTA
    nd = __reduce_add_sync(0xffffffffu, nd);
    ne = __reduce_add_sync(0xffffffffu, ne);
    if (lane == 0)
        wtot[warp] = make_uint2(nd, ne);
    __syncthreads();
    if (tid < C) {
        // what is no candidate stays
        uint2 t = make_uint2((uint32_t)(max(0, min(s1, c0) - s0) + max(0, s1 - max(s0, c1))), 0u);
        for (int i = 0; i < kSelThreads / 32; ++i)
            t.x += wtot[i].x, t.y += wtot[i].y;
        cl.map_shared_rank(slices, tid)[rank] = t;
    }
    cl.sync();   // the last access to another CTA's memory: no CTA has to stay for others
    uint32_t def_base = 0, eq_base = 0;
    for (int r = 0; r < rank; ++r) {
        def_base += slices[r].x;
        eq_base += slices[r].y;
    }
    // The ranks of one round of positions, 4 consecutive ones per thread.
    for (int j0 = s0; j0 < s1; j0 += kSelThreads * 4) {
        bool def[4], eq[4];
        uint32_t cnt = 0, k[4] = {0u, 0u, 0u, 0u};   // definite << 16 | equal
        if (j0 + tid * 4 < s1)
            keys_at(j0 + tid * 4, k);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = j0 + tid * 4 + i;
            const bool cand = j >= c0 && j < c1;
            def[i] = j < s1 && (!cand || (!none && (k[i] > T || (whole && k[i] == T))));
            eq[i] = j < s1 && cand && !none && !whole && k[i] == T;
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
            wtot[warp].x = inc;
        __syncthreads();
        const uint32_t t = lane < kSelThreads / 32 ? wtot[lane].x : 0u;
        uint32_t s = t;
#pragma unroll
        for (int o = 1; o < kSelThreads / 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o)
                s += y;
        }
        const uint32_t sum = __shfl_sync(0xffffffffu, s, kSelThreads / 32 - 1);
        const uint32_t before = __shfl_sync(0xffffffffu, s - t, warp) + inc - cnt;
        uint32_t d = def_base + (before >> 16), e = eq_base + (before & 0xffffu);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (def[i] || (eq[i] && e < ties)) {
                const uint32_t r = d + min(e, ties);
                const int j = j0 + tid * 4 + i;
                keep[r] = j;
                if (wout)
                    wout[r] = key_weight(k[i], w + j);
            }
            d += def[i] ? 1u : 0u;
            e += eq[i] ? 1u : 0u;
        }
        def_base += sum >> 16;
        eq_base += sum & 0xffffu;
    }
}

// Moves the kept tokens of one new block and KV head.  Grid: x = block of the
// sequence's new table, y = KV head, z = sequence.  8 threads per row and
// 128-byte half; each thread moves 16 bytes of K and of V.
// Bound by memory: 8 sequences x 4 heads of 32K cut to 4K (E4M3), 67 MB read and written,
// take 12.7 us, 5.3 TB/s.
template <int KVT, int BS>
__global__ void __launch_bounds__(BS * 8) evict_move_kernel(const EvictParams p)
{
    constexpr bool kBlk = kv_has_block_scale(KVT);
    constexpr int kHalves = kv_elem_bytes(KVT);
    __shared__ float sk[BS], sv[BS];
    const int i = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    const int m = min(evict_tokens(p, b), p.budget);
    if (i * BS >= m) {
        // (wait all the same: in a call whose sequences are all empty nobody else
        // would, and this grid, which stands for the call in its stream, could end
        // before the kernel it depends on)
        asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
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
    // One CTA for each kSliceTarget positions that a row can have, at most 8: for
    // rows of 32K, 8 CTAs take 17.6 us, 4 take 18.5 us and one 38 us.
    const long long most =
        min(p.weight_stride, (long long)p.max_blocks_per_seq * block_size);
    int C = 1;
    while (C < kMaxCluster && most > (long long)C * kSliceTarget)
        C *= 2;
    const long long slice = ((most + C - 1) / C + 3) / 4 * 4 * 4;   // bytes
    const bool fits = slice <= kSelSmemMax;
    auto kern = fits ? evict_select_kernel<true> : evict_select_kernel<false>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)C, (unsigned)p.num_kv_heads, (unsigned)p.batch);
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = fits ? (size_t)slice : 0;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)C;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         fits ? kSelSmemMax : 0);
    if (e == cudaSuccess)
        e = cudaLaunchKernelEx(&cfg, kern, p);
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
