// Decode attention that also accumulates every key's softmax weight, for
// eviction by accumulated attention weight.
//
// Mathematics.  With s_rj the scaled score of query row r and key j and
// lse_r = ln sum_j e^s_rj, the weight of key j in KV head h is
//   W[j] += sum over the KV head's rows r = (query token, query head) of
//           e^(s_rj - lse_r).
// The normaliser is known only after the last split, so the split kernel
// stores the scores it has in registers (fp32, log2 units) and a second kernel
// turns them into weights: 4 bytes written and read per (row, key), which with
// 8 rows is a quarter of the 256 bytes of K and V, and mostly stays in the
// 126 MB L2; reading K again for a second Q K^T would cost 128 bytes per key
// from DRAM.  No atomics: every W element has one writer, so results do not
// depend on the order of CTAs.
#include "decode_split.cuh"

namespace pkvq {
namespace {

constexpr int kWThreads = 256;
// 8 sequences of 16K with 4 KV heads make 512 such chunks and 32 merging CTAs: at
// four CTAs per SM they run at once (2, 4 or 8 keys per thread with 5, 3 or 2 CTAs
// per SM: the whole call takes 45.2, 42.6 or 40.5 us, with 4 and 4 40.7 us).
constexpr int kKeysPerThread = 4;
// Keys per CTA.  With more than 8 score rows a key's scores are spread over the
// lanes of a warp instead (a thread that walks 120 rows of its own key alone made
// 40 of 61 us of a 15-token, 8-head call over 1,120 keys), and a CTA takes fewer.
template <int RR>
constexpr int kChunkOf = RR ? kWThreads * kKeysPerThread : 128;
constexpr int kMaxRows = 256;   // 16 query tokens x 16 heads per KV head

// Grid: x < chunks: keys [x * kChunkOf<RR>, ...) of (KV head y, sequence z); the
// remaining CTAs merge the partial states of 8 output rows each.
// RR: score rows per key (1, 2, 4, 8), or 0 for any multiple of 4.
template <int BS, int RR>
__global__ void __launch_bounds__(kWThreads, 4)
decode_weights_kernel(const DecodeParams p, const int chunks)
{
    __shared__ float lse2[kMaxRows];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.y, b = blockIdx.z;
    // The next call's kernels wait for this grid's completion themselves.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const SplitInfo si = find_split<BS>(p, -1, b);
    // the split kernel's partial states and scores
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // After a wait that gave up (there or in an earlier call) they are not all there:
    // the accumulator, which outlives this call, then stays as it was.
    __shared__ bool failed;
    if (threadIdx.x == 0)
        failed = device_wait_failed(p.status);

    if ((int)blockIdx.x >= chunks) {
        const int rr = ((int)blockIdx.x - chunks) * (kWThreads / 32) + warp;
        if (rr < p.rows && si.nsplit > 1) {   // (a single split wrote the final row itself)
            // (4 splits at a time: the other CTAs pay for this branch's registers)
            MergeRow<4> mr;
            mr.row0 = (size_t)((rr / p.rows_per_cta) * p.num_kv_heads + h) * p.num_splits *
                          p.rows_per_cta + rr % p.rows_per_cta;
            mr.stride = p.rows_per_cta;
            mr.load(p, si.first, si.nsplit, 0, lane);
            mr.finish(p, si.first, si.nsplit, b, h, rr, lane);
        }
        return;
    }

    const int R = RR ? RR : p.score_rows;
    const int lo = si.blk0 * BS;   // scores exist for keys lo .. ctx - 1
    const int hi = min(si.ctx, min(p.score_keys, (int)min(p.weight_stride, (long long)INT_MAX)));
    constexpr int kChunk = kChunkOf<RR>;
    const int c0 = blockIdx.x * kChunk;
    if (c0 >= hi || c0 + kChunk <= lo)
        return;   // (a CTA-wide decision)
    const float *sc = p.scores + ((size_t)b * p.num_kv_heads + h) * p.score_keys * R;
    float *W = p.weights + ((size_t)b * p.num_kv_heads + h) * p.weight_stride;

    // this thread's scores and weights are on their way while the row
    // normalisers are combined
    constexpr int kKeys = RR ? kKeysPerThread : 1;
    float v[kKeys][RR ? RR : 1], w[kKeys];
#pragma unroll
    for (int k = 0; k < (RR ? kKeys : 0); ++k) {
        const int key = c0 + k * kWThreads + threadIdx.x;
        w[k] = 0.0f;
        if (key >= lo && key < hi) {
            w[k] = W[key];
            if constexpr (RR != 0) {
                const float *src = sc + (size_t)key * RR;
                if constexpr (RR >= 4) {
#pragma unroll
                    for (int i = 0; i < RR; i += 4) {
                        const float4 x = *reinterpret_cast<const float4 *>(src + i);
                        v[k][i] = x.x, v[k][i + 1] = x.y, v[k][i + 2] = x.z, v[k][i + 3] = x.w;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < RR; ++i)
                        v[k][i] = src[i];
                }
            }
        }
    }
    // log2-sum-exp2 of every row from its splits' (max, sum) states, all rows at
    // once: a warp per row for up to 8 rows, otherwise `lp` lanes (a power of
    // two); rows that see no key (and padding rows) get +inf: weight 0
    auto row_state = [&](int r, int sub, int lp, float &M, float &L) {
        M = -INFINITY, L = 0.0f;
        if (r < p.rows) {
            const size_t row0 = (size_t)((r / p.rows_per_cta) * p.num_kv_heads + h) *
                                    p.num_splits * p.rows_per_cta + r % p.rows_per_cta;
            for (int s = sub; s < si.nsplit; s += lp) {
                const float2 ml = *reinterpret_cast<const float2 *>(
                    p.ws_ml + (row0 + (size_t)(si.first + s) * p.rows_per_cta) * 2);
                const float m = fmaxf(M, ml.x), mu = m == -INFINITY ? 0.0f : m;
                L = L * fast_exp2(M - mu) + ml.y * fast_exp2(ml.x - mu);
                M = m;
            }
        }
    };
    auto join = [&](int o, float &M, float &L) {
        const float m2 = __shfl_xor_sync(0xffffffffu, M, o);
        const float l2 = __shfl_xor_sync(0xffffffffu, L, o);
        const float m = fmaxf(M, m2), mu = m == -INFINITY ? 0.0f : m;
        L = L * fast_exp2(M - mu) + l2 * fast_exp2(m2 - mu);
        M = m;
    };
    float M, L;
    if constexpr (RR != 0) {
        for (int r = warp; r < RR; r += kWThreads / 32) {
            row_state(r, lane, 32, M, L);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                join(o, M, L);
            if (lane == 0)
                lse2[r] = L > 0.0f ? M + log2f(L) : INFINITY;
        }
    } else {
        int lp = 32;
        while (kWThreads / lp < R)
            lp /= 2;
        const int r = threadIdx.x / lp, sub = threadIdx.x % lp;
        row_state(r, sub, lp, M, L);
        for (int o = lp / 2; o > 0; o >>= 1)
            join(o, M, L);
        if (sub == 0 && r < R)
            lse2[r] = L > 0.0f ? M + log2f(L) : INFINITY;
    }
    __syncthreads();
    if (failed)
        return;
    if constexpr (RR != 0) {
#pragma unroll
        for (int k = 0; k < kKeys; ++k) {
            const int key = c0 + k * kWThreads + threadIdx.x;
            if (key < lo || key >= hi)
                continue;
            float a = 0.0f;
#pragma unroll
            for (int i = 0; i < RR; ++i)
                a += fast_exp2(v[k][i] - lse2[i]);
            W[key] = w[k] + a;
        }
    } else {
        // `per` lanes (a power of two) share a key, 4 rows each at a time
        int per = 4;
        while (per < 32 && per * 4 < R)
            per *= 2;
        const int sub = lane % per, kpw = 32 / per;   // keys of a warp at a time
        const int end = min(hi, c0 + kChunk);
        constexpr int kU = 4;                         // and their loads in flight
        for (int k0 = c0 + warp * kpw * kU; k0 < end; k0 += (kWThreads / 32) * kpw * kU) {
            float a[kU];
#pragma unroll
            for (int u = 0; u < kU; ++u)
                a[u] = 0.0f;
            for (int i = 4 * sub; i < R; i += 4 * per) {
                float4 x[kU];
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    const int key = k0 + u * kpw + lane / per;
                    x[u] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                    if (key >= lo && key < end)
                        x[u] = *reinterpret_cast<const float4 *>(sc + (size_t)key * R + i);
                }
#pragma unroll
                for (int u = 0; u < kU; ++u)
                    a[u] += (fast_exp2(x[u].x - lse2[i]) + fast_exp2(x[u].y - lse2[i + 1])) +
                            (fast_exp2(x[u].z - lse2[i + 2]) + fast_exp2(x[u].w - lse2[i + 3]));
            }
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int key = k0 + u * kpw + lane / per;
                for (int o = per / 2; o > 0; o >>= 1)
                    a[u] += __shfl_xor_sync(0xffffffffu, a[u], o);
                if (sub == 0 && key >= lo && key < end)
                    W[key] += a[u];
            }
        }
    }
}

template <int BS, int RR>
cudaError_t launch_w(const DecodeParams &p, cudaStream_t stream)
{
    const int chunks = (p.score_keys + kChunkOf<RR> - 1) / kChunkOf<RR>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(chunks + (p.rows + kWThreads / 32 - 1) / (kWThreads / 32)),
                       (unsigned)p.num_kv_heads, (unsigned)p.batch);
    cfg.blockDim = dim3(kWThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, decode_weights_kernel<BS, RR>, p, chunks);
}

template <int BS>
cudaError_t launch_rr(const DecodeParams &p, cudaStream_t stream)
{
    switch (p.score_rows) {
    case 1: return launch_w<BS, 1>(p, stream);
    case 2: return launch_w<BS, 2>(p, stream);
    case 4: return launch_w<BS, 4>(p, stream);
    case 8: return launch_w<BS, 8>(p, stream);
    default: return launch_w<BS, 0>(p, stream);
    }
}

}  // namespace

int weights_split_occupancy(int kv_dtype, int nt, int block_size)
{
    return split_occupancy_any<true>(kv_dtype, nt, block_size);
}

cudaError_t launch_decode_weights(const DecodeParams &p, const DecodePlan &plan, int kv_dtype,
                                  const CUtensorMap &kmap, const CUtensorMap &vmap,
                                  cudaStream_t stream)
{
    cudaError_t e = launch_split_any<true>(kv_dtype, plan.nt, p, kmap, vmap, stream);
    if (e != cudaSuccess)
        return e;
    switch (p.block_size) {
    case 16: return launch_rr<16>(p, stream);
    case 32: return launch_rr<32>(p, stream);
    case 64: return launch_rr<64>(p, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace pkvq
