// Causal attention over packed whole prompts (pkvq_prompt_attn): fp16 or bf16
// Q, K and V as the projections leave them, on the 5th-generation tensor
// cores (tcgen05, accumulators in tensor memory).
//
// Mathematics.  S = softmax_scale Q K^T, O = softmax(S) V per (sequence, query
// head), key j visible to token i iff max(0, i - w + 1) <= j <= i (w the
// sliding window, if any).  One pass over the keys with a running maximum m
// and sum l per row (fp32): p = 2^(kS - m), O += p V, out = O / l.  O is
// rescaled only when a row's maximum grew by more than 2^8, so p <= 256.
//
// A CTA owns two adjacent query tiles A and B of 128 rows: a tile is 128 / G
// tokens x the G query heads of one KV head, so every K/V tile serves all heads
// of its group and a diagonal tile wastes little.  Key tiles hold 80 keys: then
// tensor memory takes, per query tile, S (80 columns), P (40, two per column)
// and O (128), all apart: S(j+1) = Q K(j+1)^T is issued as soon as the softmax
// has S(j) in registers, and a tile's softmax never waits for the tensor core.
// (128-key tiles fit only with P over S; each tile's next S then waited for its
// P V, 1,600 of 3,800 cycles per tile.)
// Warp roles (11 warps):
//   warps 0-3  softmax of tile A, warps 4-7 of tile B: thread i owns row i, its
//              80 scores in registers.
//   warp 8     TMA producer: Q tiles (one 3-D box: 64 d x G heads x tokens, so
//              the rows land packed), then K and V tiles through a ring of 20 KB
//              stages; any token and head stride that TMA takes serves.
//   warp 9     issues S = Q K^T, warp 10 P V, of each tile in turn.  (One issuer
//              for both spent 100 cycles on each barrier that was already
//              complete, and an MMA's issue waits for the tensor core to take
//              it: 2,450 cycles per pair of tiles, half of them issuing.)
// Measured: one 8K prompt, 32 / 4 heads, fp16: 505-525 us, 1,050-1,090 TFLOP/s of
// useful work (floor 323 us at the 1,700 TFLOP/s burst rate, 390 at the 1,409
// that the 1 kW power cap sustains); 7 packed prompts up to 2K, 32 / 8 heads, bf16:
// 137 us.  Power bounds the long prompt (the clock falls to 1.5-1.65 GHz): a
// quarter of the exponentials on the FMA pipe (556 us against 544 in the 128-key
// form) or P stored after all of them (580 against 524) cost more than they hid.
// A sequence's last K/V tile may run into the next sequence: scores behind the
// end are masked, and the V rows there are zeroed in shared memory first (0
// times another prompt's infinity would be NaN).
#include "common.cuh"
#include "internal.h"
#include "tc.cuh"

#include <climits>
#include <cuda_bf16.h>
#include <math.h>

namespace pkvq {
namespace {

constexpr int kThreads = 352;
constexpr int kKT = kPromptKeys;  // keys per tile
constexpr int kStages = 8;        // ring of K and V tiles
constexpr int kQTile = 32768;     // 128 rows x 128 x 2 bytes, two 64-wide halves
constexpr int kTile = kKT * 256;
constexpr int kWarpLoad = 8, kWarpQk = 9, kWarpPv = 10;
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kRescaleLog2 = 8.0f;

// tensor memory columns
constexpr uint32_t kTmS = 0, kTmP = kKT, kTmO = 256;   // + 128 * tile
static_assert(kKT + kKT / 2 <= 128 && kKT % 16 == 0, "S and P of a tile");

// shared memory, from a 1024-byte aligned base
constexpr int kOffQ = 0;                          // 2 tiles
constexpr int kOffKV = 2 * kQTile;                // kStages tiles
constexpr int kOffBars = kOffKV + kStages * kTile;
constexpr int kNumBars = 2 + 2 * kStages + 4 * 2 + 2;
static_assert(kTile % 1024 == 0, "128-byte swizzle");
constexpr int kOffTaddr = kOffBars + kNumBars * 8;
constexpr size_t kSmemAlloc = kOffTaddr + 16 + 1024;
static_assert(kSmemAlloc <= 227 * 1024, "shared memory budget");

struct Bars {
    uint64_t *q_full;                  // [tile]
    uint64_t *kv_full, *kv_empty;      // [kStages]
    uint64_t *s_full, *s_empty;        // [tile] S written / in registers
    uint64_t *p_full, *pv_done;        // [tile]
    uint64_t *mma_done;                // [issuer] its products have retired
};

__device__ __forceinline__ Bars carve_bars(uint8_t *smem)
{
    uint64_t *b = reinterpret_cast<uint64_t *>(smem + kOffBars);
    Bars r;
    r.q_full = b;
    r.kv_full = r.q_full + 2;
    r.kv_empty = r.kv_full + kStages;
    r.s_full = r.kv_empty + kStages;
    r.s_empty = r.s_full + 2;
    r.p_full = r.s_empty + 2;
    r.pv_done = r.p_full + 2;
    r.mma_done = r.pv_done + 2;
    return r;
}

__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, uint32_t *status)
{
    const bool ok = mbar_wait(bar, parity, status);
    return __all_sync(0xffffffffu, ok);
}

// 3-D tiled tensor copy global -> shared (no multicast); x in elements, the
// callers pass 0 or 64 (128 bytes).
__device__ __forceinline__ void tma_tile_3d_g2s(uint32_t dst, const CUtensorMap *map, int32_t x,
                                                int32_t y, int32_t z, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

template <bool BF>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    if constexpr (BF) {
        __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<uint32_t *>(&h);
    } else {
        return pack_half2(lo, hi);
    }
}

// Geometry of one query tile: key tiles jbase .. jbase + ntiles - 1.
struct QTile {
    int q0, pos_hi, ntiles;
};

__device__ __forceinline__ QTile make_qtile(int tile, int tpt, int len, int jbase)
{
    QTile t{tile * tpt, -1, 0};
    if (t.q0 < len) {
        t.pos_hi = min(len, t.q0 + tpt) - 1;
        t.ntiles = t.pos_hi / kKT + 1 - jbase;
    }
    return t;
}

template <bool BF>
__global__ void __launch_bounds__(kThreads, 1)
prompt_attn_kernel(const __grid_constant__ CUtensorMap qmap,
                   const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap, const PromptParams p)
{
    constexpr uint32_t kType = BF ? (1u << 7) | (1u << 10) : 0u;   // A and B format
    constexpr uint32_t kIdescQK = idesc_f16_f32(128, kKT, false) | kType;
    constexpr uint32_t kIdescPV = idesc_f16_f32(128, 128, true) | kType;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const Bars bars = carve_bars(smem);
    uint32_t *taddr_smem = reinterpret_cast<uint32_t *>(smem + kOffTaddr);

    const int pair = gridDim.x - 1 - blockIdx.x;   // longest work first
    const int h = blockIdx.y, b = blockIdx.z;
    const int tok0 = p.cu_seqlens[b];
    // (never past the rows that there are)
    const int len = (int)min((long long)p.cu_seqlens[b + 1], p.total) - tok0;
    const int tpt = p.tokens_per_tile, G = p.group;
    if (tok0 < 0 || 2 * pair * tpt >= len || device_wait_failed(p.status))
        return;
    const int jbase = p.window > 0 ? max(0, 2 * pair * tpt - p.window + 1) / kKT : 0;
    const QTile qt[2] = {make_qtile(2 * pair, tpt, len, jbase),
                         make_qtile(2 * pair + 1, tpt, len, jbase)};
    const int ntiles = max(qt[0].ntiles, qt[1].ntiles);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.q_full[i], 1);
            mbar_init(&bars.s_full[i], 1);
            mbar_init(&bars.s_empty[i], 4);
            mbar_init(&bars.p_full[i], 4);
            mbar_init(&bars.pv_done[i], 1);
        }
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&bars.kv_full[s], 1);
            mbar_init(&bars.kv_empty[s], 1);
        }
        mbar_init(&bars.mma_done[0], 1);
        mbar_init(&bars.mma_done[1], 1);
        fence_mbar_init();
    }
    if (warp == kWarpQk) {
        tmem_alloc(taddr_smem, 512);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *taddr_smem;

    // ring entries in the order the MMAs take them: K(0) K(1) V(0) K(2) V(1) ...
    auto k_entry = [&](int j) { return j == 0 ? 0 : 2 * j - 1; };
    auto v_entry = [&](int j) { return j == ntiles - 1 ? 2 * j + 1 : 2 * j + 2; };

    if (warp == kWarpLoad) {
        // ---------------------------------------------- copy producer --
        const uint32_t qbytes = (uint32_t)(tpt * G) * 256u;
        auto load_q = [&](int x) {
            if (qt[x].ntiles > 0 && lane == 0) {
                mbar_arrive_expect_tx(&bars.q_full[x], qbytes);
                const uint32_t dst = sbase + kOffQ + x * kQTile;
                tma_tile_3d_g2s(dst, &qmap, 0, h * G, tok0 + qt[x].q0, &bars.q_full[x]);
                tma_tile_3d_g2s(dst + kQTile / 2, &qmap, 64, h * G, tok0 + qt[x].q0,
                                &bars.q_full[x]);
            }
        };
        load_q(0);
        int issued = 0;
        for (int i = 0; i < 2 * ntiles; ++i) {
            const int s = i % kStages;
            if (i >= kStages && !warp_wait(&bars.kv_empty[s], ((i - kStages) / kStages) & 1, p.status))
                break;
            // entry i: K for 0 and odd i, V for the others (the last one is a V)
            const bool isv = i > 0 && ((i & 1) == 0 || i == 2 * ntiles - 1);
            const int j = isv ? (i == 2 * ntiles - 1 ? ntiles - 1 : i / 2 - 1) : (i + 1) / 2;
            if (lane == 0) {
                mbar_arrive_expect_tx(&bars.kv_full[s], kTile);
                const CUtensorMap *m = isv ? &vmap : &kmap;
                const uint32_t dst = sbase + kOffKV + s * kTile;
                const int tok = tok0 + (jbase + j) * kKT;
                tma_tile_3d_g2s(dst, m, 0, h, tok, &bars.kv_full[s]);
                tma_tile_3d_g2s(dst + kTile / 2, m, 64, h, tok, &bars.kv_full[s]);
            }
            __syncwarp();
            issued = i + 1;
            if (i == 0)
                load_q(1);
        }
        // every copy lands before shared memory is released (they have long
        // been consumed unless a wait gave up)
        for (int i = max(0, issued - kStages); i < issued; ++i)
            warp_wait(&bars.kv_full[i % kStages], (i / kStages) & 1, nullptr);
        for (int x = 0; x < 2; ++x)
            if (qt[x].ntiles > 0 && (x == 0 || issued > 0))
                warp_wait(&bars.q_full[x], 0, nullptr);
    } else if (warp == kWarpQk) {
        // ------------------------------------------------ Q K^T issuer --
        const uint64_t qd0 = desc_sw128(sbase + kOffQ, 16, 1024);
        const uint64_t kd0 = desc_sw128(sbase + kOffKV, 16, 1024);
        bool ok = true;
        for (int j = 0; ok && j < ntiles; ++j) {
            const int i = k_entry(j), s = i % kStages;
            const uint64_t kd = kd0 + (uint64_t)((s * kTile) >> 4);
            ok = warp_wait(&bars.kv_full[s], (i / kStages) & 1, p.status);
            for (int x = 0; ok && x < 2; ++x) {
                if (j >= qt[x].ntiles)
                    continue;
                // S_x(j - 1) is in registers
                ok = j == 0 ? warp_wait(&bars.q_full[x], 0, p.status)
                            : warp_wait(&bars.s_empty[x], (j - 1) & 1, p.status);
                if (!ok)
                    break;
                tc_fence_after();
                const uint64_t qd = qd0 + (uint64_t)((x * kQTile) >> 4);
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    mma_f16_ss_elect(
                        tmem + kTmS + x * 128,
                        qd + (uint64_t)(((ks >> 2) * (kQTile / 2) + (ks & 3) * 32) >> 4),
                        kd + (uint64_t)(((ks >> 2) * (kTile / 2) + (ks & 3) * 32) >> 4), kIdescQK,
                        ks > 0 ? 1u : 0u);
                mma_commit_elect(&bars.s_full[x]);
            }
            if (ok)
                mma_commit_elect(&bars.kv_empty[s]);
        }
        mma_commit_elect(&bars.mma_done[0]);
        warp_wait(&bars.mma_done[0], 0, p.status);
    } else if (warp == kWarpPv) {
        // --------------------------------------------------- P V issuer --
        const uint64_t vd0 = desc_sw128(sbase + kOffKV, kTile / 2, 1024);
        bool ok = true;
        for (int j = 0; ok && j < ntiles; ++j) {
            const int i = v_entry(j), s = i % kStages;
            const uint64_t vd = vd0 + (uint64_t)((s * kTile) >> 4);
            ok = warp_wait(&bars.kv_full[s], (i / kStages) & 1, p.status);
            const int rows = len - (jbase + j) * kKT;   // of this sequence in the tile
            if (ok && rows < kKT) {
                uint8_t *v = smem + kOffKV + s * kTile;
                const uint4 z = make_uint4(0u, 0u, 0u, 0u);
                for (int o = rows * 128 + lane * 16; o < kTile / 2; o += 512) {
                    *reinterpret_cast<uint4 *>(v + o) = z;
                    *reinterpret_cast<uint4 *>(v + kTile / 2 + o) = z;
                }
                fence_async_smem();
                __syncwarp();
            }
            for (int x = 0; ok && x < 2; ++x) {
                if (j >= qt[x].ntiles)
                    continue;
                ok = warp_wait(&bars.p_full[x], j & 1, p.status);
                if (!ok)
                    break;
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < kKT / 16; ++ks)
                    mma_f16_ts_elect(tmem + kTmO + x * 128, tmem + kTmP + x * 128 + ks * 8,
                                     vd + (uint64_t)((ks * 2048) >> 4), kIdescPV,
                                     (j > 0 || ks > 0) ? 1u : 0u);
                mma_commit_elect(&bars.pv_done[x]);
            }
            if (ok)
                mma_commit_elect(&bars.kv_empty[s]);
        }
        mma_commit_elect(&bars.mma_done[1]);
        warp_wait(&bars.mma_done[1], 0, p.status);
    } else {
        // ------------------------------------------------------ softmax --
        const int x = warp >> 2;
        const int r = tid - 128 * x;         // row == TMEM lane
        const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t ts = tl + kTmS + x * 128, tp = tl + kTmP + x * 128;
        const uint32_t to = tl + kTmO + x * 128;
        const QTile T = qt[x];
        const int pos = T.q0 + r / G;
        const bool valid = r < tpt * G && pos < len && T.ntiles > 0;
        const int lo = p.window > 0 ? pos - p.window + 1 : INT_MIN;
        const int lo_hi = p.window > 0 ? T.pos_hi - p.window + 1 : INT_MIN;
        const float kf = p.scale_log2;   // > 0
        float m_used = -INFINITY, l = 0.0f;   // m in units of the raw scores
        bool ok = true;
        for (int j = 0; j < T.ntiles; ++j) {
            if (!warp_wait(&bars.s_full[x], j & 1, p.status)) {
                ok = false;
                break;
            }
            tc_fence_after();
            float v[kKT];
            {
                uint32_t ua[32], ub[32], uc[16];
                tmem_ld80(ts, ua, ub, uc);
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    v[c] = __uint_as_float(ua[c]);
                    v[32 + c] = __uint_as_float(ub[c]);
                }
#pragma unroll
                for (int c = 0; c < 16; ++c)
                    v[64 + c] = __uint_as_float(uc[c]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&bars.s_empty[x]);
            if (p.negate) {
#pragma unroll
                for (int c = 0; c < kKT; ++c)
                    v[c] = -v[c];
            }
            const int key0 = (jbase + j) * kKT;
            if (key0 + kKT - 1 > T.q0 || key0 < lo_hi) {
#pragma unroll
                for (int c = 0; c < kKT; ++c)
                    if (key0 + c > pos || key0 + c < lo)
                        v[c] = -INFINITY;
            }
            const float mx = max3(max3(max16(v), max16(v + 16), max16(v + 32)), max16(v + 48),
                                  max16(v + 64));
            // P and O are free once P V of the previous tile has completed
            if (j > 0 && !warp_wait(&bars.pv_done[x], (j - 1) & 1, p.status)) {
                ok = false;
                break;
            }
            tc_fence_after();
            // lazy rescale: only when the max grew by more than 2^8
            const bool need = m_used != -INFINITY && (mx - m_used) * kf > kRescaleLog2;
            if (__any_sync(0xffffffffu, need)) {
                const float corr = need ? fast_exp2((m_used - mx) * kf) : 1.0f;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    uint32_t o[16];
                    tmem_ld16(to + 16 * q, o);
#pragma unroll
                    for (int c = 0; c < 16; ++c)
                        o[c] = __float_as_uint(__uint_as_float(o[c]) * corr);
                    tmem_st16(to + 16 * q, o);
                }
                if (need) {
                    l *= corr;
                    m_used = mx;
                }
            }
            if (m_used == -INFINITY)
                m_used = mx;   // first finite max (O is still empty)
            const float nm = m_used == -INFINITY ? 0.0f : -m_used * kf;
            const float2 nm2 = make_float2(nm, nm), kf2 = make_float2(kf, kf);
            float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                             make_float2(0.f, 0.f)};
#pragma unroll
            for (int g = 0; g < kKT / 16; ++g) {
                uint32_t pk[8];
#pragma unroll
                for (int c = 0; c < 16; c += 2) {
                    const int cc = 16 * g + c;
                    const float2 d = __ffma2_rn(make_float2(v[cc], v[cc + 1]), kf2, nm2);
                    const float2 e = make_float2(fast_exp2(d.x), fast_exp2(d.y));
                    acc[(c >> 1) & 3] = __fadd2_rn(acc[(c >> 1) & 3], e);
                    pk[c / 2] = pack2<BF>(e.x, e.y);
                }
                tmem_st8(tp + 8 * g, pk);
            }
            const float2 a = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
            l += a.x + a.y;
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&bars.p_full[x]);
        }

        // ---- epilogue: O / l ----
        const bool have_o =
            ok && T.ntiles > 0 && warp_wait(&bars.pv_done[x], (T.ntiles - 1) & 1, p.status);
        if (have_o)
            tc_fence_after();
        const float f = have_o && l > 0.0f ? 1.0f / l : 0.0f;
        const size_t qrow = (size_t)(tok0 + pos) * p.num_q_heads + (size_t)h * G + r % G;
        uint16_t *dst = p.out + qrow * kHeadDim;
        if (have_o) {   // warp-uniform
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t o[32];
                tmem_ld32(to + 32 * q, o);
                if (valid) {
#pragma unroll
                    for (int c = 0; c < 32; c += 8) {
                        uint4 w;
                        w.x = pack2<BF>(__uint_as_float(o[c]) * f, __uint_as_float(o[c + 1]) * f);
                        w.y = pack2<BF>(__uint_as_float(o[c + 2]) * f, __uint_as_float(o[c + 3]) * f);
                        w.z = pack2<BF>(__uint_as_float(o[c + 4]) * f, __uint_as_float(o[c + 5]) * f);
                        w.w = pack2<BF>(__uint_as_float(o[c + 6]) * f, __uint_as_float(o[c + 7]) * f);
                        *reinterpret_cast<uint4 *>(dst + 32 * q + c) = w;
                    }
                }
            }
            if (valid && p.lse)
                p.lse[qrow] = l > 0.0f ? (m_used * kf + log2f(l)) * kLn2 : -INFINITY;
        }
    }

    __syncthreads();
    if (warp == kWarpQk) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace

cudaError_t launch_prompt_attn(const PromptParams &p, const CUtensorMap &qmap,
                               const CUtensorMap &kmap, const CUtensorMap &vmap,
                               cudaStream_t stream)
{
    auto kern = p.bf16 ? prompt_attn_kernel<true> : prompt_attn_kernel<false>;
    cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemAlloc);
    if (e != cudaSuccess)
        return e;
    const dim3 grid((unsigned)((p.q_tiles + 1) / 2), (unsigned)p.num_kv_heads, (unsigned)p.batch);
    kern<<<grid, kThreads, kSmemAlloc, stream>>>(qmap, kmap, vmap, p);
    return cudaGetLastError();
}

}  // namespace pkvq
