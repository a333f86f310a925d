// Decode attention: the split plan, the merge kernel and the launches (the
// split kernel itself is in decode_split.cuh).
#include "decode_split.cuh"

#include <stdlib.h>

namespace pkvq {
namespace {

// Merge of the split partial states by a separate kernel, one warp per
// output row; programmatic dependent launch lets it start while the split
// kernel's last CTAs finish.  (A variant in which the last CTA of each
// sequence merged its splits itself, found through arrival counters, took
// the same time on the batch-8 x 32K workload and needed a zeroed
// workspace.)
template <int BS>
__global__ void __launch_bounds__(128) decode_merge_kernel(const DecodeParams p)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long gw = (long long)blockIdx.x * 4 + warp;
    const long long total = (long long)p.batch * p.num_kv_heads * p.rows;
    if (gw >= total)
        return;
    const int rr = (int)(gw % p.rows);
    const int h = (int)((gw / p.rows) % p.num_kv_heads);
    const int b = (int)(gw / ((long long)p.rows * p.num_kv_heads));
    // slots first .. first + nsplit - 1 of unit (row group, KV head) y
    const int y = (rr / p.rows_per_cta) * p.num_kv_heads + h;
    MergeRow<16> mr;
    mr.row0 = (size_t)y * p.num_splits * p.rows_per_cta + rr % p.rows_per_cta;
    mr.stride = p.rows_per_cta;
    // The slots of sequence b come from the context lengths, inputs the split
    // kernel does not write: they are found while the split kernel's last
    // CTAs still run, and only the partials wait for its completion.
    const SplitInfo si = find_split<BS>(p, -1, b);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (si.nsplit <= 1)
        return;   // a single split wrote the final row itself
    mr.load(p, si.first, si.nsplit, 0, lane);
    mr.finish(p, si.first, si.nsplit, b, h, rr, lane);
}

}  // namespace

bool decode_plan(int kv_dtype, int batch, int q_len, int num_q_heads, int num_kv_heads,
                 int block_size, int max_context_len, bool weights, DecodePlan *plan)
{
    if (batch <= 0 || q_len <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads)
        return false;
    const int group = num_q_heads / num_kv_heads;
    const int rows = q_len * group;
    // More than 16 rows per KV head (up to 128): the tensor-core kernel, one
    // CTA for all rows, so every code is fetched and converted once; the
    // mma.sync kernel would split the rows into groups that each convert it.
    // (With weights the scores leave through the mma.sync kernel, in row groups.)
    plan->tc = !weights && rows > 16 && rows <= 128;
    plan->nt = plan->tc ? 0 : (rows <= 8 ? 1 : 2);
    plan->rows_per_cta = plan->tc ? rows : 8 * plan->nt;
    plan->row_groups = (rows + plan->rows_per_cta - 1) / plan->rows_per_cta;
    const int max_blocks = (max_context_len + block_size - 1) / block_size;
    const int units = num_kv_heads * plan->row_groups;   // grid y: (row group, KV head)
    // splits: tensor-core kernel in whole 64-key tiles, at least 256 keys;
    // mma.sync kernel at least kMinBlocksPerWarp blocks per warp
    // (block-scaled formats and calls with weights: one loop iteration per warp, 2
    // blocks of 16 tokens or one larger; a short sequence then takes more CTAs)
    const bool fine = weights || kv_has_block_scale(kv_dtype);
    const int min_blocks = plan->tc ? 256 / block_size
                           : !fine  ? kWarps * kMinBlocksPerWarp
                                    : kWarps * (block_size == 16 ? 2 : 1);
    plan->split_min_blocks = min_blocks;
    plan->split_gran = plan->tc ? 64 / block_size : 1;
    // C CTA slots per unit, at most `ctas_per_sm` CTAs on every SM (3, or
    // what fits), all resident in one wave, each slot given about the same
    // number of blocks on the device.  Rounding the count up instead would
    // put one more CTA on some SMs, and those SMs' CTAs would all finish last
    // (a memory-bound CTA gets a share of its SM's bandwidth); more resident
    // CTAs keep more copies in flight.  At least one slot per sequence, and
    // no more slots than splits of kMinBlocksPerWarp blocks per warp.
    // PKVQ_DECODE_CTAS_PER_SM (1..16) replaces the target as given, even
    // beyond what fits in one wave.
    // (the tensor-core kernel takes most of an SM's shared memory: one CTA)
    int ctas_per_sm =
        plan->tc ? 1
                 : min(3, weights ? weights_split_occupancy(kv_dtype, plan->nt, block_size)
                                  : split_occupancy_any<false>(kv_dtype, plan->nt, block_size));
    if (const char *env = getenv("PKVQ_DECODE_CTAS_PER_SM")) {
        const int v = atoi(env);
        if (v >= 1 && v <= 16)
            ctas_per_sm = v;
    }
    const long long target = (long long)ctas_per_sm * device_sm_count();
    long long C = max((long long)batch, target / units);
    const long long useful = (long long)batch * max(1, max_blocks / min_blocks);
    C = min(C, max((long long)batch, useful));
    if (C > (1LL << 30))
        return false;
    plan->num_splits = (int)C;
    // the split every slot gets when all sequences hold max_context_len tokens
    plan->uniform_bpc = split_blocks((long long)batch * max_blocks, (int)C, batch, max_blocks,
                                     plan->split_min_blocks, plan->split_gran);
    plan->uniform_splits = max(1, (max_blocks + plan->uniform_bpc - 1) / plan->uniform_bpc);
    // Spread: verify 4 x 64K (ragged) 79.4 -> 76.9 us, 1 x 1K 13.9 -> 13.2 us, 8 x
    // 32K unchanged at 55.3 us; with weights 8 x 16K 42.8 -> 45.0 us, so not there.
    // (The older formats keep the partition, and so the bits, that they had.)
    plan->spread = !weights && kv_has_block_scale(kv_dtype);
    plan->uniform_more = 0;
    plan->uniform_bpc_more = plan->uniform_bpc;
    if (plan->spread && max_blocks > 0) {
        const int us = plan->uniform_splits;
        if (spread_more(max_blocks, us, min_blocks))
            plan->uniform_more = (int)min((long long)batch, C - (long long)us * batch);
        plan->uniform_bpc_more = spread_blocks(max_blocks, us + 1, plan->split_gran);
        plan->uniform_bpc = spread_blocks(max_blocks, us, plan->split_gran);
    }
    const size_t partials = C > batch ? (size_t)units * C * plan->rows_per_cta *
                                            (kHeadDim + 2) * sizeof(float)
                                      : 0;
    plan->workspace_bytes = partials;
    if (weights) {
        // [partials, always with the (max, sum) states][scores]
        plan->state_bytes = (size_t)units * C * plan->rows_per_cta * (kHeadDim + 2) * sizeof(float);
        plan->score_rows = rows <= 2 ? rows : (rows + 3) / 4 * 4;
        plan->score_keys = max(1, max_blocks) * block_size;
        plan->workspace_bytes = plan->state_bytes + (size_t)batch * num_kv_heads *
                                                        plan->score_keys * plan->score_rows *
                                                        sizeof(float);
    }
    return true;
}

cudaError_t launch_decode(const DecodeParams &p, const DecodePlan &plan, int kv_dtype,
                          const CUtensorMap &kmap, const CUtensorMap &vmap, cudaStream_t stream)
{
    cudaError_t e;
    if (plan.tc)
        e = launch_decode_tc(p, kv_dtype, kmap, vmap, stream);
    else
        e = launch_split_any<false>(kv_dtype, plan.nt, p, kmap, vmap, stream);
    if (e != cudaSuccess || p.num_splits <= p.batch)
        return e;   // one slot per sequence: every CTA wrote final rows
    const long long rows_total = (long long)p.batch * p.num_kv_heads * p.rows;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((rows_total + 3) / 4));
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = 0;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    switch (p.block_size) {
    case 16: return cudaLaunchKernelEx(&cfg, decode_merge_kernel<16>, p);
    case 32: return cudaLaunchKernelEx(&cfg, decode_merge_kernel<32>, p);
    case 64: return cudaLaunchKernelEx(&cfg, decode_merge_kernel<64>, p);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace pkvq
