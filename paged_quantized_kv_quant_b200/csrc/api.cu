// C ABI of libpkvq.so: argument validation, tensor-map setup and dispatch.
// Every check happens on the host before any launch; nothing here allocates
// device memory or synchronizes the host with the device (except
// pkvq_device_status, a diagnostic).
#include "../../include/pkvq.h"
#include "common.cuh"
#include "internal.h"

#include <cudaTypedefs.h>
#include <math.h>
#include <mutex>
#include <stdio.h>
#include <stdlib.h>

namespace pkvq {

__device__ uint32_t g_status_word;

namespace {

constexpr int kMaxDevices = 64;
constexpr int kMaxGridYZ = 65535;   // CUDA's limit of a grid's y and z

uint32_t *status_ptr()
{
    static uint32_t *ptrs[kMaxDevices] = {};
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices)
        return nullptr;
    std::lock_guard<std::mutex> lock(mu);
    if (!ptrs[dev]) {
        void *p = nullptr;
        if (cudaGetSymbolAddress(&p, g_status_word) != cudaSuccess)
            return nullptr;
        ptrs[dev] = static_cast<uint32_t *>(p);
    }
    return ptrs[dev];
}

bool aligned16(const void *p)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return fn;
}

pkvq_status check_cache(const pkvq_cache *c)
{
    if (!c || !c->k_cache || !c->v_cache)
        return PKVQ_ERR_INVALID_ARG;
    if (c->dtype != PKVQ_KV_FP8_E4M3 && c->dtype != PKVQ_KV_INT8 &&
        c->dtype != PKVQ_KV_FP8_E5M2 && c->dtype != PKVQ_KV_FP16 &&
        c->dtype != PKVQ_KV_INT8_BLOCK && c->dtype != PKVQ_KV_E4M3_BLOCK)
        return PKVQ_ERR_UNSUPPORTED;
    if (c->head_dim != kHeadDim)
        return PKVQ_ERR_UNSUPPORTED;
    if (c->block_size != 16 && c->block_size != 32 && c->block_size != 64)
        return PKVQ_ERR_UNSUPPORTED;
    if (c->num_blocks <= 0 || c->num_kv_heads <= 0)
        return PKVQ_ERR_INVALID_ARG;
    // tensor-map row coordinates are int32
    if ((long long)c->num_blocks * c->num_kv_heads * c->block_size >= (1LL << 31))
        return PKVQ_ERR_UNSUPPORTED;
    if (kv_has_head_scale(c->dtype)) {
        if (!c->k_scale || !c->v_scale)
            return PKVQ_ERR_INVALID_ARG;
    } else if (c->dtype == PKVQ_KV_INT8) {
        if (!c->k_scale_tok || !c->v_scale_tok)
            return PKVQ_ERR_INVALID_ARG;
        if (!aligned16(c->k_scale_tok) || !aligned16(c->v_scale_tok))
            return PKVQ_ERR_MISALIGNED;
    } else if (kv_has_block_scale(c->dtype)) {
        if (!c->k_scale_blk || !c->v_scale_blk)
            return PKVQ_ERR_INVALID_ARG;
        if (!aligned16(c->k_scale_blk) || !aligned16(c->v_scale_blk))
            return PKVQ_ERR_MISALIGNED;
    }
    if (!aligned16(c->k_cache) || !aligned16(c->v_cache))
        return PKVQ_ERR_MISALIGNED;
    return PKVQ_OK;
}

pkvq_status cache_maps(const pkvq_cache *c, CUtensorMap *km, CUtensorMap *vm)
{
    const uint64_t rows = (uint64_t)c->num_blocks * c->num_kv_heads * c->block_size;
    const int row_bytes = kHeadDim * kv_elem_bytes(c->dtype);
    if (!make_cache_tensor_map(km, c->k_cache, rows, c->block_size, row_bytes) ||
        !make_cache_tensor_map(vm, c->v_cache, rows, c->block_size, row_bytes))
        return PKVQ_ERR_CUDA;
    return PKVQ_OK;
}

int scale_stride(const pkvq_cache *c)
{
    return c->scale_per_layer ? 0 : 1;
}

thread_local char t_last_error[256] = "";

pkvq_status from_cuda(cudaError_t e, const char *what = "launch")
{
    if (e == cudaSuccess)
        return PKVQ_OK;
    snprintf(t_last_error, sizeof(t_last_error), "%s: %s (%d)", what, cudaGetErrorString(e),
             (int)e);
    return PKVQ_ERR_CUDA;
}

constexpr float kLog2e = 1.4426950408889634f;

}  // namespace

bool make_cache_tensor_map(CUtensorMap *map, const void *base, uint64_t rows, int box_rows,
                           int row_bytes)
{
    auto fn = encode_fn();
    if (!fn)
        return false;
    cuuint64_t dims[2] = {(cuuint64_t)row_bytes, rows};
    cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
    cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides,
                    box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

bool make_rows_tensor_map(CUtensorMap *map, const void *base, bool bf16, int64_t tokens,
                          int heads, int64_t token_stride, int64_t head_stride, int box_heads,
                          int box_tokens)
{
    auto fn = encode_fn();
    if (!fn)
        return false;
    cuuint64_t dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)heads, (cuuint64_t)tokens};
    cuuint64_t strides[2] = {(cuuint64_t)head_stride * 2, (cuuint64_t)token_stride * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
              const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int device_sm_count()
{
    static int counts[kMaxDevices] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices)
        return 148;
    if (!counts[dev]) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
            n = 148;
        counts[dev] = n;
    }
    return counts[dev];
}

}  // namespace pkvq

using namespace pkvq;

extern "C" {

const char *pkvq_last_error(void)
{
    return t_last_error;
}

const char *pkvq_version(void)
{
    return "0.2.0";
}

const char *pkvq_status_string(pkvq_status s)
{
    switch (s) {
    case PKVQ_OK: return "ok";
    case PKVQ_ERR_INVALID_ARG: return "invalid argument";
    case PKVQ_ERR_UNSUPPORTED: return "unsupported configuration";
    case PKVQ_ERR_MISALIGNED: return "pointer not 16-byte aligned";
    case PKVQ_ERR_WORKSPACE_TOO_SMALL: return "workspace too small";
    case PKVQ_ERR_DEVICE: return "device-side check failed";
    case PKVQ_ERR_CUDA: return "CUDA runtime error";
    }
    return "unknown status";
}

pkvq_status pkvq_device_status(uint32_t *status_out, int32_t clear)
{
    if (!status_out)
        return PKVQ_ERR_INVALID_ARG;
    uint32_t *p = status_ptr();
    if (!p)
        return PKVQ_ERR_CUDA;
    if (cudaMemcpy(status_out, p, sizeof(uint32_t), cudaMemcpyDeviceToHost) != cudaSuccess)
        return PKVQ_ERR_CUDA;
    if (clear && cudaMemset(p, 0, sizeof(uint32_t)) != cudaSuccess)
        return PKVQ_ERR_CUDA;
    return PKVQ_OK;
}

pkvq_status pkvq_kv_write_quant(const pkvq_cache *cache, const void *k, const void *v,
                                const int32_t *slot_mapping, int32_t num_tokens, void *stream)
{
    pkvq_status st = check_cache(cache);
    if (st != PKVQ_OK)
        return st;
    if (kv_has_block_scale(cache->dtype))
        return PKVQ_ERR_UNSUPPORTED;   // pkvq_kv_write_block_quant
    if (num_tokens < 0)
        return PKVQ_ERR_INVALID_ARG;
    if (num_tokens == 0)
        return PKVQ_OK;
    if (!k || !v || !slot_mapping)
        return PKVQ_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v))
        return PKVQ_ERR_MISALIGNED;
    KvWriteParams p{};
    p.k_cache = static_cast<uint8_t *>(cache->k_cache);
    p.v_cache = static_cast<uint8_t *>(cache->v_cache);
    p.k_scale = cache->k_scale;
    p.v_scale = cache->v_scale;
    p.scale_stride = scale_stride(cache);
    p.k_scale_tok = static_cast<uint16_t *>(cache->k_scale_tok);
    p.v_scale_tok = static_cast<uint16_t *>(cache->v_scale_tok);
    p.k = static_cast<const __half *>(k);
    p.v = static_cast<const __half *>(v);
    p.slot_mapping = slot_mapping;
    p.num_tokens = num_tokens;
    p.num_kv_heads = cache->num_kv_heads;
    p.num_blocks = cache->num_blocks;
    p.block_size = cache->block_size;
    p.status = status_ptr();
    if (!p.status)
        return PKVQ_ERR_CUDA;
    return from_cuda(launch_kv_write_quant(p, cache->dtype, static_cast<cudaStream_t>(stream)));
}

namespace {

// Two warps for each 16 rows of every block and head that the call may touch,
// within CUDA's limit of blocks in a grid.
bool block_write_grid_fits(const pkvq_cache *cache, int32_t batch, int32_t max_new_len)
{
    const long long touched =
        ((long long)max_new_len + cache->block_size - 2) / cache->block_size + 1;
    const long long units = touched * batch;
    return units < (1LL << 31) && cache->num_kv_heads <= kMaxGridYZ &&
           units * cache->num_kv_heads * (cache->block_size / 16) < (1LL << 33) - 8;
}

KvWriteBlockParams block_write_params(const pkvq_cache *cache, const void *k, const void *v,
                                      int64_t num_tokens, const int32_t *cu_seqlens_new,
                                      const int32_t *block_table, int32_t max_blocks_per_seq,
                                      const int32_t *context_lens, int32_t batch,
                                      int32_t max_new_len, uint32_t *status)
{
    KvWriteBlockParams p{};
    p.k_cache = static_cast<uint8_t *>(cache->k_cache);
    p.v_cache = static_cast<uint8_t *>(cache->v_cache);
    p.k_scale_blk = cache->k_scale_blk;
    p.v_scale_blk = cache->v_scale_blk;
    p.k = static_cast<const __half *>(k);
    p.v = static_cast<const __half *>(v);
    p.num_tokens = num_tokens;
    p.cu_seqlens_new = cu_seqlens_new;
    p.block_table = block_table;
    p.context_lens = context_lens;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.batch = batch;
    p.max_new_len = p.q_len = max_new_len;
    p.num_kv_heads = cache->num_kv_heads;
    p.num_blocks = cache->num_blocks;
    p.block_size = cache->block_size;
    p.status = status;
    return p;
}

}  // namespace

pkvq_status pkvq_kv_write_block_quant(const pkvq_cache *cache, const void *k, const void *v,
                                      int64_t num_tokens, const int32_t *cu_seqlens_new,
                                      const int32_t *block_table, int32_t max_blocks_per_seq,
                                      const int32_t *context_lens, int32_t batch,
                                      int32_t max_new_len, void *stream)
{
    pkvq_status st = check_cache(cache);
    if (st != PKVQ_OK)
        return st;
    if (!kv_has_block_scale(cache->dtype))
        return PKVQ_ERR_UNSUPPORTED;   // pkvq_kv_write_quant
    if (batch < 0 || max_new_len < 0 || max_blocks_per_seq < 0 || num_tokens < 0)
        return PKVQ_ERR_INVALID_ARG;
    if (batch == 0 || max_new_len == 0 || num_tokens == 0)
        return PKVQ_OK;
    if (!k || !v || !cu_seqlens_new || !block_table || !context_lens)
        return PKVQ_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v))
        return PKVQ_ERR_MISALIGNED;
    if (!block_write_grid_fits(cache, batch, max_new_len))
        return PKVQ_ERR_UNSUPPORTED;
    uint32_t *status = status_ptr();
    if (!status)
        return PKVQ_ERR_CUDA;
    return from_cuda(launch_kv_write_block(
        block_write_params(cache, k, v, num_tokens, cu_seqlens_new, block_table,
                           max_blocks_per_seq, context_lens, batch, max_new_len, status),
        cache->dtype, static_cast<cudaStream_t>(stream)));
}

size_t pkvq_decode_workspace_bytes(int32_t batch, int32_t q_len, int32_t num_q_heads,
                                   int32_t max_context_len, const pkvq_cache *cache)
{
    if (check_cache(cache) != PKVQ_OK || batch <= 0 || q_len <= 0 || q_len > 16 ||
        max_context_len < 0 || num_q_heads <= 0 || num_q_heads % cache->num_kv_heads)
        return 0;
    DecodePlan plan;
    if (!decode_plan(cache->dtype, batch, q_len, num_q_heads, cache->num_kv_heads, cache->block_size,
                     max_context_len, false, &plan))
        return 0;
    return plan.workspace_bytes;
}

size_t pkvq_decode_weights_workspace_bytes(int32_t batch, int32_t q_len, int32_t num_q_heads,
                                           int32_t max_context_len, const pkvq_cache *cache)
{
    if (check_cache(cache) != PKVQ_OK || batch <= 0 || q_len <= 0 || q_len > 16 ||
        max_context_len < 0 || num_q_heads <= 0 || num_q_heads % cache->num_kv_heads ||
        num_q_heads / cache->num_kv_heads > 16)
        return 0;
    DecodePlan plan;
    if (!decode_plan(cache->dtype, batch, q_len, num_q_heads, cache->num_kv_heads, cache->block_size,
                     max_context_len, true, &plan))
        return 0;
    return plan.workspace_bytes;
}

pkvq_status pkvq_paged_attn_decode(const pkvq_cache *cache, const void *q, void *out,
                                   float *lse_out, const int32_t *block_table,
                                   int32_t max_blocks_per_seq, const int32_t *context_lens,
                                   int32_t batch, int32_t q_len, int32_t num_q_heads,
                                   int32_t max_context_len, float softmax_scale,
                                   void *workspace, size_t workspace_bytes, void *stream)
{
    return pkvq_paged_attn_decode_ex(cache, q, out, lse_out, block_table, max_blocks_per_seq,
                                     context_lens, batch, q_len, num_q_heads, max_context_len,
                                     softmax_scale, nullptr, workspace, workspace_bytes, stream);
}

namespace {

// Decode, optionally appending the step's new tokens (k_new / v_new: the
// keys and values of each sequence's last q_len positions) first.
pkvq_status decode_impl(const pkvq_cache *cache, const void *k_new, const void *v_new,
                        const void *q, void *out, float *lse_out, const int32_t *block_table,
                        int32_t max_blocks_per_seq, const int32_t *context_lens, int32_t batch,
                        int32_t q_len, int32_t num_q_heads, int32_t max_context_len,
                        float softmax_scale, const pkvq_attn_opts *opts, void *workspace,
                        size_t workspace_bytes, void *stream, float *weights = nullptr,
                        int64_t weight_stride = 0)
{
    if (opts && opts->sliding_window < 0)
        return PKVQ_ERR_INVALID_ARG;
    pkvq_status st = check_cache(cache);
    if (st != PKVQ_OK)
        return st;
    if (batch < 0 || q_len < 1 || q_len > 16 || num_q_heads <= 0 || max_context_len < 0 ||
        max_blocks_per_seq < 0)
        return PKVQ_ERR_INVALID_ARG;
    if (num_q_heads % cache->num_kv_heads)
        return PKVQ_ERR_INVALID_ARG;
    const int group = num_q_heads / cache->num_kv_heads;
    if (group > 16)
        return PKVQ_ERR_UNSUPPORTED;
    if (!isfinite(softmax_scale))
        return PKVQ_ERR_INVALID_ARG;
    if (batch == 0)
        return PKVQ_OK;
    if (!q || !out || !block_table || !context_lens)
        return PKVQ_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(out))
        return PKVQ_ERR_MISALIGNED;
    if ((long long)max_blocks_per_seq * cache->block_size < max_context_len)
        return PKVQ_ERR_INVALID_ARG;
    DecodePlan plan;
    if (!decode_plan(cache->dtype, batch, q_len, num_q_heads, cache->num_kv_heads, cache->block_size,
                     max_context_len, weights != nullptr, &plan))
        return PKVQ_ERR_INVALID_ARG;
    if (plan.workspace_bytes > 0) {
        if (!workspace || workspace_bytes < plan.workspace_bytes)
            return PKVQ_ERR_WORKSPACE_TOO_SMALL;
        if (!aligned16(workspace))
            return PKVQ_ERR_MISALIGNED;
    }
    CUtensorMap km, vm;
    st = cache_maps(cache, &km, &vm);
    if (st != PKVQ_OK)
        return st;
    DecodeParams p{};
    p.k_cache = static_cast<const uint8_t *>(cache->k_cache);
    p.v_cache = static_cast<const uint8_t *>(cache->v_cache);
    const bool head_scale = kv_has_head_scale(cache->dtype);
    p.k_scale = head_scale ? cache->k_scale : nullptr;
    p.v_scale = head_scale ? cache->v_scale : nullptr;
    p.scale_stride = scale_stride(cache);
    p.k_scale_tok = static_cast<const uint16_t *>(cache->k_scale_tok);
    p.v_scale_tok = static_cast<const uint16_t *>(cache->v_scale_tok);
    // (the last fields of pkvq_cache are read for these formats only)
    const bool blk_scale = kv_has_block_scale(cache->dtype);
    p.k_scale_blk = blk_scale ? cache->k_scale_blk : nullptr;
    p.v_scale_blk = blk_scale ? cache->v_scale_blk : nullptr;
    p.window = opts ? opts->sliding_window : 0;
    p.query_pos = opts ? opts->query_pos : nullptr;
    p.q = static_cast<const __half *>(q);
    p.out = static_cast<__half *>(out);
    p.lse = lse_out;
    p.block_table = block_table;
    p.context_lens = context_lens;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.batch = batch;
    p.q_len = q_len;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = cache->num_kv_heads;
    p.group = group;
    p.num_blocks = cache->num_blocks;
    p.block_size = cache->block_size;
    p.rows = q_len * group;
    p.rows_per_cta = plan.rows_per_cta;
    p.row_groups = plan.row_groups;
    p.num_splits = plan.num_splits;
    p.uniform_splits = plan.uniform_splits;
    p.uniform_bpc = plan.uniform_bpc;
    p.uniform_more = plan.uniform_more;
    p.uniform_bpc_more = plan.uniform_bpc_more;
    p.spread = plan.spread;
    p.split_min_blocks = plan.split_min_blocks;
    p.split_gran = plan.split_gran;
    p.scale_log2 = softmax_scale * kLog2e;
    // workspace: [partial O][partial (m, l)]
    float *ws = static_cast<float *>(workspace);
    const size_t n_rows_ws = (size_t)cache->num_kv_heads * plan.row_groups * plan.num_splits *
                             plan.rows_per_cta;
    p.ws_o = plan.workspace_bytes ? ws : nullptr;
    p.ws_ml = plan.workspace_bytes ? ws + n_rows_ws * kHeadDim : nullptr;
    p.status = status_ptr();
    if (!p.status)
        return PKVQ_ERR_CUDA;
    cudaStream_t st_ = static_cast<cudaStream_t>(stream);
    if (weights) {
        p.scores = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + plan.state_bytes);
        p.weights = weights;
        p.weight_stride = weight_stride;
        p.score_keys = plan.score_keys;
        p.score_rows = plan.score_rows;
        return from_cuda(launch_decode_weights(p, plan, cache->dtype, km, vm, st_));
    }
    if (k_new) {
        if (kv_has_block_scale(cache->dtype)) {
            // a block's scale follows from all its new tokens: the block
            // write kernel runs just before
            if (!block_write_grid_fits(cache, batch, q_len))
                return PKVQ_ERR_UNSUPPORTED;
            const cudaError_t e = launch_kv_write_block(
                block_write_params(cache, k_new, v_new, (int64_t)batch * q_len, nullptr, block_table,
                                   max_blocks_per_seq, context_lens, batch, q_len, p.status),
                cache->dtype, st_);
            if (e != cudaSuccess)
                return from_cuda(e);
        } else if (plan.tc) {
            // the tensor-core kernel reads whole tiles through one copy ring:
            // the new tokens are written by the KV write kernel just before
            KvWriteParams w{};
            w.k_cache = static_cast<uint8_t *>(cache->k_cache);
            w.v_cache = static_cast<uint8_t *>(cache->v_cache);
            w.k_scale = cache->k_scale;
            w.v_scale = cache->v_scale;
            w.scale_stride = scale_stride(cache);
            w.k_scale_tok = static_cast<uint16_t *>(cache->k_scale_tok);
            w.v_scale_tok = static_cast<uint16_t *>(cache->v_scale_tok);
            w.k = static_cast<const __half *>(k_new);
            w.v = static_cast<const __half *>(v_new);
            w.slot_mapping = nullptr;
            w.block_table = block_table;
            w.context_lens = context_lens;
            w.max_blocks_per_seq = max_blocks_per_seq;
            w.q_len = q_len;
            w.num_tokens = batch * q_len;
            w.num_kv_heads = cache->num_kv_heads;
            w.num_blocks = cache->num_blocks;
            w.block_size = cache->block_size;
            w.status = p.status;
            const cudaError_t e = launch_kv_write_quant(w, cache->dtype, st_);
            if (e != cudaSuccess)
                return from_cuda(e);
        } else {
            // the split kernel: each CTA writes the new tokens of its blocks
            p.k_new = static_cast<const __half *>(k_new);
            p.v_new = static_cast<const __half *>(v_new);
        }
    }
    return from_cuda(launch_decode(p, plan, cache->dtype, km, vm, st_));
}

}  // namespace

pkvq_status pkvq_paged_attn_decode_ex(const pkvq_cache *cache, const void *q, void *out,
                                      float *lse_out, const int32_t *block_table,
                                      int32_t max_blocks_per_seq, const int32_t *context_lens,
                                      int32_t batch, int32_t q_len, int32_t num_q_heads,
                                      int32_t max_context_len, float softmax_scale,
                                      const pkvq_attn_opts *opts, void *workspace,
                                      size_t workspace_bytes, void *stream)
{
    return decode_impl(cache, nullptr, nullptr, q, out, lse_out, block_table,
                       max_blocks_per_seq, context_lens, batch, q_len, num_q_heads,
                       max_context_len, softmax_scale, opts, workspace, workspace_bytes, stream);
}

pkvq_status pkvq_paged_attn_decode_append(const pkvq_cache *cache, const void *k_new,
                                          const void *v_new, const void *q, void *out,
                                          float *lse_out, const int32_t *block_table,
                                          int32_t max_blocks_per_seq,
                                          const int32_t *context_lens, int32_t batch,
                                          int32_t q_len, int32_t num_q_heads,
                                          int32_t max_context_len, float softmax_scale,
                                          const pkvq_attn_opts *opts, void *workspace,
                                          size_t workspace_bytes, void *stream)
{
    if (opts && opts->query_pos)
        return PKVQ_ERR_INVALID_ARG;   // the new tokens are the last q_len positions
    if (batch > 0) {
        if (!k_new || !v_new)
            return PKVQ_ERR_INVALID_ARG;
        if (!aligned16(k_new) || !aligned16(v_new))
            return PKVQ_ERR_MISALIGNED;
    }
    return decode_impl(cache, k_new, v_new, q, out, lse_out, block_table, max_blocks_per_seq,
                       context_lens, batch, q_len, num_q_heads, max_context_len, softmax_scale,
                       opts, workspace, workspace_bytes, stream);
}

pkvq_status pkvq_paged_attn_decode_weights(const pkvq_cache *cache, const void *q, void *out,
                                           float *lse_out, const int32_t *block_table,
                                           int32_t max_blocks_per_seq,
                                           const int32_t *context_lens, int32_t batch,
                                           int32_t q_len, int32_t num_q_heads,
                                           int32_t max_context_len, float softmax_scale,
                                           const pkvq_attn_opts *opts, float *weights,
                                           int64_t weight_stride, void *workspace,
                                           size_t workspace_bytes, void *stream)
{
    if (batch > 0 && (!weights || weight_stride < max_context_len))
        return PKVQ_ERR_INVALID_ARG;
    if (cache && (batch > kMaxGridYZ || cache->num_kv_heads > kMaxGridYZ))
        return PKVQ_ERR_UNSUPPORTED;   // the weights kernel's grid
    return decode_impl(cache, nullptr, nullptr, q, out, lse_out, block_table, max_blocks_per_seq,
                       context_lens, batch, q_len, num_q_heads, max_context_len, softmax_scale,
                       opts, workspace, workspace_bytes, stream, weights, weight_stride);
}

pkvq_status pkvq_kv_evict(const pkvq_cache *cache, const float *weights, int64_t weight_stride,
                          const int32_t *block_table, int32_t max_blocks_per_seq,
                          const int32_t *context_lens, int32_t batch, int32_t budget,
                          int32_t num_sink, int32_t num_recent, const int32_t *dst_block_table,
                          int32_t dst_max_blocks, int32_t *keep_out, int32_t *new_context_lens,
                          float *weights_out, int64_t weight_out_stride, void *stream)
{
    pkvq_status st = check_cache(cache);
    if (st != PKVQ_OK)
        return st;
    if (batch < 0 || budget < 1 || num_sink < 0 || num_recent < 0 ||
        (long long)num_sink + num_recent > budget || max_blocks_per_seq < 0 ||
        dst_max_blocks < 0 || (long long)dst_max_blocks * cache->block_size < budget ||
        weight_stride < 0 || (weights_out && weight_out_stride < budget))
        return PKVQ_ERR_INVALID_ARG;
    if (batch > kMaxGridYZ || cache->num_kv_heads > kMaxGridYZ || budget > (1 << 30))
        return PKVQ_ERR_UNSUPPORTED;   // the launch grid; 32-bit positions
    if (batch == 0)
        return PKVQ_OK;
    if (!weights || !block_table || !context_lens || !dst_block_table || !keep_out ||
        !new_context_lens || new_context_lens == context_lens)
        return PKVQ_ERR_INVALID_ARG;
    if (weights_out) {   // the two accumulators must not overlap
        const uintptr_t rows = (uintptr_t)batch * (uintptr_t)cache->num_kv_heads;
        const uintptr_t a = reinterpret_cast<uintptr_t>(weights);
        const uintptr_t b = reinterpret_cast<uintptr_t>(weights_out);
        if (a < b + rows * (uintptr_t)weight_out_stride * 4 &&
            b < a + rows * (uintptr_t)weight_stride * 4)
            return PKVQ_ERR_INVALID_ARG;
    }
    EvictParams p{};
    p.k_cache = static_cast<uint8_t *>(cache->k_cache);
    p.v_cache = static_cast<uint8_t *>(cache->v_cache);
    p.k_scale_tok = static_cast<uint16_t *>(cache->k_scale_tok);
    p.v_scale_tok = static_cast<uint16_t *>(cache->v_scale_tok);
    const bool blk_scale = kv_has_block_scale(cache->dtype);
    p.k_scale_blk = blk_scale ? cache->k_scale_blk : nullptr;
    p.v_scale_blk = blk_scale ? cache->v_scale_blk : nullptr;
    p.weights = weights;
    p.weight_stride = weight_stride;
    p.weights_out = weights_out;
    p.weight_out_stride = weight_out_stride;
    p.block_table = block_table;
    p.context_lens = context_lens;
    p.dst_block_table = dst_block_table;
    p.keep = keep_out;
    p.new_context_lens = new_context_lens;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.dst_max_blocks = dst_max_blocks;
    p.block_size = cache->block_size;
    p.batch = batch;
    p.num_kv_heads = cache->num_kv_heads;
    p.num_blocks = cache->num_blocks;
    p.budget = budget;
    p.sink = num_sink;
    p.recent = num_recent;
    p.status = status_ptr();
    if (!p.status)
        return PKVQ_ERR_CUDA;
    return from_cuda(launch_evict(p, cache->dtype, cache->block_size,
                                  static_cast<cudaStream_t>(stream)));
}

pkvq_status pkvq_prompt_attn(const pkvq_prompt *t, void *out, float *lse_out,
                             const int32_t *cu_seqlens, int32_t batch, int32_t max_len,
                             float softmax_scale, int32_t sliding_window, void *stream)
{
    if (!t || batch < 0 || max_len < 0 || t->total < 0 || t->num_q_heads <= 0 ||
        t->num_kv_heads <= 0 || t->num_q_heads % t->num_kv_heads || sliding_window < 0 ||
        !isfinite(softmax_scale))
        return PKVQ_ERR_INVALID_ARG;
    const int group = t->num_q_heads / t->num_kv_heads;
    if (t->head_dim != kHeadDim || (t->dtype != PKVQ_FP16 && t->dtype != PKVQ_BF16) ||
        group > 128 || batch > kMaxGridYZ || t->num_kv_heads > kMaxGridYZ)
        return PKVQ_ERR_UNSUPPORTED;
    if (batch == 0 || max_len == 0 || t->total == 0)
        return PKVQ_OK;
    if (!t->q || !t->k || !t->v || !out || !cu_seqlens)
        return PKVQ_ERR_INVALID_ARG;
    const void *base[3] = {t->q, t->k, t->v};
    const int64_t ts[3] = {t->q_token_stride, t->k_token_stride, t->v_token_stride};
    const int64_t hs[3] = {t->q_head_stride, t->k_head_stride, t->v_head_stride};
    if (!aligned16(out))
        return PKVQ_ERR_MISALIGNED;
    for (int i = 0; i < 3; ++i) {
        // rows are 128 contiguous elements; a stride of at most 2^40 bytes
        if (ts[i] < kHeadDim || hs[i] < kHeadDim || ts[i] >= (1LL << 38) || hs[i] >= (1LL << 38))
            return PKVQ_ERR_INVALID_ARG;
        if (!aligned16(base[i]) || ts[i] % 8 || hs[i] % 8)
            return PKVQ_ERR_MISALIGNED;
    }
    const bool bf16 = t->dtype == PKVQ_BF16;
    PromptParams p{};
    p.tokens_per_tile = 128 / group;
    CUtensorMap m[3];
    for (int i = 0; i < 3; ++i)
        if (!make_rows_tensor_map(&m[i], base[i], bf16, t->total,
                                  i == 0 ? t->num_q_heads : t->num_kv_heads, ts[i], hs[i],
                                  i == 0 ? group : 1, i == 0 ? p.tokens_per_tile : kPromptKeys))
            return PKVQ_ERR_CUDA;
    p.out = static_cast<uint16_t *>(out);
    p.lse = lse_out;
    p.cu_seqlens = cu_seqlens;
    p.total = t->total;
    p.batch = batch;
    p.num_q_heads = t->num_q_heads;
    p.num_kv_heads = t->num_kv_heads;
    p.group = group;
    p.q_tiles = (int)(((long long)max_len + p.tokens_per_tile - 1) / p.tokens_per_tile);
    p.window = sliding_window;
    // a scale of 0 becomes one whose scores all round to 0, so that a masked
    // score (-inf) stays one
    const float s = softmax_scale == 0.0f ? 1e-30f : softmax_scale;
    p.scale_log2 = fabsf(s) * kLog2e;
    p.negate = s < 0.0f;
    p.bf16 = bf16;
    p.status = status_ptr();
    if (!p.status)
        return PKVQ_ERR_CUDA;
    return from_cuda(launch_prompt_attn(p, m[0], m[1], m[2], static_cast<cudaStream_t>(stream)));
}

pkvq_status pkvq_paged_attn_prefill(const pkvq_cache *cache, const void *q, void *out,
                                    float *lse_out, const int32_t *cu_seqlens_q,
                                    const int32_t *block_table, int32_t max_blocks_per_seq,
                                    const int32_t *context_lens, int32_t batch,
                                    int32_t max_q_len, int32_t num_q_heads,
                                    float softmax_scale, void *workspace,
                                    size_t workspace_bytes, void *stream)
{
    return pkvq_paged_attn_prefill_ex(cache, q, out, lse_out, cu_seqlens_q, block_table,
                                      max_blocks_per_seq, context_lens, batch, max_q_len,
                                      num_q_heads, softmax_scale, nullptr, workspace,
                                      workspace_bytes, stream);
}

pkvq_status pkvq_paged_attn_prefill_ex(const pkvq_cache *cache, const void *q, void *out,
                                       float *lse_out, const int32_t *cu_seqlens_q,
                                       const int32_t *block_table, int32_t max_blocks_per_seq,
                                       const int32_t *context_lens, int32_t batch,
                                       int32_t max_q_len, int32_t num_q_heads,
                                       float softmax_scale, const pkvq_attn_opts *opts,
                                       void *workspace, size_t workspace_bytes, void *stream)
{
    (void)workspace;
    (void)workspace_bytes;
    if (opts && opts->sliding_window < 0)
        return PKVQ_ERR_INVALID_ARG;
    if (opts && opts->query_pos)
        return PKVQ_ERR_UNSUPPORTED;
    pkvq_status st = check_cache(cache);
    if (st != PKVQ_OK)
        return st;
    if (batch < 0 || max_q_len < 0 || num_q_heads <= 0 || max_blocks_per_seq < 0)
        return PKVQ_ERR_INVALID_ARG;
    if (num_q_heads % cache->num_kv_heads)
        return PKVQ_ERR_INVALID_ARG;
    const int group = num_q_heads / cache->num_kv_heads;
    if (group > 128)
        return PKVQ_ERR_UNSUPPORTED;
    if (!isfinite(softmax_scale))
        return PKVQ_ERR_INVALID_ARG;
    if (batch == 0 || max_q_len == 0)
        return PKVQ_OK;
    if (!q || !out || !cu_seqlens_q || !block_table || !context_lens)
        return PKVQ_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(out))
        return PKVQ_ERR_MISALIGNED;
    CUtensorMap km, vm;
    st = cache_maps(cache, &km, &vm);
    if (st != PKVQ_OK)
        return st;
    PrefillParams p{};
    p.k_cache = static_cast<const uint8_t *>(cache->k_cache);
    p.v_cache = static_cast<const uint8_t *>(cache->v_cache);
    const bool head_scale = kv_has_head_scale(cache->dtype);
    p.k_scale = head_scale ? cache->k_scale : nullptr;
    p.v_scale = head_scale ? cache->v_scale : nullptr;
    p.scale_stride = scale_stride(cache);
    // (the last fields of pkvq_cache are read for these formats only)
    const bool blk_scale = kv_has_block_scale(cache->dtype);
    p.k_scale_blk = blk_scale ? cache->k_scale_blk : nullptr;
    p.v_scale_blk = blk_scale ? cache->v_scale_blk : nullptr;
    p.window = opts ? opts->sliding_window : 0;
    p.k_scale_tok = static_cast<const uint16_t *>(cache->k_scale_tok);
    p.v_scale_tok = static_cast<const uint16_t *>(cache->v_scale_tok);
    p.q = static_cast<const __half *>(q);
    p.out = static_cast<__half *>(out);
    p.lse = lse_out;
    p.cu_seqlens_q = cu_seqlens_q;
    p.block_table = block_table;
    p.context_lens = context_lens;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.batch = batch;
    p.max_q_len = max_q_len;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = cache->num_kv_heads;
    p.group = group;
    p.num_blocks = cache->num_blocks;
    p.block_size = cache->block_size;
    p.tokens_per_tile = 128 / group;   // 128 query rows per CTA
    p.q_tiles = (max_q_len + p.tokens_per_tile - 1) / p.tokens_per_tile;
    p.scale_log2 = softmax_scale * kLog2e;
    p.status = status_ptr();
    if (!p.status)
        return PKVQ_ERR_CUDA;
    return from_cuda(launch_prefill_tc(p, cache->dtype, km, vm, static_cast<cudaStream_t>(stream)));
}

pkvq_status pkvq_merge_attn_states(const void *parts_out, const float *parts_lse,
                                   int32_t num_parts, int64_t n_rows, int32_t head_dim,
                                   void *out, float *lse_out, void *stream)
{
    if (head_dim != kHeadDim)
        return PKVQ_ERR_UNSUPPORTED;
    if (num_parts < 1 || num_parts > 64 || n_rows < 0)
        return PKVQ_ERR_INVALID_ARG;
    if (n_rows == 0)
        return PKVQ_OK;
    if (!parts_out || !parts_lse || !out)
        return PKVQ_ERR_INVALID_ARG;
    if (!aligned16(parts_out) || !aligned16(out))
        return PKVQ_ERR_MISALIGNED;
    MergeParams p{};
    p.parts_out = static_cast<const __half *>(parts_out);
    p.parts_lse = parts_lse;
    p.out = static_cast<__half *>(out);
    p.lse = lse_out;
    p.parts = num_parts;
    p.rows = n_rows;
    return from_cuda(launch_merge_states(p, static_cast<cudaStream_t>(stream)));
}

pkvq_status pkvq_kv_copy_blocks(const pkvq_cache *dst, const pkvq_cache *src,
                                const int32_t *pairs, int32_t n, void *stream)
{
    pkvq_status st = check_cache(dst);
    if (st != PKVQ_OK)
        return st;
    st = check_cache(src);
    if (st != PKVQ_OK)
        return st;
    if (dst->dtype != src->dtype || dst->block_size != src->block_size ||
        dst->num_kv_heads != src->num_kv_heads || dst->head_dim != src->head_dim)
        return PKVQ_ERR_INVALID_ARG;
    if (n < 0)
        return PKVQ_ERR_INVALID_ARG;
    if (n == 0)
        return PKVQ_OK;
    if (!pairs)
        return PKVQ_ERR_INVALID_ARG;
    CopyParams p{};
    p.src_k = static_cast<const uint8_t *>(src->k_cache);
    p.src_v = static_cast<const uint8_t *>(src->v_cache);
    p.dst_k = static_cast<uint8_t *>(dst->k_cache);
    p.dst_v = static_cast<uint8_t *>(dst->v_cache);
    const bool int8 = src->dtype == PKVQ_KV_INT8;
    p.src_ks = int8 ? static_cast<const uint16_t *>(src->k_scale_tok) : nullptr;
    p.src_vs = int8 ? static_cast<const uint16_t *>(src->v_scale_tok) : nullptr;
    p.dst_ks = int8 ? static_cast<uint16_t *>(dst->k_scale_tok) : nullptr;
    p.dst_vs = int8 ? static_cast<uint16_t *>(dst->v_scale_tok) : nullptr;
    const bool blk = kv_has_block_scale(src->dtype);
    p.src_kb = blk ? src->k_scale_blk : nullptr;
    p.src_vb = blk ? src->v_scale_blk : nullptr;
    p.dst_kb = blk ? dst->k_scale_blk : nullptr;
    p.dst_vb = blk ? dst->v_scale_blk : nullptr;
    p.num_kv_heads = src->num_kv_heads;
    p.pairs = pairs;
    p.n = n;
    p.block_bytes = (long long)src->num_kv_heads * src->block_size * kHeadDim *
                    kv_elem_bytes(src->dtype);
    p.block_scales = int8 ? src->num_kv_heads * src->block_size : 0;
    p.src_blocks = src->num_blocks;
    p.dst_blocks = dst->num_blocks;
    p.status = status_ptr();
    if (!p.status)
        return PKVQ_ERR_CUDA;
    return from_cuda(launch_copy_blocks(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
