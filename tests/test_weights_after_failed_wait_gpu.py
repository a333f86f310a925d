"""GPU: decode with weights after a device-side wait that gave up (the status word's
bit 0): kernels skip their work, and the accumulated weights, which outlive the call,
stay as they were.  No wait is made to fail: a host driver, linked with the library's
own objects, calls the launch with a status word of the test's."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import paged_quantized_kv_quant_b200 as pk
from paged_quantized_kv_quant_b200 import build as pkbuild
from pkvq_ref64 import D, lay_out, random_cache
from test_block_scale_gpu import SCALE, cuda, queries

pytestmark = pytest.mark.gpu

DRIVER = r"""
#include "internal.h"
#include "common.cuh"
#include "pkvq.h"
using namespace pkvq;
extern "C" __attribute__((visibility("default"))) int
decode_weights_with_status(const pkvq_cache *c, const void *q, void *out, const int32_t *table, int cols,
                           const int32_t *lens, int batch, int q_len, int hq, int max_len, float scale,
                           float *weights, long long stride, void *ws, unsigned *status)
{
    DecodePlan plan;
    if (!decode_plan(c->dtype, batch, q_len, hq, c->num_kv_heads, c->block_size, max_len, true, &plan))
        return -1;
    CUtensorMap m[2];
    const uint64_t rows = (uint64_t)c->num_blocks * c->num_kv_heads * c->block_size;
    if (!make_cache_tensor_map(&m[0], c->k_cache, rows, c->block_size, kHeadDim) ||
        !make_cache_tensor_map(&m[1], c->v_cache, rows, c->block_size, kHeadDim))
        return -2;
    DecodeParams p{};
    p.k_cache = (const uint8_t *)c->k_cache, p.v_cache = (const uint8_t *)c->v_cache;
    p.k_scale_blk = c->k_scale_blk, p.v_scale_blk = c->v_scale_blk;
    p.q = (const __half *)q, p.out = (__half *)out;
    p.block_table = table, p.context_lens = lens, p.max_blocks_per_seq = cols;
    p.batch = batch, p.q_len = q_len, p.num_q_heads = hq, p.num_kv_heads = c->num_kv_heads;
    p.group = hq / c->num_kv_heads, p.num_blocks = c->num_blocks, p.block_size = c->block_size;
    p.rows = q_len * p.group, p.rows_per_cta = plan.rows_per_cta, p.row_groups = plan.row_groups;
    p.num_splits = plan.num_splits, p.uniform_splits = plan.uniform_splits, p.uniform_bpc = plan.uniform_bpc;
    p.uniform_more = plan.uniform_more, p.uniform_bpc_more = plan.uniform_bpc_more, p.spread = plan.spread;
    p.split_min_blocks = plan.split_min_blocks, p.split_gran = plan.split_gran;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.ws_o = (float *)ws;
    p.ws_ml = p.ws_o + (size_t)c->num_kv_heads * plan.row_groups * plan.num_splits * plan.rows_per_cta * kHeadDim;
    p.scores = (float *)((uint8_t *)ws + plan.state_bytes);
    p.weights = weights, p.weight_stride = stride, p.score_keys = plan.score_keys, p.score_rows = plan.score_rows;
    p.status = status;
    return (int)launch_decode_weights(p, plan, c->dtype, m[0], m[1], nullptr);
}
"""


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    pkbuild.build()
    d = tmp_path_factory.mktemp("failedwait")
    objdir = os.path.join(pkbuild.PKG, "_build", "release")
    objs = [os.path.join(objdir, os.path.basename(s)[:-3] + ".o") for s in pkbuild._sources()]
    if not all(os.path.exists(o) for o in objs):
        pkbuild.build(force=True)
    src, lib = d / "driver.cu", d / "driver.so"
    src.write_text(DRIVER)
    subprocess.run([pkbuild.NVCC, *pkbuild.ARCH, "-std=c++17", "-Xcompiler", "-fPIC", "-shared",
                    "-I", pkbuild.CSRC, "-I", os.path.join(pkbuild.ROOT, "include"), str(src), *objs, "-o", str(lib)],
                   check=True, capture_output=True)
    f = ctypes.CDLL(str(lib)).decode_weights_with_status
    P, I = ctypes.c_void_p, ctypes.c_int
    f.argtypes = [P, P, P, P, I, P, I, I, I, I, ctypes.c_float, P, ctypes.c_longlong, P, P]
    return f


@pytest.mark.parametrize("hq,ql", [(8, 1), (32, 1), (32, 5)])    # 2, 8 and 40 rows per KV head
def test_accumulator_is_left_alone(driver, hq, ql):
    hkv, bs, ctx = 4, 16, [1500, 40]
    blocks, table, _ = lay_out(ctx, bs, 121)
    cache = random_cache(pk.KV_INT8_BLOCK, blocks, bs, hkv, 122)
    q = cuda(queries(np.random.default_rng(123), 2, ql, hq, D))
    t, c = cuda(table), cuda(np.int32(ctx))
    W0 = torch.rand((2, hkv, 1500), device="cuda")
    # (NaN in the workspace: what a skipped pass must not have read)
    need = pk.decode_weights_workspace_bytes(cache, 2, ql, hq, 1500)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    expect = W0.clone()
    pk.paged_attn_decode_weights(cache, q, t, c, 1500, SCALE, expect)
    for bits in (1, 3, 0):
        W = W0.clone()
        status = torch.tensor([bits], dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        cs = cache.struct()
        rc = driver(ctypes.byref(cs), q.data_ptr(), out.data_ptr(), t.data_ptr(), t.shape[1], c.data_ptr(), 2, ql, hq,
                    1500, SCALE, W.data_ptr(), 1500, ws.data_ptr(), status.data_ptr())
        torch.cuda.synchronize()
        assert rc == 0 and int(status) == bits
        assert torch.equal(W, expect if bits == 0 else W0)
