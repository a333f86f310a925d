"""GPU: appending decode steps over block-scaled caches, enqueued back to back.  Each
step's write kernel and the decode kernel behind it overlap on the device; every step
makes the scales that the decode reads grow."""
import numpy as np
import pytest
import torch

import paged_quantized_kv_quant_b200 as pk
from pkvq_ref64 import BLOCK, D, lay_out, random_cache
from test_block_scale_gpu import SCALE, cuda, queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,ql", [(8, 8, 1), (32, 4, 1), (32, 4, 5)])
@pytest.mark.parametrize("fmt", BLOCK)
def test_steps_equal_write_wait_decode(fmt, hq, hkv, ql):
    bs, steps, B = 16, 24, 48
    r = np.random.default_rng(101)
    start = r.integers(1, 60, B).astype(np.int32)
    last = start + steps * ql
    blocks, table, _ = lay_out(last, bs, 102)
    a, b = (random_cache(fmt, blocks, bs, hkv, 103) for _ in "ab")
    for c in (a, b):
        c.k_scale_blk *= 1e-2
        c.v_scale_blk *= 1e-2
    t = cuda(table)
    new = [[cuda((r.standard_normal((B, ql, hkv, D)) * 1.3 ** i).astype(np.float16)) for _ in "kv"]
           for i in range(steps)]
    q = [cuda(queries(r, B, ql, hq, D)) for _ in range(steps)]
    ctx = [cuda((start + (i + 1) * ql).astype(np.int32)) for i in range(steps)]
    cu = cuda(np.arange(B + 1, dtype=np.int32) * ql)
    most = int(last.max())
    torch.cuda.synchronize()
    outs = [pk.paged_attn_decode_append(a, *new[i], q[i], t, ctx[i], most, SCALE) for i in range(steps)]
    torch.cuda.synchronize()
    for i in range(steps):
        k, v = (x.view(B * ql, hkv, D) for x in new[i])
        pk.kv_write_block_quant(b, k, v, cu, t, ctx[i], ql)
        torch.cuda.synchronize()
        assert torch.equal(outs[i], pk.paged_attn_decode(b, q[i], t, ctx[i], most, SCALE)), i
    for name in ("k_cache", "v_cache", "k_scale_blk", "v_scale_blk"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name
    assert pk.device_status() == 0
