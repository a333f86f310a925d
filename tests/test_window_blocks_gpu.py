"""GPU: with a sliding window, no block below every query's window is read: its table
entry may be gone (-1), and its memory may hold anything."""
import numpy as np
import pytest
import torch

import paged_quantized_kv_quant_b200 as pk
from pkvq_ref64 import ALL, BLOCK, D, lay_out, random_cache
from test_block_scale_gpu import SCALE, cuda, queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bs", [16, 32, 64])
@pytest.mark.parametrize("fmt", ALL)
def test_blocks_below_the_window_are_not_read(fmt, bs):
    hq, hkv, window = 16, 2, 100
    ctx = [1000, 513, 470]
    r = np.random.default_rng(151)
    blocks, table, _ = lay_out(ctx, bs, 152)
    for ql in (1, 5, 33, 400):
        a, b = (random_cache(fmt, blocks, bs, hkv, 153) for _ in "ab")
        gone = table.copy()
        for i, c in enumerate(ctx):
            first = max(0, c - ql - window + 1) // bs
            lost = gone[i, :first].copy()
            gone[i, :first] = -1
            for x in lost:
                b.k_cache[int(x)] = b.v_cache[int(x)] = 0x7F      # NaN in every floating-point format
                for s in (b.k_scale_tok, b.v_scale_tok, b.k_scale_blk, b.v_scale_blk):
                    if s is not None:
                        s[int(x)] = float("nan")
        c = cuda(np.int32(ctx))
        res = []
        for cache, t in ((a, cuda(table)), (b, cuda(gone))):
            if ql <= 16:
                q = cuda(queries(np.random.default_rng(154), 3, ql, hq, D))
                lse = torch.empty((3, ql, hq), device="cuda")
                out = pk.paged_attn_decode(cache, q, t, c, 1000, SCALE, lse=lse, sliding_window=window)
                res.append((out, lse))
                W = torch.zeros((3, hkv, 1000), device="cuda")
                out = pk.paged_attn_decode_weights(cache, q, t, c, 1000, SCALE, W, sliding_window=window)
                res[-1] += (out, W)
            else:
                q = cuda(queries(np.random.default_rng(154), 3 * ql, hq, D))
                lse = torch.empty((3 * ql, hq), device="cuda")
                out = pk.paged_attn_prefill(cache, q, cuda(np.arange(4, dtype=np.int32) * ql), t, c, ql, SCALE,
                                            lse=lse, sliding_window=window)
                res.append((out, lse))
        for x, y in zip(*res):
            assert torch.isfinite(y).all() and torch.equal(x, y), ql
    assert pk.device_status() == 0
