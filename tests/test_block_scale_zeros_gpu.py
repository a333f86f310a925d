"""GPU: block-scaled caches in which some blocks hold nothing but zero values (V
scale 0).  Their keys take their share of the softmax, often the largest one, and the
other blocks' values must keep their precision beside them, through every attention
kernel."""
import numpy as np
import pytest
import torch

import paged_quantized_kv_quant_b200 as pk
from pkvq_ref64 import BLOCK, D, Host, attention, half_step, lay_out, lse_bound, random_cache
from test_block_scale_gpu import SCALE, cuda

pytestmark = pytest.mark.gpu

# (Hq, Hkv, query tokens): mma.sync decode of 4 and 16 rows, tensor-core decode of 40
# and 96 rows, prefill
KERNELS = [(8, 2, 1), (16, 1, 1), (32, 4, 5), (16, 2, 12), (8, 2, 150)]
# (x where the other blocks' values are of about 2^x; how many nats the zero blocks'
# keys score above the rest)
LEVELS = [(0, 10.0), (-6, 10.0), (-7, 0.0), (-13, 0.0), (-17, 0.0)]


def make(fmt, hq, hkv, ql, bs, level, gap, seed=91):
    """Three sequences: zero blocks among others, no zero block, nothing but zeros."""
    r = np.random.default_rng(seed)
    ctx = [700, 203, 90 + ql]
    blocks, table, _ = lay_out(ctx, bs, seed + 1)
    cache = random_cache(fmt, blocks, bs, hkv, seed + 2)
    unit = 2.0 ** -(7 if fmt == pk.KV_E4M3_BLOCK else 5)     # the scale of values of about 1
    v_scale = unit * 2.0 ** level
    cache.k_scale_blk[:], cache.v_scale_blk[:] = unit, v_scale
    zero = [int(table[0][i]) for i in (0, 3, 3 + 200 // bs)] + [int(x) for x in table[2] if x >= 0]
    one = 64 if fmt == pk.KV_INT8_BLOCK else 0x68        # the code of 64
    for z in zero:
        cache.v_cache[z], cache.v_scale_blk[z] = 0, 0.0
        cache.k_cache[z], cache.k_scale_blk[z] = one, 1 / 64      # keys of all ones
    # a query's component along the ones is worth `gap` nats on those keys
    q = 1.5 * r.standard_normal((3, ql, hq, D)) + gap / (D * SCALE)
    return cache, table, ctx, q.astype(np.float16), 448 * v_scale if one != 64 else 127 * v_scale


def check(out, lse, q, host, table, ctx, ql, hq, vmax, what=""):
    G = hq // host.hkv
    for b, n in enumerate(ctx):
        pos = n - ql + np.arange(ql)
        for h in range(host.hkv):
            keys, vals = host.rows("k", table[b], h, n), host.rows("v", table[b], h, n)
            live = np.abs(vals).max(1) > 0
            for g in range(h * G, (h + 1) * G):
                ref, rl, p, a, sabs = attention(q[b, :, g].astype(float), keys, vals, pos, SCALE)
                # the output's rounding; each weight's own rounding and its score's error
                # (as out_bound).  Weights are rounded against the largest one of a block
                # that holds values: a weight below 2^-14 of that loses at most 2^-25 of
                # it, times the largest value.
                top = p[:, live].max(1, initial=0.0)
                es = 2 * 129 * 2.0 ** -23 * sabs + 2.0 ** -18
                bound = half_step(ref) * 1.01 + (2.0 ** -11 + es) * a + (n * 2.0 ** -25 * vmax * top)[:, None]
                err = np.abs(out[b, :, g] - ref)
                assert (err <= bound).all(), \
                    f"{what} seq {b} head {g}: error {err.max():.2e}, output {np.abs(ref).max():.2e}, " \
                    f"{float((err / bound).max()):.1f} of its bound"
                assert (np.abs(lse[b, :, g] - rl) <= lse_bound(sabs)).all(), what


@pytest.mark.parametrize("level,gap", LEVELS)
@pytest.mark.parametrize("hq,hkv,ql", KERNELS)
@pytest.mark.parametrize("fmt", BLOCK)
def test_values_beside_blocks_of_zeros(fmt, hq, hkv, ql, level, gap):
    bs = 64 if ql == 12 else 16
    cache, table, ctx, q, vmax = make(fmt, hq, hkv, ql, bs, level, gap)
    host = Host(cache)
    t, c = cuda(table), cuda(np.int32(ctx))
    lse = torch.empty((3, ql, hq), device="cuda")
    if ql <= 16:
        out = pk.paged_attn_decode(cache, cuda(q), t, c, max(ctx), SCALE, lse=lse)
    else:
        cu = cuda(np.int32([0, ql, 2 * ql, 3 * ql]))
        out = pk.paged_attn_prefill(cache, cuda(q).view(3 * ql, hq, D), cu, t, c, ql, SCALE,
                                    lse=lse.view(3 * ql, hq)).view(3, ql, hq, D)
    check(out.double().cpu().numpy(), lse.double().cpu().numpy(), q, host, table, ctx, ql, hq, vmax)
    assert (out[2] == 0).all()
    assert pk.device_status() == 0


@pytest.mark.parametrize("ql", [1, 5])
@pytest.mark.parametrize("fmt", BLOCK)
def test_decode_with_weights_beside_blocks_of_zeros(fmt, ql):
    hq, hkv = 32, 4
    cache, table, ctx, q, vmax = make(fmt, hq, hkv, ql, 16, -6, 10.0)
    host = Host(cache)
    lse = torch.empty((3, ql, hq), device="cuda")
    W = torch.zeros((3, hkv, 700), device="cuda")
    out = pk.paged_attn_decode_weights(cache, cuda(q), cuda(table), cuda(np.int32(ctx)), 700, SCALE, W, lse=lse)
    check(out.double().cpu().numpy(), lse.double().cpu().numpy(), q, host, table, ctx, ql, hq, vmax)
    # every query row spends a weight of 1 on its keys
    assert torch.allclose(W.double().sum(-1), torch.full((3, hkv), 8.0 * ql, dtype=torch.float64, device="cuda"),
                          rtol=3e-4, atol=0)
