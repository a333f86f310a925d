"""GPU: causal attention over packed whole prompts against a 64-bit reference."""
import numpy as np
import pytest
import torch

import paged_quantized_kv_quant_b200 as pk
from pkvq_ref64 import D, attention, lse_bound, out_bound

pytestmark = pytest.mark.gpu
SCALE = 1.0 / np.sqrt(D)
BITS = {torch.float16: 11, torch.bfloat16: 8}


def make(lens, hq, hkv, dt, seed=0, extra=0):
    g = torch.Generator().manual_seed(seed)
    t = sum(lens) + extra
    q, k, v = (torch.randn((t, n, D), generator=g).mul_(m).to(dt) for n, m in ((hq, 1.5), (hkv, 1), (hkv, 1)))
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
    return q, k, v, cu


def check(out, lse, q, k, v, lens, scale=SCALE, window=0, every=1):
    """Every `every`-th row of each sequence (and its first and last)."""
    dt, hq, hkv = q.dtype, q.shape[1], k.shape[1]
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    qd, kd, vd = (x.double().numpy() for x in (q, k, v))
    at = 0
    for n in lens:
        rows = np.unique(np.concatenate([np.arange(0, n, every), [n - 1]])) if n else np.zeros(0, int)
        for h in range(hq if n else 0):
            s = slice(at, at + n)
            kh, vh = kd[s, h // (hq // hkv)], vd[s, h // (hq // hkv)]
            ref, rl, _, a, sabs = attention(qd[at + rows, h], kh, vh, rows, scale, window)
            sabs = max(sabs, -sabs)
            bound = out_bound(ref, a, n, np.abs(vh).max() * 2, sabs, dt, BITS[dt])
            err = np.abs(o[at + rows, h] - ref)
            assert (err <= bound).all(), f"len {n} head {h}: {(err - bound).max():.2e} above its bound"
            assert (np.abs(l[at + rows, h] - rl) <= lse_bound(sabs)).all()
        at += n
    assert pk.device_status() == 0


def run(q, k, v, cu, lens, **kw):
    lse = torch.empty(q.shape[:2], device="cuda")
    out = pk.prompt_attn(q.cuda(), k.cuda(), v.cuda(), cu.cuda(), max(list(lens) + [0]), kw.pop("scale", SCALE),
                         lse=lse, **kw)
    return out, lse


CASES = [
    # lens, Hq, Hkv, window
    ([1], 1, 1, 0),
    ([1, 2, 3, 0, 5], 8, 2, 0),
    ([128, 127, 129], 8, 8, 0),             # G = 1: 128 tokens a tile
    ([300, 16, 257], 32, 4, 0),             # G = 8
    ([511, 33], 10, 2, 0),                  # G = 5: 125 rows of 128
    ([200, 90], 14, 2, 0),                  # G = 7
    ([65, 260], 16, 1, 0),                  # G = 16
    ([40], 128, 1, 0),                      # G = 128: one token a tile
    ([90], 130, 2, 0),                      # G = 65
    ([700, 5, 300], 8, 2, 1),               # a window of the token itself
    ([700, 5, 300], 8, 2, 100),
    ([900], 32, 4, 129),
    ([600], 4, 4, 10_000),
]


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("lens,hq,hkv,window", CASES)
def test_prompt(lens, hq, hkv, window, dt):
    q, k, v, cu = make(lens, hq, hkv, dt, seed=len(lens))
    out, lse = run(q, k, v, cu, lens, sliding_window=window)
    check(out, lse, q, k, v, lens, window=window)


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
def test_long_prompt(dt):
    lens = [2500, 1, 1300]
    q, k, v, cu = make(lens, 16, 2, dt, seed=9)
    out, lse = run(q, k, v, cu, lens)
    check(out, lse, q, k, v, lens, every=37)


@pytest.mark.parametrize("scale", [0.0, -0.1, 3.0, 1e-20])
def test_other_scales(scale):
    """Uniform weights, negated scores, scores of several hundred."""
    lens = [300, 70]
    q, k, v, cu = make(lens, 8, 2, torch.float16, seed=10)
    out, lse = run(q, k, v, cu, lens, scale=scale)
    qd = q.double()
    # the reference's own magnitudes take |scale|
    check(out, lse, (q if scale >= 0 else -q), k, v, lens, scale=abs(scale))
    assert qd.shape[0] == 370


def test_growing_maxima_rescale():
    """Keys that grow along the sequence: the running maximum rises in every tile."""
    lens = [1000]
    q, k, v, cu = make(lens, 8, 1, torch.float16, seed=11)
    q = q.abs()
    k = (k.abs() * torch.linspace(0.1, 4, 1000)[:, None, None]).half()
    out, lse = run(q, k, v, cu, lens)
    check(out, lse, q, k, v, lens)


def test_slices_of_a_fused_projection():
    lens, hq, hkv = [130, 250], 8, 2
    g = torch.Generator().manual_seed(12)
    fused = torch.randn((380, hq + 2 * hkv, D), generator=g).to(torch.bfloat16)
    fq, fk, fv = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:]
    cu = torch.tensor([0, 130, 380], dtype=torch.int32)
    f = fused.cuda()
    lse = torch.empty((380, hq), device="cuda")
    out = pk.prompt_attn(f[:, :hq], f[:, hq:hq + hkv], f[:, hq + hkv:], cu.cuda(), 250, SCALE, lse=lse)
    check(out, lse, fq.contiguous(), fk.contiguous(), fv.contiguous(), lens)
    # heads outermost
    t = [x.transpose(0, 1).contiguous().cuda().transpose(0, 1) for x in (fq, fk, fv)]
    assert torch.equal(out, pk.prompt_attn(*t, cu.cuda(), 250, SCALE))


def test_neighbours_do_not_leak():
    """A sequence's neighbours hold infinities and NaN; rows behind the last
    sequence are left as they were."""
    lens = [70, 70, 70]
    q, k, v, cu = make(lens, 8, 2, torch.float16, seed=13, extra=40)
    clean = run(q, k, v, cu, lens)
    bad = [x.clone() for x in (q, k, v)]
    for x in bad:
        x[70:140] = float("nan")
        x[210:] = float("inf")
    out = torch.full((250, 8, D), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((250, 8), 7.0, device="cuda")
    pk.prompt_attn(*(x.cuda() for x in bad), cu.cuda(), 70, SCALE, out=out, lse=lse)
    for s in (slice(0, 70), slice(140, 210)):
        assert torch.equal(out[s], clean[0][s]) and torch.equal(lse[s], clean[1][s])
    assert (out[210:] == 7).all() and (lse[210:] == 7).all()


def test_captured_on_another_stream():
    lens = [90, 300]
    q, k, v, cu = make(lens, 8, 2, torch.bfloat16, seed=14)
    ref = run(q, k, v, cu, lens)
    d = [torch.zeros_like(x).cuda() for x in (q, k, v)]
    c, out, lse = cu.cuda(), torch.empty_like(d[0]), torch.empty(q.shape[:2], device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        pk.prompt_attn(*d, c, 300, SCALE, out=out, lse=lse)
    for x, y in zip(d, (q, k, v)):
        x.copy_(y)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])


def test_agrees_with_prefill_over_an_fp16_cache():
    """The same prompt through the cache: both orders of serving agree."""
    lens, hq, hkv, bs = [333, 47], 16, 2, 16
    q, k, v, cu = make(lens, hq, hkv, torch.float16, seed=15)
    out, lse = run(q, k, v, cu, lens)
    nb = [-(-n // bs) for n in lens]
    cache = pk.PagedKVCache.allocate(pk.KV_FP16, sum(nb), bs, hkv)
    table = torch.zeros((2, max(nb)), dtype=torch.int32)
    table[0, :nb[0]] = torch.arange(nb[0], dtype=torch.int32)
    table[1, :nb[1]] = nb[0] + torch.arange(nb[1], dtype=torch.int32)
    slots = torch.cat([torch.arange(lens[0]), nb[0] * bs + torch.arange(lens[1])]).to(torch.int32)
    pk.kv_write_quant(cache, k.cuda(), v.cuda(), slots.cuda())
    lse2 = torch.empty_like(lse)
    out2 = pk.paged_attn_prefill(cache, q.cuda(), cu.cuda(), table.cuda(),
                                 torch.tensor(lens, dtype=torch.int32).cuda(), max(lens), SCALE, lse=lse2)
    # both are within their bounds of the same numbers: twice fp16's half step
    # of |out| < 8 and of P's rounding
    assert (out.double() - out2.double()).abs().max() <= 2 * (2.0 ** -9 + 2.0 ** -10 * 4)
    assert (lse - lse2).abs().max() <= 1e-4
