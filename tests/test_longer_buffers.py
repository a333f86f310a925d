"""The binding takes buffers preallocated for more sequences than a call has, and a
stream that is any object with a raw `cuda_stream`; it refuses shorter buffers and
streams of another device."""
import types

import numpy as np
import pytest
import torch

import paged_quantized_kv_quant_b200 as pk


def test_room():
    """(device -1: host tensors, whose address is never used)"""
    i32 = torch.int32
    t = torch.zeros((4, 6), dtype=i32)
    for shape in ((4, 6), (3, 6), (0, 6), (8, 3)):
        assert pk._room("t", t, i32, shape, -1) == t.data_ptr()
    assert pk._room("t", None, i32, (3,), -1) is None
    for bad in (t[:2], t[0], t.long(), t.t(), t[:, :5], None.__class__):
        with pytest.raises((ValueError, TypeError)):
            pk._room("t", bad, i32, (3, 6), -1)
    with pytest.raises(ValueError):
        pk._room("t", t, i32, (3, 6), 0)


def test_streams(monkeypatch):
    class Stream:
        def __init__(self, index, raw=7):
            self.device_index, self.cuda_stream = index, raw
    t = types.SimpleNamespace(device="cuda:0", get_device=lambda: 0)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda raw, device: Stream(0, raw))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: s)
    assert pk._on(t, Stream(0)).cuda_stream == 7
    assert pk._on(t, types.SimpleNamespace(cuda_stream=9)).cuda_stream == 9
    with pytest.raises(ValueError, match="device"):
        pk._on(t, Stream(1))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [pk.KV_FP8_E4M3, pk.KV_INT8_BLOCK])
def test_longer_buffers_give_the_same_results(fmt):
    from pkvq_ref64 import BLOCK, D, lay_out, random_cache
    from test_block_scale_gpu import SCALE, cuda, new_rows, queries
    r = np.random.default_rng(141)
    ctx, hq, hkv, bs, B = [300, 77], 8, 2, 16, 2
    blocks, table, dst = lay_out(ctx, bs, 142, spare=4)
    q, pre = cuda(queries(r, B, 1, hq, D)), cuda(queries(r, 30, hq, D))
    t, c, d = cuda(table), cuda(np.int32(ctx)), cuda(dst)
    more = lambda x: torch.cat([x, x.new_full((3, *x.shape[1:]), -7)])  # noqa: E731
    cu = cuda(np.int32([0, 20, 30]))
    k, v = (cuda(new_rows(r, B, hkv)) for _ in "kv")
    cw = cuda(np.int32([0, 1, 2]))

    def calls(grow):
        cache = random_cache(fmt, blocks, bs, hkv, 143)
        out = lambda *s: (more if grow else torch.clone)(torch.full(s, -7.0, device="cuda"))  # noqa: E731
        g = more if grow else (lambda x: x)
        res, spare = [], []

        def keep(x, n):
            res.append(x[:n].clone()), spare.append(x[n:])
        # an lse of (batch, heads, 1) for one query token was always taken
        for f, kw in ((pk.paged_attn_decode, {}), (pk.paged_attn_decode_weights, dict(W=1)), (pk.paged_attn_decode_append, dict(new=1))):
            o, l = out(B, 1, hq, D).half(), out(B, hq, 1)
            a = (k.view(B, 1, hkv, D), v.view(B, 1, hkv, D)) if "new" in kw else ()
            w = torch.zeros((B, hkv, 300), device="cuda")
            got = f(cache, *a, q, g(t), g(c), 300, SCALE, out=o, lse=l, **(dict(weights=w) if "W" in kw else {}))
            assert got is o
            keep(o, B), keep(l.view(-1, 1, hq), B)
            if "W" in kw:
                keep(w, B)
        o, l = out(30, hq, D).half(), out(30, hq)
        pk.paged_attn_prefill(cache, pre, g(cu), g(t), c, 20, SCALE, out=o, lse=l)
        keep(o, 30), keep(l, 30)
        if fmt in BLOCK:
            pk.kv_write_block_quant(cache, k, v, g(cw), g(t), c, 1)
        lens, w2, kept = pk.kv_evict(cache, w + torch.arange(300, device="cuda"), g(t), c, g(d), 40, 2, 3)
        return res + [lens, w2, kept, cache.k_cache, cache.v_cache], spare

    plain, _ = calls(False)
    grown, spare = calls(True)
    for a, b in zip(plain, grown):
        assert torch.equal(a, b)
    assert all((x == -7).all() for x in spare)
    for kw in (dict(out=torch.empty((1, 1, hq, D), device="cuda").half()), dict(lse=torch.empty((1, 1, hq), device="cuda")),
               dict(lse=torch.empty((B * hq,), device="cuda"))):
        with pytest.raises(ValueError):
            pk.paged_attn_decode(random_cache(fmt, blocks, bs, hkv, 143), q, t, c, 300, SCALE, **kw)
    raw = types.SimpleNamespace(cuda_stream=torch.cuda.current_stream().cuda_stream)
    cache = random_cache(fmt, blocks, bs, hkv, 143)
    torch.cuda.synchronize()
    assert torch.equal(pk.paged_attn_decode(cache, q, t, c, 300, SCALE, stream=raw), plain[0])
    assert pk.device_status() == 0
