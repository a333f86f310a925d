"""GPU: caches with one scale per (block, KV head): the write against its
definition bit for bit, and every attention entry point over them against a
64-bit reference."""
import numpy as np
import pytest
import torch

import paged_quantized_kv_quant_b200 as pk
from pkvq_ref64 import (BLOCK, D, QMAX, Host, attention, lay_out, lse_bound, out_bound,
                        random_cache, write_block)

pytestmark = pytest.mark.gpu
SCALE = 1.0 / np.sqrt(D)


def cuda(a):
    return torch.as_tensor(np.ascontiguousarray(a)).cuda()


def new_rows(r, t, hkv):
    """fp16 rows whose loudness differs from token to token."""
    return (r.standard_normal((t, hkv, D)) * np.exp(r.standard_normal((t, hkv, 1)))).astype(np.float16)


def assert_same(cache, host, what=""):
    for name, ref in (("k_cache", host.k), ("v_cache", host.v)):
        got = getattr(cache, name).cpu().numpy()
        assert np.array_equal(got, ref), f"{what} {name}: {(got != ref).sum()} codes differ"
    assert np.array_equal(cache.k_scale_blk.cpu().numpy(), host.ks), what
    assert np.array_equal(cache.v_scale_blk.cpu().numpy(), host.vs), what


@pytest.mark.parametrize("fmt", BLOCK)
@pytest.mark.parametrize("bs", [16, 32, 64])
@pytest.mark.parametrize("old,new", [
    ([0], [1]), ([0, 0, 0], [16, 33, 200]), ([15, 16, 17, 5], [1, 1, 1, 1]),
    ([3, 100, 63], [70, 0, 129]), ([1, 31, 47], [5, 5, 5])])
def test_write_is_bit_exact(fmt, bs, old, new):
    hkv = 3
    r = np.random.default_rng(bs + len(old))
    ctx = np.array(old) + new
    blocks, table, _ = lay_out(ctx, bs, 1)
    cache = random_cache(fmt, blocks, bs, hkv, 2)   # what it holds is old tokens and stale rows
    # some older blocks loud (their scale stays), some quiet (it grows)
    cache.k_scale_blk[::2] *= 0.01
    host = Host(cache)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    k, v = new_rows(r, cu[-1], hkv), new_rows(r, cu[-1], hkv)
    pk.kv_write_block_quant(cache, cuda(k), cuda(v), cuda(cu), cuda(table), cuda(ctx.astype(np.int32)), max(new))
    write_block(host, k, v, cu, table, ctx)
    assert_same(cache, host)
    # the same tokens again: their scales are in place, nothing changes but the
    # codes that a grown scale rounds again (there are none left)
    pk.kv_write_block_quant(cache, cuda(k), cuda(v), cuda(cu), cuda(table), cuda(ctx.astype(np.int32)), max(new))
    assert_same(cache, host, "again")


@pytest.mark.parametrize("fmt", BLOCK)
def test_write_special_values(fmt):
    """All fp16 patterns (infinities, NaN, subnormals), an all-zero block, signed zeros."""
    bs, hkv = 16, 2
    bits = np.arange(65536, dtype=np.uint16).view(np.float16)
    k = np.zeros((512, hkv, D), np.float16)
    k[:, 1] = bits.reshape(512, D)
    k[:, 0] = -0.0
    v = np.zeros_like(k)
    # blocks of subnormals only, and one of ordinary values with one infinity
    v[:256, 0] = (np.arange(256 * D, dtype=np.uint16) % 1024).view(np.float16).reshape(256, D)
    v[256:, 0] = np.random.default_rng(3).standard_normal((256, D))
    v[300, 0, 7] = np.inf
    v[316, 0, 9] = np.nan
    ctx = [512]
    blocks, table, _ = lay_out(ctx, bs, 4)
    cache = random_cache(fmt, blocks, bs, hkv, 5)
    host = Host(cache)
    cu = np.array([0, 512], np.int32)
    pk.kv_write_block_quant(cache, cuda(k), cuda(v), cuda(cu), cuda(table), cuda(np.int32(ctx)), 512)
    with np.errstate(invalid="ignore"):
        write_block(host, k, v, cu, table, ctx)
    assert_same(cache, host)


def test_step_by_step_equals_definition():
    """A prompt and 40 single-token steps: scales grow, codes are rounded again."""
    bs, hkv, fmt = 16, 2, pk.KV_INT8_BLOCK
    r = np.random.default_rng(6)
    total = 21 + 40
    blocks, table, _ = lay_out([total], bs, 7)
    cache = random_cache(fmt, blocks, bs, hkv, 8)
    host = Host(cache)
    k, v = new_rows(r, total, hkv), new_rows(r, total, hkv)
    k *= np.linspace(0.1, 3, total)[:, None, None].astype(np.float16)
    at = 0
    for n in [21] + [1] * 40:
        cu, ctx = np.array([0, n], np.int32), np.array([at + n], np.int32)
        pk.kv_write_block_quant(cache, cuda(k[at:at + n]), cuda(v[at:at + n]), cuda(cu), cuda(table), cuda(ctx), n)
        write_block(host, k[at:at + n], v[at:at + n], cu, table, ctx)
        at += n
    assert_same(cache, host)


def test_write_skips_positions_below_zero_and_foreign_rows():
    bs, hkv, fmt = 16, 1, pk.KV_E4M3_BLOCK
    blocks, table, _ = lay_out([20, 9], bs, 9)
    cache = random_cache(fmt, blocks, bs, hkv, 10)
    host = Host(cache)
    r = np.random.default_rng(11)
    k, v = new_rows(r, 25 + 9, hkv), new_rows(r, 25 + 9, hkv)
    cu, ctx = np.array([0, 25, 34], np.int32), np.array([20, 9], np.int32)   # 5 positions below 0
    pk.kv_write_block_quant(cache, cuda(k), cuda(v), cuda(cu), cuda(table), cuda(ctx), 25)
    write_block(host, k, v, cu, table, ctx)
    assert_same(cache, host)


def check_rows(out, lse, q, host, table, b, ctx, pos, hq, window=0, what="",
               scale=SCALE):
    """out / lse [rows][Hq] of one sequence against the reference."""
    G = hq // host.hkv
    for h in range(host.hkv):
        keys, vals = host.rows("k", table[b], h, ctx), host.rows("v", table[b], h, ctx)
        vmax = float(np.abs(vals).max(initial=0.0)) * 2
        if host.fmt in BLOCK:
            nb = -(-ctx // host.bs)
            vmax = max(vmax, QMAX[host.fmt] * float(host.vs[table[b][:nb], h].max(initial=0.0)))
        for g in range(h * G, (h + 1) * G):
            ref, rl, _, a, sabs = attention(q[:, g], keys, vals, pos, scale, window)
            err = np.abs(out[:, g] - ref)
            bound = out_bound(ref, a, ctx, vmax, sabs)
            assert np.isfinite(out[:, g]).all() and (err <= bound).all(), \
                f"{what} seq {b} head {g}: {float((err - bound).max()):.2e} above its bound"
            fin = np.isfinite(rl)
            assert np.array_equal(np.isfinite(lse[:, g]), fin), what
            assert (np.abs(lse[:, g] - rl)[fin] <= lse_bound(sabs)).all(), what


def queries(r, *shape):
    return (1.5 * r.standard_normal(shape)).astype(np.float16)


DECODE = [
    # fmt, Hq, Hkv, bs, contexts, q_len, window
    (pk.KV_INT8_BLOCK, 8, 2, 16, [1, 2, 16, 17, 0], 1, 0),
    (pk.KV_E4M3_BLOCK, 8, 2, 16, [5000, 33, 700], 1, 0),
    (pk.KV_INT8_BLOCK, 32, 4, 16, [6001], 1, 0),
    (pk.KV_E4M3_BLOCK, 6, 1, 32, [1999, 64], 1, 0),
    (pk.KV_INT8_BLOCK, 5, 5, 64, [130, 65, 1000], 1, 0),       # MHA
    (pk.KV_INT8_BLOCK, 16, 1, 64, [777, 3], 1, 0),             # 16 rows
    (pk.KV_E4M3_BLOCK, 8, 4, 16, [900, 3], 5, 0),              # q_len > context for one
    (pk.KV_INT8_BLOCK, 32, 4, 16, [3000, 100, 2], 5, 0),       # 40 rows: tensor-core kernel
    (pk.KV_E4M3_BLOCK, 32, 4, 32, [2500, 641], 5, 0),
    (pk.KV_INT8_BLOCK, 32, 4, 64, [1500], 16, 0),              # 128 rows
    (pk.KV_E4M3_BLOCK, 16, 1, 16, [1100, 31], 9, 0),           # 144 rows: row groups
    (pk.KV_INT8_BLOCK, 8, 2, 16, [3000, 40, 90], 1, 50),
    (pk.KV_E4M3_BLOCK, 32, 4, 16, [2000, 400], 5, 133),
]


@pytest.mark.parametrize("fmt,hq,hkv,bs,ctx,ql,window", DECODE)
def test_decode(fmt, hq, hkv, bs, ctx, ql, window):
    r = np.random.default_rng(12)
    blocks, table, _ = lay_out(ctx, bs, 13)
    cache = random_cache(fmt, blocks, bs, hkv, 14)
    host = Host(cache)
    # what lies behind the contexts, and every block outside them, is poison
    for b, c in enumerate(ctx):
        if c % bs:
            cache.k_cache[int(table[b][c // bs]), :, c % bs:] = 0x7F
            cache.v_cache[int(table[b][c // bs]), :, c % bs:] = 0x7F
    used = np.unique(table[table >= 0])
    free = np.setdiff1d(np.arange(blocks), used)
    for t in (cache.k_scale_blk, cache.v_scale_blk):
        t[cuda(free)] = float("nan")
    q = queries(r, len(ctx), ql, hq, D)
    lse = torch.empty((len(ctx), ql, hq), device="cuda")
    out = pk.paged_attn_decode(cache, cuda(q), cuda(table), cuda(np.int32(ctx)), max(ctx), SCALE, lse=lse,
                               sliding_window=window)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, c in enumerate(ctx):
        check_rows(out[b], lse[b], q[b].astype(float), host, table, b, c, c - ql + np.arange(ql), hq, window)
    assert pk.device_status() == 0


@pytest.mark.parametrize("fmt,hq,ql,bs", [(pk.KV_INT8_BLOCK, 8, 1, 16), (pk.KV_E4M3_BLOCK, 8, 2, 32),
                                          (pk.KV_INT8_BLOCK, 16, 5, 16)])
def test_many_sequences_share_the_splits(fmt, hq, ql, bs):
    """More than 32 sequences of very different lengths: every key has a split."""
    r = np.random.default_rng(54)
    hkv = 2
    ctx = [int(x) for x in r.choice([0, 1, 15, 16, 17, 200, 700, 1500], 43)]
    blocks, table, _ = lay_out(ctx, bs, 55)
    cache = random_cache(fmt, blocks, bs, hkv, 56)
    host = Host(cache)
    q = queries(r, len(ctx), ql, hq, D)
    lse = torch.empty((len(ctx), ql, hq), device="cuda")
    # (the bound may lie above every length)
    out = pk.paged_attn_decode(cache, cuda(q), cuda(table), cuda(np.int32(ctx)), table.shape[1] * bs, SCALE, lse=lse)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, c in enumerate(ctx):
        check_rows(out[b], lse[b], q[b].astype(float), host, table, b, c, c - ql + np.arange(ql), hq)


@pytest.mark.parametrize("fmt", BLOCK)
def test_decode_scale_zero_huge_and_tiny(fmt):
    """Blocks whose V scale is 0 (all codes 0), 2^9 and 2^-33: no overflow, no lost rows."""
    bs, hkv, hq, ctx = 16, 1, 4, [400]
    blocks, table, _ = lay_out(ctx, bs, 15)
    cache = random_cache(fmt, blocks, bs, hkv, 16)
    cache.v_scale_blk[:] = 2.0 ** -33
    cache.k_scale_blk[int(table[0][3])] = 0.0
    cache.k_cache[int(table[0][3])] = 0
    cache.v_scale_blk[int(table[0][4])] = 0.0
    cache.v_cache[int(table[0][4])] = 0
    r = np.random.default_rng(17)
    for loud in (None, 7):
        if loud is not None:
            cache.v_scale_blk[int(table[0][loud])] = 500.0
        host = Host(cache)
        q = queries(r, 1, 1, hq, D)
        lse = torch.empty((1, 1, hq), device="cuda")
        out = pk.paged_attn_decode(cache, cuda(q), cuda(table), cuda(np.int32(ctx)), 400, SCALE, lse=lse)
        # (an output over 65504 is fp16's infinity: keep it below)
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        check_rows(out[0], lse[0], q[0].astype(float), host, table, 0, 400, np.array([399]), hq)


PREFILL = [
    # fmt, Hq, Hkv, bs, contexts, chunks, window
    (pk.KV_INT8_BLOCK, 8, 1, 16, [300], [300], 0),
    (pk.KV_E4M3_BLOCK, 32, 4, 16, [200, 1000, 5], [200, 37, 0], 0),
    (pk.KV_INT8_BLOCK, 8, 8, 32, [129, 64], [129, 1], 0),
    (pk.KV_E4M3_BLOCK, 12, 2, 64, [700], [333], 0),
    (pk.KV_INT8_BLOCK, 16, 2, 16, [1000, 80], [400, 80], 100),
]


@pytest.mark.parametrize("fmt,hq,hkv,bs,ctx,chunk,window", PREFILL)
def test_prefill(fmt, hq, hkv, bs, ctx, chunk, window):
    r = np.random.default_rng(18)
    blocks, table, _ = lay_out(ctx, bs, 19)
    cache = random_cache(fmt, blocks, bs, hkv, 20)
    host = Host(cache)
    cu = np.concatenate([[0], np.cumsum(chunk)]).astype(np.int32)
    q = queries(r, cu[-1], hq, D)
    lse = torch.empty((cu[-1], hq), device="cuda")
    out = pk.paged_attn_prefill(cache, cuda(q), cuda(cu), cuda(table), cuda(np.int32(ctx)), max(chunk), SCALE,
                                lse=lse, sliding_window=window)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, (c, n) in enumerate(zip(ctx, chunk)):
        s = slice(cu[b], cu[b + 1])
        check_rows(out[s], lse[s], q[s].astype(float), host, table, b, c, c - n + np.arange(n), hq, window)
    assert pk.device_status() == 0


@pytest.mark.parametrize("scale", [0.0, -0.07, 1e-25])
@pytest.mark.parametrize("ql,hq", [(1, 8), (5, 16), (12, 16), (150, 8)])
def test_other_softmax_scales(scale, ql, hq):
    """Uniform weights and negated scores, in all four kernels (mma.sync decode,
    tensor-core decode up to 64 and up to 128 rows, prefill)."""
    fmt, bs, hkv, ctx = pk.KV_INT8_BLOCK, 16, 2, [333]
    blocks, table, _ = lay_out(ctx, bs, 51)
    cache = random_cache(fmt, blocks, bs, hkv, 52)
    host = Host(cache)
    q = queries(np.random.default_rng(53), ql, hq, D)
    t, c = cuda(table), cuda(np.int32(ctx))
    lse = torch.empty((ql, hq), device="cuda")
    if ql <= 16:
        out = pk.paged_attn_decode(cache, cuda(q[None]), t, c, 333, scale, lse=lse[None])[0]
    else:
        out = pk.paged_attn_prefill(cache, cuda(q), cuda(np.int32([0, ql])), t, c, ql, scale, lse=lse)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    sign = -1.0 if scale < 0 else 1.0     # the reference's magnitudes take |scale|
    check_rows(out, lse, sign * q.astype(float), host, table, 0, 333, 333 - ql + np.arange(ql), hq,
               scale=abs(scale))


@pytest.mark.parametrize("fmt", BLOCK)
@pytest.mark.parametrize("hq,hkv,ql", [(8, 2, 1), (8, 2, 3), (32, 4, 5)])
def test_append_equals_write_then_decode(fmt, hq, hkv, ql):
    bs, ctx = 16, [500, 18, 33]
    r = np.random.default_rng(21)
    blocks, table, _ = lay_out(ctx, bs, 22)
    a = random_cache(fmt, blocks, bs, hkv, 23)
    b = random_cache(fmt, blocks, bs, hkv, 23)
    k, v = new_rows(r, len(ctx) * ql, hkv), new_rows(r, len(ctx) * ql, hkv)
    q = cuda(queries(r, len(ctx), ql, hq, D))
    cu = cuda(np.arange(len(ctx) + 1, dtype=np.int32) * ql)
    t, c = cuda(table), cuda(np.int32(ctx))
    pk.kv_write_block_quant(a, cuda(k), cuda(v), cu, t, c, ql)
    oa = pk.paged_attn_decode(a, q, t, c, max(ctx), SCALE)
    shape = (len(ctx), ql, hkv, D)
    ob = pk.paged_attn_decode_append(b, cuda(k).view(shape), cuda(v).view(shape), q, t, c, max(ctx), SCALE)
    assert torch.equal(oa, ob)
    assert torch.equal(a.k_cache, b.k_cache) and torch.equal(a.v_cache, b.v_cache)
    assert torch.equal(a.k_scale_blk, b.k_scale_blk) and torch.equal(a.v_scale_blk, b.v_scale_blk)


@pytest.mark.parametrize("fmt", BLOCK)
def test_copy_blocks_moves_the_scales(fmt):
    src = random_cache(fmt, 9, 16, 3, 24)
    dst = random_cache(fmt, 7, 16, 3, 25)
    keep = Host(dst)
    pairs = torch.tensor([[0, 3], [8, 1], [4, 6]], dtype=torch.int32, device="cuda")
    pk.kv_copy_blocks(dst, src, pairs)
    torch.cuda.synchronize()
    for s, d in pairs.tolist():
        assert torch.equal(dst.k_cache[d], src.k_cache[s]) and torch.equal(dst.v_cache[d], src.v_cache[s])
        assert torch.equal(dst.k_scale_blk[d], src.k_scale_blk[s])
        assert torch.equal(dst.v_scale_blk[d], src.v_scale_blk[s])
    for d in (0, 2, 4, 5):
        assert np.array_equal(dst.k_cache[d].cpu().numpy(), keep.k[d])
        assert np.array_equal(dst.k_scale_blk[d].cpu().numpy(), keep.ks[d])


def test_captured_step_replays_on_another_stream():
    """Write and decode of one step, captured once and replayed with new inputs."""
    fmt, bs, hq, hkv, ctx = pk.KV_E4M3_BLOCK, 16, 8, 2, [700, 90]
    r = np.random.default_rng(26)
    blocks, table, _ = lay_out(ctx, bs, 27)
    cache = random_cache(fmt, blocks, bs, hkv, 28)
    host = Host(cache)
    t, c = cuda(table), cuda(np.int32(ctx))
    k, v = (torch.zeros((2, 1, hkv, D), dtype=torch.float16, device="cuda") for _ in "kv")
    q = torch.zeros((2, 1, hq, D), dtype=torch.float16, device="cuda")
    out = torch.empty_like(q)
    lse = torch.empty((2, 1, hq), device="cuda")
    ws = torch.empty(max(1, pk.decode_workspace_bytes(cache, 2, 1, hq, max(ctx))), dtype=torch.uint8, device="cuda")
    before = [x.clone() for x in (cache.k_cache, cache.v_cache, cache.k_scale_blk, cache.v_scale_blk)]

    def step():
        pk.paged_attn_decode_append(cache, k, v, q, t, c, max(ctx), SCALE, out=out, lse=lse, workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for x, y in zip((cache.k_cache, cache.v_cache, cache.k_scale_blk, cache.v_scale_blk), before):
        x.copy_(y)
    kn, vn, qn = new_rows(r, 2, hkv), new_rows(r, 2, hkv), queries(r, 2, 1, hq, D)
    k.copy_(cuda(kn).view(2, 1, hkv, D)), v.copy_(cuda(vn).view(2, 1, hkv, D)), q.copy_(cuda(qn))
    graph.replay()
    torch.cuda.synchronize()
    write_block(host, kn, vn, np.array([0, 1, 2]), table, ctx)
    assert_same(cache, host)
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, n in enumerate(ctx):
        check_rows(o[b], l[b], qn[b].astype(float), host, table, b, n, np.array([n - 1]), hq)
