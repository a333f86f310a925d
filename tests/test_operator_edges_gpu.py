"""GPU: the block-scaled caches, weights, eviction and prompt attention at their
edges: offsets past 32 bits, other streams, the entry point without workspace,
explicit query positions, the bounds-checking build, padded and empty batches,
and the calls that the binding refuses."""
import ctypes

import numpy as np
import pytest
import torch

import paged_quantized_kv_quant_b200 as pk
from paged_quantized_kv_quant_b200 import build as pkbuild
from pkvq_ref64 import BLOCK, D, Host, lay_out, random_cache, write_block
from test_block_scale_gpu import SCALE, assert_same, check_rows, cuda, new_rows, queries
from test_evict_gpu import run_weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", BLOCK)
def test_offsets_past_32_bits(fmt):
    """The same call on a small pool and in the last blocks of a pool of over
    2^32 bytes: the same bits."""
    bs, hq, hkv, ctx, budget = 64, 8, 2, [900, 130], 100
    r = np.random.default_rng(61)
    blocks, table, dst = lay_out(ctx, bs, 62, spare=2)
    small = random_cache(fmt, blocks, bs, hkv, 63)
    big_blocks = (1 << 32) // (hkv * bs * D) + 1000
    shift = big_blocks - blocks
    big = pk.PagedKVCache(fmt, *(torch.empty((big_blocks, hkv, bs, D), dtype=torch.uint8, device="cuda") for _ in "kv"),
                          k_scale_blk=torch.ones((big_blocks, hkv), device="cuda"),
                          v_scale_blk=torch.ones((big_blocks, hkv), device="cuda"))
    for a, b in ((small.k_cache, big.k_cache), (small.v_cache, big.v_cache),
                 (small.k_scale_blk, big.k_scale_blk), (small.v_scale_blk, big.v_scale_blk)):
        b[shift:] = a
    k, v, q = new_rows(r, 33, hkv), new_rows(r, 33, hkv), cuda(queries(r, 2, 1, hq, D))
    cu, c = cuda(np.int32([0, 30, 33])), cuda(np.int32(ctx))
    got = []
    for cache, t, d in ((small, table, dst), (big, np.where(table >= 0, table + shift, -1), dst + shift)):
        t, d = cuda(t.astype(np.int32)), cuda(d.astype(np.int32))
        pk.kv_write_block_quant(cache, cuda(k), cuda(v), cu, t, c, 30)
        W = torch.zeros((2, hkv, 900), device="cuda")
        out, lse = run_weights(cache, q, t, c, W)
        out2 = pk.paged_attn_prefill(cache, q.view(2, hq, D), cuda(np.int32([0, 1, 2])), t, c, 1, SCALE)
        out3 = pk.paged_attn_decode(cache, q.expand(2, 5, hq, D).contiguous(), t, c, 900, SCALE)
        lens, w2, keep = pk.kv_evict(cache, W, t, c, d, budget, 4, 20)
        out4 = pk.paged_attn_decode(cache, q, d, lens, budget, SCALE)
        got.append([out, lse, W, out2, out3, lens, w2, keep, out4])
    for a, b in zip(*got):
        assert torch.equal(a, b)
    for a, b in ((small.k_cache, big.k_cache), (small.v_cache, big.v_cache),
                 (small.k_scale_blk, big.k_scale_blk), (small.v_scale_blk, big.v_scale_blk)):
        assert torch.equal(b[shift:], a)
    assert pk.device_status() == 0


def test_two_streams_at_once():
    """The same steps on two streams with their own caches and workspaces,
    enqueued without waiting, equal the steps alone."""
    hq, hkv, bs, ctx = 16, 2, 16, [3000, 500]
    r = np.random.default_rng(64)
    blocks, table, dst = lay_out(ctx, bs, 65, spare=16)
    t, c, d = cuda(table), cuda(np.int32(ctx)), cuda(dst)
    qs = [cuda(queries(r, 2, 1, hq, D)) for _ in range(2)]
    pr = [[torch.randn((400, n, D), device="cuda").half() for n in (hq, hkv, hkv)] for _ in range(2)]
    cu = cuda(np.int32([0, 150, 400]))

    def steps(i, cache, stream=None):
        W = torch.zeros((2, hkv, 3000), device="cuda")
        o = [pk.prompt_attn(*pr[i], cu, 250, SCALE, stream=stream)]
        for _ in range(5):
            o.append(pk.paged_attn_decode_weights(cache, qs[i], t, c, 3000, SCALE, W, stream=stream))
        o += list(pk.kv_evict(cache, W, t, c, d, 256, 4, 16, stream=stream)) + [W]
        return o

    alone = [steps(i, random_cache(BLOCK[i], blocks, bs, hkv, 66)) for i in range(2)]
    caches = [random_cache(BLOCK[i], blocks, bs, hkv, 66) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    both = []
    for i in range(2):
        with torch.cuda.stream(streams[i]):
            both.append(steps(i, caches[i], stream=streams[i]))
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


@pytest.mark.parametrize("fmt", BLOCK)
def test_decode_without_workspace(fmt):
    ctx, hq, hkv, bs = [2000, 77], 8, 2, 16
    blocks, table, _ = lay_out(ctx, bs, 67)
    cache = random_cache(fmt, blocks, bs, hkv, 68)
    q = cuda(queries(np.random.default_rng(69), 2, 1, hq, D))
    t, c = cuda(table), cuda(np.int32(ctx))
    ref = pk.paged_attn_decode(cache, q, t, c, 2000, SCALE)
    out = torch.empty_like(q)
    cs = cache.struct()
    rc = pk._lib().pkvq_paged_attn_decode_noalloc(
        ctypes.byref(cs), q.data_ptr(), out.data_ptr(), None, t.data_ptr(), t.shape[1], c.data_ptr(),
        2, 1, hq, 2000, ctypes.c_float(SCALE), torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and torch.equal(out, ref)


@pytest.mark.parametrize("fmt", BLOCK)
@pytest.mark.parametrize("ql", [1, 5])
def test_query_positions(fmt, ql):
    """Positions given per query (-1: sees nothing), with and without weights."""
    ctx, hq, hkv, bs = [300, 64], 32, 4, 16
    r = np.random.default_rng(70)
    blocks, table, _ = lay_out(ctx, bs, 71)
    cache = random_cache(fmt, blocks, bs, hkv, 72)
    host = Host(cache)
    pos = np.array([r.integers(-1, n, ql) for n in ctx], np.int32)
    pos[1, 0] = -1
    q = queries(r, 2, ql, hq, D)
    t, c = cuda(table), cuda(np.int32(ctx))
    for weights in (False, True):
        lse = torch.empty((2, ql, hq), device="cuda")
        if weights:
            W = torch.zeros((2, hkv, 300), device="cuda")
            out = pk.paged_attn_decode_weights(cache, cuda(q), t, c, 300, SCALE, W, lse=lse, query_pos=cuda(pos))
            rows = (pos >= 0).sum(1) * (hq // hkv)       # every row that sees a key spends 1
            assert torch.allclose(W.double().sum(-1).cpu(), torch.tensor(rows)[:, None].double().expand(2, hkv),
                                  rtol=3e-4, atol=0)
        else:
            out = pk.paged_attn_decode(cache, cuda(q), t, c, 300, SCALE, lse=lse, query_pos=cuda(pos))
        o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for b, n in enumerate(ctx):
            check_rows(o[b], l[b], q[b].astype(float), host, table, b, n, pos[b], hq)


def test_checked_build_gives_the_same_bits():
    """In-range calls: the bounds-checking build's results and a clean status."""
    path = pkbuild.build(bounds_check=True)
    ctx, hq, hkv, bs = [700, 45], 8, 2, 16
    blocks, table, dst = lay_out(ctx, bs, 73, spare=8)
    r = np.random.default_rng(74)
    k, v, q = new_rows(r, 20, hkv), new_rows(r, 20, hkv), cuda(queries(r, 2, 1, hq, D))
    cu, t, c, d = cuda(np.int32([0, 17, 20])), cuda(table), cuda(np.int32(ctx)), cuda(dst)
    p = [cuda(queries(r, 200, n, D)) for n in (hq, hkv, hkv)]

    def calls(fmt):
        cache = random_cache(fmt, blocks, bs, hkv, 75)
        if fmt in BLOCK:
            pk.kv_write_block_quant(cache, cuda(k), cuda(v), cu, t, c, 17)
        W = torch.zeros((2, hkv, 700), device="cuda")
        out, lse = run_weights(cache, q, t, c, W)
        res = list(pk.kv_evict(cache, W, t, c, d, 100, 2, 9))
        prompt = pk.prompt_attn(*p, cuda(np.int32([0, 150, 200])), 150, SCALE)
        return res + [out, lse, W, cache.k_cache, cache.v_cache, prompt]

    for fmt in BLOCK + (pk.KV_INT8,):
        a = calls(fmt)
        assert pk.device_status() == 0
        with pk.use_library(path):
            b = calls(fmt)
            assert pk.device_status() == 0
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_empty_calls_do_nothing():
    cache = random_cache(pk.KV_INT8_BLOCK, 4, 16, 2, 76)
    host = Host(cache)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    h16 = lambda *s: torch.zeros(s, dtype=torch.float16, device="cuda")  # noqa: E731
    f32 = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    pk.kv_write_block_quant(cache, h16(0, 2, D), h16(0, 2, D), i32(1), i32(0, 3), i32(0), 0)
    pk.kv_write_block_quant(cache, h16(5, 2, D), h16(5, 2, D), i32(3), i32(2, 3), i32(2), 4)   # no new tokens
    assert pk.paged_attn_decode_weights(cache, h16(0, 1, 4, D), i32(0, 3), i32(0), 16, 1.0, f32(0, 2, 16)).shape[0] == 0
    lens, w, keep = pk.kv_evict(cache, f32(0, 2, 16), i32(0, 3), i32(0), i32(0, 3), 4)
    assert lens.numel() == 0 and keep.shape == (0, 2, 4)
    assert pk.prompt_attn(h16(0, 4, D), h16(0, 2, D), h16(0, 2, D), i32(1), 0, 1.0).shape == (0, 4, D)
    out = pk.prompt_attn(h16(3, 4, D), h16(3, 2, D), h16(3, 2, D), i32(2), 5, 1.0, out=torch.ones((3, 4, D), device="cuda").half())
    assert (out == 1).all()                              # one empty sequence: nothing is written
    # sequences of no tokens among others keep their accumulators and get zeros
    W = torch.ones((2, 2, 32), device="cuda")
    out, lse = run_weights(cache, torch.ones((2, 1, 4, D), device="cuda").half(), i32(2, 3), i32(2), W)
    assert (out == 0).all() and torch.isinf(lse).all() and (W == 1).all()
    lens, w, keep = pk.kv_evict(cache, W, i32(2, 3), i32(2), i32(2, 1), 8)
    assert (lens == 0).all() and (keep == -1).all() and (w == 0).all()
    assert_same(cache, host)


def test_rows_that_are_not_there_are_skipped():
    """Sequence boundaries that point outside K and V write nothing and fault nothing."""
    blocks, table, _ = lay_out([40, 40], 16, 77)
    cache = random_cache(pk.KV_E4M3_BLOCK, blocks, 16, 2, 78)
    host = Host(cache)
    r = np.random.default_rng(79)
    k, v = new_rows(r, 20, 2), new_rows(r, 20, 2)
    ctx = np.int32([40, 40])
    pk.kv_write_block_quant(cache, cuda(k), cuda(v), cuda(np.int32([0, 20, 60])), cuda(table), cuda(ctx), 40)
    write_block(host, k, v, np.array([0, 20]), table, ctx[:1])
    assert_same(cache, host)
    q, kk = cuda(queries(r, 20, 4, D)), cuda(queries(r, 20, 2, D))
    out = torch.full((24, 4, D), 3.0, dtype=torch.float16, device="cuda")
    pk.prompt_attn(q, kk, kk, cuda(np.int32([0, 20, 60, 50])), 40, SCALE, out=out[:20])
    assert (out[20:] == 3).all() and (out[:20] != 3).any()
    pk.prompt_attn(q, kk, kk, cuda(np.int32([-9, 20])), 40, SCALE, out=out[:20].fill_(3))
    assert (out == 3).all()
    assert pk.device_status() == 0


def test_binding_refuses_what_the_kernels_cannot_take():
    cache = random_cache(pk.KV_INT8_BLOCK, 8, 16, 2, 80)
    t, c = torch.zeros((2, 4), dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    q = torch.zeros((2, 1, 4, D), dtype=torch.float16, device="cuda")
    W = torch.zeros((2, 2, 64), device="cuda")
    good = dict(cache=cache, q=q, block_table=t, context_lens=c, max_context_len=64, softmax_scale=1.0)
    for kw in (dict(q=q.float()), dict(q=q[..., :64]), dict(q=q.transpose(1, 2)), dict(q=q[0]),
               dict(block_table=t[:1]), dict(block_table=t.long()), dict(block_table=t[:, ::2]),
               dict(context_lens=c[:1]), dict(context_lens=c.cpu()), dict(context_lens=c[:, None])):
        # (PkvqError: a transposed q is one query head of two KV heads, which the library refuses)
        with pytest.raises((ValueError, TypeError, pk.PkvqError)):
            pk.paged_attn_decode(**{**good, **kw})
        with pytest.raises((ValueError, TypeError, pk.PkvqError)):
            pk.paged_attn_decode_weights(**{**good, **kw}, weights=W)
    for w in (W[:1], W[:, :1], W.double(), W[..., ::2], W.cpu(), W[0]):
        with pytest.raises((ValueError, TypeError)):
            pk.paged_attn_decode_weights(**good, weights=w)
    with pytest.raises(pk.PkvqError):
        pk.paged_attn_decode_weights(**good, weights=W[..., :32].contiguous())
    with pytest.raises(pk.PkvqError):                    # a workspace for fewer sequences
        pk.paged_attn_decode_weights(**good, weights=W, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(pk.PkvqError):                    # not this format's write
        pk.kv_write_quant(cache, *(q[:, 0, :2].contiguous() for _ in "kv"), c)
    x = torch.zeros((30, 4, D), dtype=torch.float16, device="cuda")
    cu = torch.tensor([0, 30], dtype=torch.int32, device="cuda")
    for a in ((x, x[:, :2], x[:, :2].float()), (x.float(),) * 3, (x, x[:, :3], x[:, :3]), (x, x[:20, :2], x[:20, :2]),
              (x[..., ::2], x[:, :2, ::2], x[:, :2, ::2]), (x, x[:, :2].cpu(), x[:, :2]),
              (x[:, 1:, 4:], x[:, :1, 4:], x[:, :1, 4:])):
        with pytest.raises((ValueError, TypeError, pk.PkvqError)):
            pk.prompt_attn(*a, cu, 30, 1.0)
    flat = torch.zeros(30 * 2 * D + 4, dtype=torch.float16, device="cuda")
    off = flat[4:].view(30, 2, D)                        # 8 bytes off a 16-byte boundary
    with pytest.raises(pk.PkvqError):
        pk.prompt_attn(x, off, off, cu, 30, 1.0)
    with pytest.raises(ValueError):                      # scales of another pool
        pk.PagedKVCache(pk.KV_INT8_BLOCK, cache.k_cache, cache.v_cache, k_scale_blk=cache.k_scale_blk[:4],
                        v_scale_blk=cache.v_scale_blk).struct()
    assert pk.device_status() == 0


def test_a_cache_object_follows_its_tensors():
    """The kept C struct is renewed when a tensor of the cache is replaced."""
    a, b = (random_cache(pk.KV_INT8_BLOCK, 8, 16, 2, s) for s in (81, 82))
    t, c = torch.arange(4, dtype=torch.int32, device="cuda")[None], torch.tensor([50], dtype=torch.int32, device="cuda")
    q = cuda(queries(np.random.default_rng(83), 1, 1, 4, D))
    call = lambda x: pk.paged_attn_decode(x, q, t, c, 50, SCALE)  # noqa: E731
    oa, ob = call(a), call(b)
    assert not torch.equal(oa, ob)
    a.k_cache, a.v_cache, a.k_scale_blk, a.v_scale_blk = b.k_cache, b.v_cache, b.k_scale_blk, b.v_scale_blk
    assert torch.equal(call(a), ob)
    a.v_scale_blk = a.v_scale_blk.double()
    with pytest.raises(TypeError):
        call(a)
