"""GPU: decode that accumulates attention weights, and eviction by them,
against 64-bit references, for every cache format."""
import numpy as np
import pytest
import torch

import paged_quantized_kv_quant_b200 as pk
from pkvq_ref64 import ALL, BLOCK, D, Host, attention, evict, lay_out, random_cache, write_block
from test_block_scale_gpu import SCALE, assert_same, check_rows, cuda, new_rows, queries

pytestmark = pytest.mark.gpu

STEPS = [
    # Hq, Hkv, bs, contexts, q_len, window
    (8, 2, 16, [701, 1, 17, 0], 1, 0),
    (32, 4, 16, [5000, 4999, 33], 1, 0),          # several splits
    (4, 4, 32, [600, 31], 1, 0),                  # one row per KV head
    (4, 2, 64, [1300], 1, 0),                     # two rows
    (6, 2, 16, [400, 50], 1, 0),                  # three rows (padded to four)
    (16, 1, 16, [900], 1, 0),                     # sixteen rows
    (8, 2, 32, [1025, 3, 2], 5, 0),               # 20 rows: two row groups; q_len > context
    (32, 4, 16, [2100, 64], 5, 0),                # 40 rows
    (16, 1, 64, [500], 16, 0),                    # 256 rows
    (8, 2, 16, [2000, 20], 1, 77),
    (8, 2, 16, [900, 5], 3, 40),
]


def run_weights(cache, q, table, ctx, weights, **kw):
    lse = torch.empty(q.shape[:3], device="cuda")
    out = pk.paged_attn_decode_weights(cache, q, table, ctx, int(ctx.max()), SCALE, weights, lse=lse, **kw)
    return out, lse


@pytest.mark.parametrize("fmt", ALL)
@pytest.mark.parametrize("hq,hkv,bs,ctx,ql,window", STEPS)
def test_weights(fmt, hq, hkv, bs, ctx, ql, window):
    r = np.random.default_rng(31)
    blocks, table, _ = lay_out(ctx, bs, 32)
    cache = random_cache(fmt, blocks, bs, hkv, 33)
    host = Host(cache)
    q = queries(r, len(ctx), ql, hq, D)
    W0 = r.uniform(0, 1, (len(ctx), hkv, max(ctx) + 5)).astype(np.float32)
    W = cuda(W0)
    t, c = cuda(table), cuda(np.int32(ctx))
    out, lse = run_weights(cache, cuda(q), t, c, W, sliding_window=window)
    # (row groups instead of the tensor-core kernel may round P elsewhere: the
    # same bounds, not the same bits, as paged_attn_decode)
    o, l, w = out.double().cpu().numpy(), lse.double().cpu().numpy(), W.double().cpu().numpy()
    G = hq // hkv
    for b, n in enumerate(ctx):
        pos = n - ql + np.arange(ql)
        check_rows(o[b], l[b], q[b].astype(float), host, table, b, n, pos, hq, window)
        for h in range(hkv):
            ref, mass = W0[b, h].astype(np.float64).copy(), 0.0
            keys, vals = host.rows("k", table[b], h, n), host.rows("v", table[b], h, n)
            worst = np.zeros(n)
            for g in range(h * G, (h + 1) * G):
                _, _, p, _, sabs = attention(q[b, :, g].astype(float), keys, vals, pos, SCALE, window)
                ref[:n] += p.sum(0)
                # a weight's relative error: its score's and its normaliser's
                # (129 fp32 products each, truncated), the exponentials' 2^-21
                worst += p.sum(0) * (2 * 129 * 2.0 ** -23 * sabs + 2.0 ** -19)
            bound = worst + 2.0 ** -22 * (np.abs(ref[:n]) + 1)   # sums of fp32 numbers
            assert (np.abs(w[b, h, :n] - ref[:n]) <= bound).all()
            assert np.array_equal(w[b, h, n:], W0[b, h, n:].astype(np.float64))
            live = np.abs(w[b, h, :n] - ref[:n])
            assert np.linalg.norm(live) <= 2e-5 * max(1e-30, np.linalg.norm(ref[:n]))
    # the same call gives the same bits
    W2 = cuda(W0)
    out2, lse2 = run_weights(cache, cuda(q), t, c, W2, sliding_window=window)
    assert torch.equal(out, out2) and torch.equal(lse, lse2) and torch.equal(W, W2)
    assert pk.device_status() == 0


def test_weights_rows_sum_to_the_number_of_query_rows():
    """Every query row spends a weight of 1, however large the scores are."""
    fmt, bs, hq, hkv, ctx = pk.KV_FP16, 16, 8, 2, [3000, 40]
    blocks, table, _ = lay_out(ctx, bs, 34)
    cache = random_cache(fmt, blocks, bs, hkv, 35)
    W = torch.zeros((2, hkv, 3000), device="cuda")
    q = cuda(queries(np.random.default_rng(36), 2, 1, hq, D) * np.float16(30))
    run_weights(cache, q, cuda(table), cuda(np.int32(ctx)), W)
    assert torch.allclose(W.double().sum(-1), torch.full((2, hkv), 4.0, dtype=torch.float64, device="cuda"),
                          atol=0, rtol=3e-4)   # 2 * 129 * 2^-23 * sabs (~ 10) in the scores


EVICT = [
    # contexts, budget, sink, recent, bs
    ([500, 90, 0, 1], 65, 4, 16, 16),
    ([64, 65, 63], 64, 1, 1, 32),
    ([1000, 200], 33, 0, 0, 64),
    ([300, 301], 20, 5, 15, 16),             # nothing to choose: sinks and recent fill the budget
    ([5000, 4097, 4096], 1000, 4, 100, 16),  # several ranking rounds
    ([40], 1, 0, 1, 16),
    ([40], 1, 0, 0, 16),
    ([33], 100, 4, 4, 16),                   # below the budget: all stay
]


@pytest.mark.parametrize("fmt", ALL)
@pytest.mark.parametrize("ctx,budget,sink,recent,bs", EVICT)
def test_evict(fmt, ctx, budget, sink, recent, bs):
    hkv = 3
    r = np.random.default_rng(37)
    spare = -(-budget // bs)
    blocks, table, dst = lay_out(ctx, bs, 38, spare=spare)
    cache = random_cache(fmt, blocks, bs, hkv, 39)
    host = Host(cache)
    w = np.exp(2 * r.standard_normal((len(ctx), hkv, max(ctx) + 3))).astype(np.float32)
    w[:, 1] = np.round(w[:, 1])                    # many equal weights, zeros among them
    w[:, 2] = 0.25                                 # nothing but equal weights
    for b, c in enumerate(ctx):                    # destination entries behind the new length: not read
        dst[b, -(-min(c, budget) // bs):] = -1
    lens, wout, keep = pk.kv_evict(cache, cuda(w), cuda(table), cuda(np.int32(ctx)), cuda(dst), budget,
                                   num_sink=sink, num_recent=recent)
    rk, rw, rl = evict(host, w, table, ctx, dst, budget, sink, recent, wout.shape[2])
    assert np.array_equal(keep.cpu().numpy(), rk)
    assert np.array_equal(wout.cpu().numpy(), rw)
    assert np.array_equal(lens.cpu().numpy(), rl)
    for name, ref in (("k_cache", host.k), ("v_cache", host.v)):
        assert np.array_equal(getattr(cache, name).cpu().numpy(), ref), name
    if fmt in BLOCK:
        assert_same(cache, host)
    if fmt == pk.KV_INT8:
        assert np.array_equal(cache.k_scale_tok.cpu().numpy(), host.ks)
        assert np.array_equal(cache.v_scale_tok.cpu().numpy(), host.vs)
    assert pk.device_status() == 0


@pytest.mark.parametrize("n,stride,budget,sink,recent", [
    (40_000, 40_000, 5001, 4, 333),          # a whole cluster, odd slices
    (40_000, 70_000, 39_999, 0, 0),          # one token goes
    (20_001, 20_001, 17, 3, 5),
    (4097, 500_000, 100, 4, 4),              # a row much shorter than its stride
    (400_000, 400_001, 1000, 4, 64)])        # keys do not fit shared memory
def test_evict_long_rows(n, stride, budget, sink, recent):
    bs, hkv = 64, 2
    r = np.random.default_rng(48)
    blocks, table, dst = lay_out([n, n // 3], bs, 49, spare=-(-budget // bs))
    cache = pk.PagedKVCache.allocate(pk.KV_FP8_E4M3, blocks, bs, hkv, k_scale=[1.0] * hkv, v_scale=[1.0] * hkv)
    g = torch.Generator(device="cuda").manual_seed(50)
    for t in (cache.k_cache, cache.v_cache):
        t.random_(0, 127, generator=g)
    w = np.exp(2 * r.standard_normal((2, hkv, stride))).astype(np.float32)
    w[:, 1] = np.floor(w[:, 1])              # ties by the thousand
    ctx = np.int32([n, n // 3])
    kc, vc = cache.k_cache.clone(), cache.v_cache.clone()
    lens, wout, keep = pk.kv_evict(cache, cuda(w), cuda(table), cuda(ctx), cuda(dst), budget, sink, recent)
    keep, wout = keep.cpu().numpy(), wout.cpu().numpy()
    for b, c in enumerate(ctx):
        m = min(c, budget)
        assert int(lens[b]) == m
        for h in range(hkv):
            if c <= budget:
                pick = np.arange(c)
            else:
                mid = w[b, h, sink:c - recent]
                best = np.argsort(-mid, kind="stable")[:budget - sink - recent] + sink
                pick = np.concatenate([np.arange(sink), np.sort(best), np.arange(c - recent, c)])
            assert np.array_equal(keep[b, h, :m], pick) and (keep[b, h, m:] == -1).all()
            assert np.array_equal(wout[b, h, :m], w[b, h, pick]) and (wout[b, h, m:] == 0).all()
            src, to = table[b][pick // bs], dst[b][np.arange(m) // bs]
            for new, old in ((cache.k_cache, kc), (cache.v_cache, vc)):
                assert torch.equal(new[cuda(to).long(), h, cuda(np.arange(m) % bs)],
                                   old[cuda(src).long(), h, cuda(pick % bs)])


def test_evict_odd_weights():
    """Infinities, NaN, negative and signed zero weights have a fixed order."""
    fmt, bs, hkv, n, budget = pk.KV_FP8_E4M3, 16, 1, 64, 24
    w = np.zeros((1, 1, n), np.float32)
    w[0, 0, :] = np.tile(np.float32([np.nan, -0.0, 0.0, -1.0, 2.0 ** -149, np.inf, -np.inf, 3.0]), 8)
    for budget in range(1, n + 1):
        blocks, table, dst = lay_out([n], bs, 40, spare=-(-budget // bs))
        cache = random_cache(fmt, blocks, bs, hkv, 41)
        host = Host(cache)
        _, wout, keep = pk.kv_evict(cache, cuda(w), cuda(table), cuda(np.int32([n])), cuda(dst), budget)
        rk, rw, _ = evict(host, w, table, [n], dst, budget, 0, 0, n)
        assert np.array_equal(keep.cpu().numpy(), rk), budget
        assert np.array_equal(wout.cpu().numpy().view(np.uint32), rw.view(np.uint32)), budget


@pytest.mark.parametrize("fmt", [pk.KV_INT8_BLOCK, pk.KV_FP8_E4M3, pk.KV_INT8])
def test_a_run_of_steps_with_eviction(fmt):
    """Prompt write, steps with weights, eviction, steps on the smaller cache."""
    bs, hq, hkv, n0, steps, budget = 16, 8, 2, 150, 3, 60
    r = np.random.default_rng(42)
    total = n0 + 2 * steps
    blocks, table, dst = lay_out([total, total - 70], bs, 43, spare=-(-(budget + steps) // bs))
    cache = random_cache(fmt, blocks, bs, hkv, 44)
    dst_full, ctx = dst, np.int32([n0, n0 - 70])
    W = torch.zeros((2, hkv, total), device="cuda")

    def write(k, v, n, ctx, tab):
        if fmt in BLOCK:
            cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
            pk.kv_write_block_quant(cache, cuda(k), cuda(v), cuda(cu), cuda(tab), cuda(ctx), max(n))
        else:
            slots = [int(tab[b][p // bs]) * bs + p % bs for b in range(2) for p in range(ctx[b] - n[b], ctx[b])]
            pk.kv_write_quant(cache, cuda(k), cuda(v), cuda(np.int32(slots)))

    write(new_rows(r, ctx.sum(), hkv), new_rows(r, ctx.sum(), hkv), ctx.tolist(), ctx, table)
    tab = table
    for phase in range(2):
        for _ in range(steps):
            ctx = (ctx + 1).astype(np.int32)
            write(new_rows(r, 2, hkv), new_rows(r, 2, hkv), [1, 1], ctx, tab)
            host, W0 = Host(cache), W.double().cpu().numpy()
            q = queries(r, 2, 1, hq, D)
            out, lse = run_weights(cache, cuda(q), cuda(tab), cuda(ctx), W)
            o, l, w = out.double().cpu().numpy(), lse.double().cpu().numpy(), W.double().cpu().numpy()
            for b in range(2):
                n = int(ctx[b])
                check_rows(o[b], l[b], q[b].astype(float), host, tab, b, n, np.array([n - 1]), hq)
                for h in range(hkv):
                    ref = W0[b, h].copy()
                    for g in range(h * 4, h * 4 + 4):
                        ref[:n] += attention(q[b, :, g].astype(float), host.rows("k", tab[b], h, n),
                                             host.rows("v", tab[b], h, n), [n - 1], SCALE)[2][0]
                    assert np.linalg.norm(w[b, h] - ref) <= 2e-5 * np.linalg.norm(ref)
        if phase == 0:
            host, W0 = Host(cache), W.cpu().numpy()
            lens, W, keep = pk.kv_evict(cache, W, cuda(tab), cuda(ctx), cuda(dst_full), budget, 4, 20)
            rk, rw, rl = evict(host, W0, tab, ctx, dst_full, budget, 4, 20, W.shape[2])
            assert np.array_equal(keep.cpu().numpy(), rk) and np.array_equal(W.cpu().numpy(), rw)
            assert np.array_equal(cache.k_cache.cpu().numpy(), host.k)
            ctx, tab = rl.copy(), dst_full
    assert pk.device_status() == 0


def test_captured_weights_and_eviction_replay():
    """Two captured graphs share one workspace, one after the other."""
    fmt, bs, hq, hkv, ctx, budget = pk.KV_FP8_E4M3, 16, 8, 2, [900, 300], 128
    r = np.random.default_rng(45)
    blocks, table, dst = lay_out(ctx, bs, 46, spare=budget // bs)
    cache = random_cache(fmt, blocks, bs, hkv, 47)
    t, c, d = cuda(table), cuda(np.int32(ctx)), cuda(dst)
    qs = [cuda(queries(r, 2, 1, hq, D)) for _ in range(2)]
    ws = torch.empty(pk.decode_weights_workspace_bytes(cache, 2, 1, hq, 900), dtype=torch.uint8, device="cuda")

    def fresh():
        return [torch.zeros((2, hkv, 900), device="cuda") for _ in range(2)]

    def call(q, W, out, res):
        pk.paged_attn_decode_weights(cache, q, t, c, 900, SCALE, W, out=out, workspace=ws)
        pk.kv_evict(cache, W, t, c, d, budget, 4, 16, weights_out=res[0], keep=res[1], new_context_lens=res[2])

    def results():
        return [(torch.empty((2, hkv, 900), device="cuda"),
                 torch.empty((2, hkv, budget), dtype=torch.int32, device="cuda"), torch.empty_like(c)) for _ in range(2)]

    eager_w, eager_o, eager_r = fresh(), [torch.empty_like(q) for q in qs], results()
    for i in range(2):
        call(qs[i], eager_w[i], eager_o[i], eager_r[i])
    W, out, res = fresh(), [torch.empty_like(q) for q in qs], results()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call(qs[i], W[i], out[i], res[i])
        graphs.append(g)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(W[i], eager_w[i]) and torch.equal(out[i], eager_o[i])
        for a, b in zip(res[i], eager_r[i]):
            assert torch.equal(a, b)
