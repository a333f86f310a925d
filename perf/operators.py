"""Workloads of the block-scaled cache, the weight-driven eviction and the prompt attention.

Every case is one call a serving program makes.  ``run`` makes that call of
``paged_quantized_kv_quant_b200`` where ``own`` is true and computes the same
in elementary torch operations where it is false; ``exact`` computes it once
more, in 64 bits and sequence by sequence.

Kinds:
  write    quantise new tokens into a cache with one scale per (block, KV head)
  decode   attention of 1..16 new tokens per sequence over such a cache
  prefill  attention of a prompt chunk over such a cache
  weights  decode attention that also accumulates every key's softmax weight
  evict    keep the heaviest, first and most recent tokens, in new blocks
  prompt   causal attention over packed whole prompts, K and V as projected
"""
import math
import random

import torch

own = False

D = 128
FORMATS = ("e4m3", "int8", "fp16", "int8_block", "e4m3_block")
QMAX = {"int8": 127.0, "int8_block": 127.0, "e4m3": 448.0, "e4m3_block": 448.0}
SCALE = 1.0 / math.sqrt(D)


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # four prompts of different lengths land in an empty block-scaled cache
        dict(name="write_prompts", kind="write", fmt="e4m3_block", batch=4, len=8192, even=False,
             old=0, kv_heads=8, block_size=16),
        # one new token for each of 16 running sequences: blocks partly filled, some scales grow
        dict(name="write_step", kind="write", fmt="int8_block", batch=16, len=1, even=True,
             old=4000, kv_heads=8, block_size=32),
        # the smallest decode: one short sequence, latency alone
        dict(name="decode_1x1k", kind="decode", fmt="int8_block", batch=1, len=1024, even=True,
             q_len=1, q_heads=8, kv_heads=2, block_size=16),
        # an ordinary serving step: 8 sequences of 32K tokens
        dict(name="decode_8x32k", kind="decode", fmt="e4m3_block", batch=8, len=32768, even=True,
             q_len=1, q_heads=32, kv_heads=4, block_size=16),
        # draft verification (1 + 4 positions) over long contexts of different lengths
        dict(name="verify_4x64k", kind="decode", fmt="int8_block", batch=4, len=65536, even=False,
             q_len=5, q_heads=32, kv_heads=4, block_size=32),
        # a chunk of a long prompt over its cached prefix
        dict(name="prefill_2k_over_30k", kind="prefill", fmt="e4m3_block", batch=1, len=32768,
             even=True, q_len=2048, q_heads=32, kv_heads=4, block_size=64),
        # short sequences of odd lengths whose weights are tracked: latency
        dict(name="weights_3x700", kind="weights", fmt="int8", batch=3, len=701, even=False,
             q_len=1, q_heads=8, kv_heads=2, block_size=16),
        # an ordinary step with tracked weights
        dict(name="weights_8x16k", kind="weights", fmt="e4m3", batch=8, len=16384, even=True,
             q_len=1, q_heads=32, kv_heads=4, block_size=16),
        # sequences of odd lengths cut to an odd budget; codes move between block scales
        dict(name="evict_5x3k", kind="evict", fmt="int8_block", batch=5, len=2999, even=False,
             budget=501, sink=4, recent=65, kv_heads=2, block_size=16),
        # a full batch cut to an eighth
        dict(name="evict_8x32k", kind="evict", fmt="e4m3", batch=8, len=32768, even=True,
             budget=4096, sink=4, recent=512, kv_heads=4, block_size=16),
        # packed prompts of odd lengths
        dict(name="prompt_7x2k", kind="prompt", dtype="bf16", batch=7, len=2047, even=False,
             q_heads=32, kv_heads=8, window=0),
        # one long prompt
        dict(name="prompt_8k", kind="prompt", dtype="fp16", batch=1, len=8192, even=True,
             q_heads=32, kv_heads=4, window=0),
    ]


def _span(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(("write", "decode", "prefill", "weights", "evict", "prompt"))
    heads = rng.choice(((8, 2), (32, 4), (32, 8), (16, 16), (40, 8), (6, 1), (14, 2), (16, 1)))
    block = rng.choice(("int8_block", "e4m3_block"))
    c = dict(kind=kind, kv_heads=heads[1], even=rng.random() < 0.25)
    if kind != "prompt":
        c["block_size"] = rng.choice((16, 32, 64))
    if kind == "write":
        c.update(fmt=block, batch=_span(rng, 1, 32), len=_span(rng, 1, 8192),
                 old=rng.choice((0, _span(rng, 1, 4096))))
        c["len"] = max(1, min(c["len"], 131072 // (c["batch"] * heads[1])))
    elif kind in ("decode", "weights"):
        c.update(fmt=block if kind == "decode" else rng.choice(FORMATS), batch=_span(rng, 1, 32),
                 len=_span(rng, 1, 65536), q_len=rng.choice((1, 1, 1, 2, 5, rng.randint(1, 16))),
                 q_heads=heads[0])
        most = 1_000_000 if kind == "decode" else 400_000   # (token, KV head) pairs
        c["len"] = max(1, min(c["len"], most // (c["batch"] * heads[1] * (1 + c["q_len"] // 4))))
    elif kind == "prefill":
        c.update(fmt=block, batch=_span(rng, 1, 4), q_len=_span(rng, 1, 2048), q_heads=heads[0])
        c["len"] = c["q_len"] + _span(rng, 1, 16384) - 1
        c["len"] = max(c["q_len"], c["len"] // c["batch"])
    elif kind == "evict":
        c.update(fmt=rng.choice(FORMATS), batch=_span(rng, 1, 16), len=_span(rng, 16, 65536))
        c["len"] = max(16, min(c["len"], 500_000 // (c["batch"] * heads[1])))
        c["budget"] = _span(rng, 4, c["len"])
        c["sink"] = rng.randint(0, min(4, c["budget"] // 4))
        c["recent"] = rng.randint(0, c["budget"] // 2)
    else:
        c.update(dtype=rng.choice(("fp16", "bf16")), batch=_span(rng, 1, 16),
                 len=_span(rng, 1, 8192), q_heads=heads[0],
                 window=rng.choice((0, 0, 0, _span(rng, 1, 4096))))
        c["len"] = max(1, min(c["len"], int(8192 * math.sqrt(32 / (heads[0] * c["batch"])) / 1.3)))
    return c


def _lens(case):
    """Tokens of each sequence: all of `len`, or the first that long and the others shorter."""
    b, n = case["batch"], case["len"]
    if case["even"]:
        return [n] * b
    r = random.Random(1000003 * n + b)
    return [n] + [max(1, int(n * r.uniform(0.05, 1.0))) for _ in range(b - 1)]


def _old_lens(case):
    """write: tokens that each sequence already has."""
    r = random.Random(7919 * case["old"] + case["batch"])
    return [int(case["old"] * r.uniform(0.0, 1.0)) for _ in range(case["batch"])]


def _chunks(case):
    """prefill: query tokens of each sequence, the last ones of its context."""
    return [min(case["q_len"], n) for n in _lens(case)]


def work(case):
    kind, lens, hkv = case["kind"], _lens(case), case["kv_heads"]
    if kind == "prompt":
        w = case["window"]
        pairs = sum(n * (n + 1) // 2 if not w or w >= n else w * (w + 1) // 2 + (n - w) * w for n in lens)
        return {"bytes": sum(lens) * D * 2 * (2 * case["q_heads"] + 2 * hkv) + sum(lens) * case["q_heads"] * 4,
                "flops": 4 * D * case["q_heads"] * pairs}
    fmt, bs = case["fmt"], case["block_size"]
    row = 2 * hkv * (D * (2 if fmt == "fp16" else 1) + (2 if fmt == "int8" else 0))   # K and V of a token
    blk = 2 * hkv * 4 if fmt.endswith("_block") else 0                                # scales of a block
    if kind == "write":
        new = sum(lens)
        touched = sum((o + n - 1) // bs - o // bs + 1 for o, n in zip(_old_lens(case), lens))
        return {"bytes": new * (2 * hkv * D * 2 + row) + touched * blk, "flops": 0}
    cache = sum(lens) * row + sum(-(-n // bs) for n in lens) * (blk + 4)
    if kind == "evict":
        kept = sum(min(n, case["budget"]) for n in lens)
        return {"bytes": sum(lens) * hkv * 4 + 2 * kept * row + kept * hkv * (4 + 4)
                + case["batch"] * hkv * case["len"] * 4, "flops": 0}
    q = _chunks(case) if kind == "prefill" else [case["q_len"]] * case["batch"]
    pairs = sum(sum(max(0, n - m + t + 1) for t in range(m)) for n, m in zip(lens, q))
    return {"bytes": cache + sum(q) * case["q_heads"] * (2 * D * 2 + 4)
            + (sum(lens) * hkv * 8 if kind == "weights" else 0),
            "flops": 4 * D * case["q_heads"] * pairs}


# ----------------------------------------------------------------- inputs --

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _quantised(g, fmt, shape):
    """Codes (bytes) and scales of random rows [blocks][heads][block size][D] whose size differs from
    block to block, as K and V of different tokens do."""
    x = torch.randn(shape, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(shape[:2] + (1, 1), generator=g, device="cuda"))
    if fmt == "fp16":
        return x.half().view(torch.uint8), None
    if fmt == "int8":
        s = (x.abs().amax(-1) / 127.0).half()
        return (x / s[..., None].float()).round().clamp(-127, 127).to(torch.int8).view(torch.uint8), s
    over = (0, 2, 3) if fmt == "e4m3" else (2, 3)
    s = x.abs().amax(over) / QMAX[fmt]
    y = x.div_(s[:, None, None] if fmt == "e4m3" else s[..., None, None])
    if fmt == "int8_block":
        return y.round_().clamp_(-127, 127).to(torch.int8).view(torch.uint8), s
    return y.clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), s


def _make_cache(st, g, case, tokens, spare=0):
    """A pool that holds `tokens` tokens of each sequence in scattered blocks, and `spare` more blocks each."""
    bs, hkv = case["block_size"], case["kv_heads"]
    n = [-(-t // bs) for t in tokens]
    total = sum(n) + spare * len(n)
    st["blocks"] = blocks = total + total // 8 + 1
    perm = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    wide = max(n)
    take = torch.arange(wide, device="cuda")[None] < _i32(n)[:, None]
    st["table"] = torch.zeros((len(n), wide), dtype=torch.int32, device="cuda")
    st["table"][take] = perm[:sum(n)]
    if spare:
        st["dst"] = perm[sum(n):total].view(len(n), spare).contiguous()
    for x in "kv":
        st[x + "c"], st[x + "s"] = _quantised(g, case["fmt"], (blocks, hkv, bs, D))


def _handle(st, case):
    """The framework's cache object over the same memory."""
    import paged_quantized_kv_quant_b200 as pk
    kinds = dict(e4m3=pk.KV_FP8_E4M3, int8=pk.KV_INT8, fp16=pk.KV_FP16)
    fmt = case["fmt"]
    if fmt == "fp16":
        return pk.PagedKVCache(kinds[fmt], st["kc"], st["vc"])
    if fmt == "e4m3":
        return pk.PagedKVCache(kinds[fmt], st["kc"], st["vc"], k_scale=st["ks"], v_scale=st["vs"])
    if fmt == "int8":
        return pk.PagedKVCache(kinds[fmt], st["kc"], st["vc"], k_scale_tok=st["ks"], v_scale_tok=st["vs"])
    return pk.PagedKVCache(pk.KV_INT8_BLOCK if fmt == "int8_block" else pk.KV_E4M3_BLOCK, st["kc"], st["vc"],
                           k_scale_blk=st["ks"], v_scale_blk=st["vs"])


def prepare(case, seed):
    g, kind, lens = _gen(seed), case["kind"], _lens(case)
    hkv = case["kv_heads"]
    st = dict(case=case, lens=lens)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if kind == "prompt":
        dt = torch.float16 if case["dtype"] == "fp16" else torch.bfloat16
        t = sum(lens)
        st.update(q=(1.5 * randn(t, case["q_heads"], D)).to(dt), k=randn(t, hkv, D).to(dt), v=randn(t, hkv, D).to(dt),
                  cu=_i32([sum(lens[:i]) for i in range(len(lens) + 1)]))
        if own:
            st.update(out=torch.empty_like(st["q"]), lse=torch.empty((t, case["q_heads"]), device="cuda"))
        return st
    if kind == "write":
        old = _old_lens(case)
        ctx = [o + n for o, n in zip(old, lens)]
        _make_cache(st, g, case, ctx)
        t = sum(lens)
        loud = torch.exp(0.5 * randn(t, hkv, 1))
        st.update(k=(randn(t, hkv, D) * loud).half(), v=(randn(t, hkv, D) * loud).half(), ctx=_i32(ctx),
                  cu=_i32([sum(lens[:i]) for i in range(len(lens) + 1)]))
        if own:
            st["cache"] = _handle(st, case)
        return st
    _make_cache(st, g, case, lens, -(-case["budget"] // case["block_size"]) if kind == "evict" else 0)
    st["ctx"] = _i32(lens)
    if kind == "evict":
        # weights that many steps left behind: a few heavy tokens, many light ones, some never seen
        w = torch.exp(2.0 * randn(len(lens), hkv, max(lens)))
        st["weights"] = torch.where(torch.rand(w.shape, generator=g, device="cuda") < 0.1, 0.0, w)
        if own:
            st.update(cache=_handle(st, case), weights_out=torch.empty_like(w), new_lens=torch.empty_like(st["ctx"]),
                      keep=torch.empty((len(lens), hkv, case["budget"]), dtype=torch.int32, device="cuda"))
        return st
    if kind == "prefill":
        q = _chunks(case)
        st.update(cu=_i32([sum(q[:i]) for i in range(len(q) + 1)]), chunks=q,
                  q=(1.5 * randn(sum(q), case["q_heads"], D)).half())
    else:
        st["q"] = (1.5 * randn(len(lens), case["q_len"], case["q_heads"], D)).half()
        if kind == "weights":
            st["weights"] = torch.rand((len(lens), hkv, max(lens)), generator=g, device="cuda")
    if own:
        import paged_quantized_kv_quant_b200 as pk
        st.update(cache=_handle(st, case), out=torch.empty_like(st["q"]),
                  lse=torch.empty(st["q"].shape[:-1], device="cuda"))
        if kind != "prefill":
            size = pk.decode_weights_workspace_bytes if kind == "weights" else pk.decode_workspace_bytes
            st["workspace"] = torch.empty(size(st["cache"], len(lens), case["q_len"], case["q_heads"], max(lens)),
                                          dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------- the calls --

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _held(st, fmt):
    """The cache's memory as the numbers it holds, and its scales."""
    kind = torch.int8 if fmt.startswith("int8") else torch.float16 if fmt == "fp16" else torch.float8_e4m3fn
    out = {"k": st["kc"].view(kind), "v": st["vc"].view(kind)}
    if fmt in ("int8", "int8_block", "e4m3_block"):
        out.update(k_scale=st["ks"], v_scale=st["vs"])
    return out


def _run_own(st):
    import paged_quantized_kv_quant_b200 as pk
    case, kind = st["case"], st["case"]["kind"]
    if kind == "prompt":
        pk.prompt_attn(st["q"], st["k"], st["v"], st["cu"], max(st["lens"]), SCALE, out=st["out"], lse=st["lse"],
                       sliding_window=case["window"])
    elif kind == "write":
        pk.kv_write_block_quant(st["cache"], st["k"], st["v"], st["cu"], st["table"], st["ctx"], max(st["lens"]))
        return _held(st, case["fmt"])
    elif kind == "decode":
        pk.paged_attn_decode(st["cache"], st["q"], st["table"], st["ctx"], max(st["lens"]), SCALE, out=st["out"],
                             lse=st["lse"], workspace=st["workspace"])
    elif kind == "prefill":
        pk.paged_attn_prefill(st["cache"], st["q"], st["cu"], st["table"], st["ctx"], max(st["chunks"]), SCALE,
                              out=st["out"], lse=st["lse"])
    elif kind == "weights":
        pk.paged_attn_decode_weights(st["cache"], st["q"], st["table"], st["ctx"], max(st["lens"]), SCALE,
                                     st["weights"], out=st["out"], lse=st["lse"], workspace=st["workspace"])
        return {"out": st["out"], "lse": st["lse"], "weights": st["weights"]}
    else:
        pk.kv_evict(st["cache"], st["weights"], st["table"], st["ctx"], st["dst"], case["budget"],
                    num_sink=case["sink"], num_recent=case["recent"], weights_out=st["weights_out"],
                    keep=st["keep"], new_context_lens=st["new_lens"])
        return {**_held(st, case["fmt"]), "weights": st["weights_out"], "keep": st["keep"], "lens": st["new_lens"]}
    return {"out": st["out"], "lse": st["lse"]}


# ------------------------------------------------------------ plain forms --

def _run_plain(st):
    kind = st["case"]["kind"]
    if kind == "write":
        return _plain_write(st)
    if kind == "evict":
        return _plain_evict(st)
    return _plain_attention(st)


def _numbers(codes, fmt):
    """Bytes -> the fp32 numbers they stand for, before any scale."""
    kind = torch.int8 if fmt.startswith("int8") else torch.float16 if fmt == "fp16" else torch.float8_e4m3fn
    return codes.view(kind).float()


def _codes(x, fmt):
    """fp32 quotients -> bytes, to nearest even."""
    if fmt.startswith("int8"):
        return x.round().clamp(-127, 127).to(torch.int8).view(torch.uint8)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _keys(st, x):
    """All of a cache's K (x "k") or V as fp32 [B][heads][tokens][D], in each sequence's order."""
    fmt = st["case"]["fmt"]
    at = st["table"].long()
    y = _numbers(st[x + "c"][at], fmt)                       # [B][blocks][heads][bs][D]
    s = st[x + "s"]
    if fmt == "e4m3":
        y *= s[:, None, None]
    elif fmt == "int8":
        y *= s[at].float()[..., None]
    elif s is not None:
        y *= s[at][..., None, None]
    return y.permute(0, 2, 1, 3, 4).reshape(y.shape[0], y.shape[2], -1, D)


def _padded(st, x):
    """Packed rows [T][heads][D] as fp32 [B][longest][heads][D]; row i of sequence b at [b][i]."""
    n = st["cu"][1:] - st["cu"][:-1]
    i = torch.arange(max(st["chunks"] if "chunks" in st else st["lens"]), device="cuda")
    at = (st["cu"][:-1, None] + torch.minimum(i, n[:, None] - 1)).long()
    return x[at].float(), at, n


def _plain_attention(st):
    case, kind = st["case"], st["case"]["kind"]
    hkv = case["kv_heads"]
    at = None
    if kind == "prompt":
        q, at, n = _padded(st, st["q"])
        k, v = (_padded(st, st[x])[0].transpose(1, 2) for x in "kv")
        ctx, first = n, torch.zeros_like(n)
    else:
        k, v, ctx = _keys(st, "k"), _keys(st, "v"), st["ctx"]
        if kind == "prefill":
            q, at, n = _padded(st, st["q"])
        else:
            q, n = st["q"].float(), case["q_len"]
        first = ctx - n                                      # position of each sequence's first query
    B, Q, Hq = q.shape[:3]
    j = torch.arange(k.shape[2], device="cuda")
    pos = first[:, None] + torch.arange(Q, device="cuda")
    seen = (j <= pos[..., None]) & (j < ctx[:, None, None])
    if case.get("window"):
        seen &= j > pos[..., None] - case["window"]
    q = q.view(B, Q, hkv, Hq // hkv, D).permute(0, 2, 3, 1, 4).reshape(B, hkv, -1, D)
    s = (q @ k.transpose(2, 3)).mul_(SCALE).view(B, hkv, Hq // hkv, Q, -1)
    s.masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True).clamp_min(-1e30)
    p = s.sub_(m).exp_()
    sums = p.sum(-1, keepdim=True)
    lse = torch.where(sums > 0, m + sums.log(), -math.inf)[..., 0].permute(0, 3, 1, 2).reshape(B, Q, Hq)
    p /= torch.where(sums > 0, sums, 1.0)
    o = (p.view(B, hkv, -1, p.shape[-1]) @ v).view(B, hkv, Hq // hkv, Q, D)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, Q, Hq, D)
    if at is not None:                                       # packed again
        out = torch.empty_like(st["q"])
        out[at] = o.to(out.dtype)
        packed = torch.empty(out.shape[:2], device="cuda")
        packed[at] = lse
        # the rows behind a sequence's end wrote its last row: set it from that row itself
        b = torch.arange(B, device="cuda")
        out[at[:, -1]] = o[b, (n - 1).long()].to(out.dtype)
        packed[at[:, -1]] = lse[b, (n - 1).long()]
        return {"out": out, "lse": packed}
    out = {"out": o.half(), "lse": lse}
    if kind == "weights":
        st["weights"] += p.sum((2, 3))[..., :st["weights"].shape[2]]
        out["weights"] = st["weights"]
    return out


def _plain_write(st):
    case = st["case"]
    bs, fmt = case["block_size"], case["fmt"]
    n = st["cu"][1:] - st["cu"][:-1]
    start = st["ctx"] - n
    i = torch.arange((max(st["lens"]) + bs - 2) // bs + 1, device="cuda")
    # blocks that a sequence's new tokens touch (its last one again where it has fewer)
    blk = torch.minimum(start[:, None] // bs + i, (st["ctx"][:, None] - 1) // bs)
    at = st["table"].gather(1, blk.long()).long()
    pos = blk[..., None] * bs + torch.arange(bs, device="cuda")
    older = pos < start[:, None, None]
    new = ~older & (pos < st["ctx"][:, None, None])
    src = (st["cu"][:-1, None, None] + pos - start[:, None, None]).clamp(0, st["k"].shape[0] - 1).long()
    has = older.any(-1)[..., None]
    for x in "kv":
        y = st[x][src].float().nan_to_num(0.0, 65504.0, -65504.0) * new[..., None, None]
        y = y.permute(0, 1, 3, 2, 4)                         # [B][blocks][heads][bs][D]
        codes, scales = st[x + "c"], st[x + "s"]
        s_old = scales[at]
        top = y.abs().amax((3, 4))
        s = top / torch.full_like(top, QMAX[fmt])            # by a tensor: by a number it would be a product
        s = torch.where(has, torch.maximum(s, s_old), s)
        now = codes[at]
        ratio = torch.where(s > 0, s_old / s, 0.0)[..., None, None]
        again = torch.where((s > s_old)[..., None, None], _codes(_numbers(now, fmt) * ratio, fmt), now)
        put = _codes(torch.where(s > 0, 1.0, 0.0)[..., None, None] * y / torch.where(s > 0, s, 1.0)[..., None, None], fmt)
        rows = lambda m: m[:, :, None, :, None]  # noqa: E731
        codes[at] = torch.where(rows(new), put, torch.where(rows(older), again, now))
        scales[at] = s
    return _held(st, fmt)


def _plain_evict(st):
    case = st["case"]
    bs, fmt, budget = case["block_size"], case["fmt"], case["budget"]
    w, n = st["weights"], st["ctx"][:, None, None]
    j = torch.arange(w.shape[2], device="cuda")
    stays = (j < case["sink"]) | (j >= n - case["recent"]) | (n <= budget)
    key = torch.where(j < n, torch.where(stays, math.inf, w), -math.inf)
    best = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :budget]
    r = torch.arange(budget, device="cuda")
    lens = torch.minimum(st["ctx"], torch.full_like(st["ctx"], budget))
    live = (r < lens[:, None, None]).expand(-1, w.shape[1], -1)
    best = torch.nn.functional.pad(best, (0, budget - best.shape[2]))
    keep = torch.where(live, best, w.shape[2]).sort(-1).values
    heavy = torch.where(live, w.gather(2, keep.clamp_max(w.shape[2] - 1)), 0.0)
    kept = torch.zeros_like(w)
    kept[..., :min(budget, w.shape[2])] = heavy[..., :w.shape[2]]
    # rows of the new blocks, and where each comes from
    nb = st["dst"].shape[1]
    pad = nb * bs - budget
    live = torch.nn.functional.pad(live, (0, pad))
    src = torch.nn.functional.pad(torch.where(live[..., :budget], keep, 0), (0, pad))
    b = torch.arange(w.shape[0], device="cuda")[:, None, None]
    h = torch.arange(w.shape[1], device="cuda")[None, :, None]
    at = st["table"][b, src // bs].long()
    to = st["dst"].long()
    live = live.view(live.shape[0], live.shape[1], nb, bs)

    def blocks(y):                                           # [B][heads][rows]... -> [B][nb][heads][bs]...
        return y.view(y.shape[:2] + (nb, bs) + y.shape[3:]).transpose(1, 2)

    alive = live.transpose(1, 2)
    for x in "kv":
        codes, scales = st[x + "c"], st[x + "s"]
        rows = blocks(codes[at, h, src % bs])
        if fmt.endswith("_block"):
            s = blocks(scales[at, h]) * alive
            top = s.amax(-1)
            ratio = torch.where(top[..., None] > 0, s / torch.where(top > 0, top, 1.0)[..., None], 0.0)
            rows = torch.where((s < top[..., None])[..., None], _codes(_numbers(rows, fmt) * ratio[..., None], fmt), rows)
            scales[to] = torch.where(alive.any(-1), top, scales[to])
        elif fmt == "int8":
            scales[to] = torch.where(alive, blocks(scales[at, h, src % bs]), scales[to])
        codes[to] = torch.where(alive[..., None], rows, codes[to])
    keep = torch.where(r < lens[:, None, None], keep, -1).to(torch.int32)
    return {**_held(st, fmt), "weights": kept, "keep": keep, "lens": lens}


# ---------------------------------------------------------- in 64 bits --

def _f32(x):
    """The nearest fp32 number, kept in 64 bits."""
    return x.to(torch.float32).to(torch.float64)


def _round_to_codes(x, fmt):
    if fmt.startswith("int8"):
        return torch.clamp(torch.round(x), -127, 127)
    # e4m3: 3 mantissa bits, the smallest exponent -6, largest value 448
    e = torch.clamp(torch.floor(torch.log2(torch.clamp(x.abs(), min=2.0 ** -20))), min=-6.0)
    step = torch.exp2(e - 3)
    return torch.clamp(torch.round(x / step) * step, -448, 448)


def _as_bytes(x, fmt):
    return (x.to(torch.int8) if fmt.startswith("int8") else x.to(torch.float32).to(torch.float8_e4m3fn)).view(torch.uint8)


def exact(case, seed):
    """What run() returns, sequence by sequence in 64 bits."""
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["kind"] == "write":
        return _exact_write(st, case)
    if case["kind"] == "evict":
        return _exact_evict(st, case)
    return _exact_attention(st, case)


def _exact_attention(st, case):
    kind, hkv = case["kind"], case["kv_heads"]
    group = case["q_heads"] // hkv
    window = case.get("window") or 1 << 40
    rows, lses = [], []
    weights = st["weights"].double() if kind == "weights" else None
    for b, n in enumerate(st["lens"]):
        if kind == "prompt":
            lo = int(st["cu"][b])
            q = st["q"][lo:lo + n].double()
            k, v = st["k"][lo:lo + n].double(), st["v"][lo:lo + n].double()
        else:
            q = st["q"][int(st["cu"][b]):int(st["cu"][b + 1])].double() if kind == "prefill" else st["q"][b].double()
            k = v = None
        out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
        lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
        place = torch.arange(n - q.shape[0], n, device="cuda")
        j = torch.arange(n, device="cuda")
        hidden = (j[None] > place[:, None]) | (j[None] <= place[:, None] - window)
        some = ~hidden.all(1)
        for h in range(hkv):
            kh = k[:, h] if k is not None else _exact_rows(st, case, "k", b, h, n)
            vh = v[:, h] if v is not None else _exact_rows(st, case, "v", b, h, n)
            for g in range(h * group, (h + 1) * group):
                s = (q[:, g] @ kh.T) / math.sqrt(D)
                s[hidden] = -math.inf
                z = torch.logsumexp(s, 1)
                p = torch.exp(s[some] - z[some, None])
                out[some, g], lse[some, g] = p @ vh, z[some]
                if weights is not None:
                    weights[b, h, :n] += p.sum(0)
        rows.append(out)
        lses.append(lse)
    if kind in ("decode", "weights"):
        res = {"out": torch.stack(rows), "lse": torch.stack(lses)}
        return {**res, "weights": weights} if weights is not None else res
    return {"out": torch.cat(rows), "lse": torch.cat(lses)}


def _exact_numbers(codes, fmt):
    kind = {"fp16": torch.float16, "int8": torch.int8, "int8_block": torch.int8}.get(fmt, torch.float8_e4m3fn)
    return codes.contiguous().view(kind).double()


def _exact_rows(st, case, x, b, h, n):
    """The first n tokens of sequence b, head h."""
    bs, fmt = case["block_size"], case["fmt"]
    at = st["table"][b, :-(-n // bs)].long()
    y = _exact_numbers(st[x + "c"][at, h], fmt)
    s = st[x + "s"]
    if fmt == "e4m3":
        y = y * s[h].double()
    elif fmt == "int8":
        y = y * s[at, h].double()[..., None]
    elif s is not None:
        y = y * s[at, h].double()[..., None, None]
    return y.reshape(-1, D)[:n]


def _exact_write(st, case):
    bs, fmt = case["block_size"], case["fmt"]
    for b, n in enumerate(st["lens"]):
        ctx, lo = int(st["ctx"][b]), int(st["cu"][b])
        start = ctx - n
        first, last = start // bs, (ctx - 1) // bs
        at = st["table"][b, first:last + 1].long()
        head = start - first * bs                            # older tokens in the first block
        tail = (last + 1) * bs - ctx                         # rows behind the context in the last
        for x in "kv":
            new = st[x][lo:lo + n].double().transpose(0, 1)  # [heads][n][D]
            y = torch.nn.functional.pad(new, (0, 0, head, tail)).view(new.shape[0], -1, bs, D).transpose(0, 1)
            s = y.abs().amax((2, 3))
            s = _f32(s / torch.full_like(s, QMAX[fmt]))
            s_old = st[x + "s"][at].double()
            if head:
                s[0] = torch.maximum(s[0], s_old[0])
            codes = _exact_numbers(st[x + "c"][at], fmt)
            res = _round_to_codes(_f32(y / torch.where(s > 0, s, torch.ones_like(s))[..., None, None]), fmt)
            if head:
                again = _round_to_codes(_f32(codes[0] * _f32(s_old[0] / s[0])[:, None, None]), fmt)
                res[0, :, :head] = torch.where((s[0] > s_old[0])[:, None, None], again, codes[0])[:, :head]
            if tail:
                res[-1, :, bs - tail:] = codes[-1, :, bs - tail:]
            st[x + "c"][at] = _as_bytes(res, fmt)
            st[x + "s"][at] = s.float()
    return _held(st, fmt)


def _exact_evict(st, case):
    bs, fmt, budget = case["block_size"], case["fmt"], case["budget"]
    B, H, S = st["weights"].shape
    kept = torch.zeros((B, H, S), dtype=torch.float64, device="cuda")
    keep = torch.full((B, H, budget), -1, dtype=torch.int32, device="cuda")
    for b, n in enumerate(st["lens"]):
        m = min(n, budget)
        for h in range(H):
            w = st["weights"][b, h, :n].double()
            if n <= budget:
                pick = torch.arange(n, device="cuda")
            else:
                lo, hi = case["sink"], n - case["recent"]
                mid = torch.sort(w[lo:hi], descending=True, stable=True).indices[:budget - lo - case["recent"]] + lo
                pick = torch.cat([torch.arange(lo, device="cuda"), torch.sort(mid).values, torch.arange(hi, n, device="cuda")])
            keep[b, h, :m] = pick.to(torch.int32)
            kept[b, h, :m] = w[pick]
            src, row = st["table"][b, pick // bs].long(), pick % bs
            to = st["dst"][b, torch.arange(m, device="cuda") // bs].long()
            put = torch.arange(m, device="cuda") % bs
            for x in "kv":
                vals = st[x + "c"][src, h, row]
                s = st[x + "s"]
                if fmt.endswith("_block"):
                    own_s = s[src, h].double()
                    top = torch.zeros(st["blocks"], dtype=torch.float64, device="cuda")
                    top = top.scatter_reduce(0, to, own_s, "amax")
                    mine = top[to]
                    moved = _round_to_codes(_f32(_exact_numbers(vals, fmt) * _f32(own_s / torch.where(mine > 0, mine, 1.0))[:, None]), fmt)
                    vals = torch.where((own_s < mine)[:, None], _as_bytes(moved, fmt), vals)
                    s[to, h] = mine.float()
                elif fmt == "int8":
                    s[to, h, put] = s[src, h, row]
                st[x + "c"][to, h, put] = vals
    lens = torch.tensor([min(n, budget) for n in st["lens"]], dtype=torch.int32, device="cuda")
    return {**_held(st, fmt), "weights": kept, "keep": keep, "lens": lens}
