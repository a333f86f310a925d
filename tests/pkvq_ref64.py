"""Plain 64-bit references (numpy, CPU) of the block-scaled cache, the weight
accumulation, the eviction and the prompt attention, and small seeded cases.
They share no code with the kernels."""
from __future__ import annotations

import numpy as np
import torch

import paged_quantized_kv_quant_b200 as pk

D = 128
QMAX = {pk.KV_INT8_BLOCK: 127.0, pk.KV_E4M3_BLOCK: 448.0}
BLOCK = (pk.KV_INT8_BLOCK, pk.KV_E4M3_BLOCK)
ALL = (pk.KV_FP8_E4M3, pk.KV_INT8, pk.KV_FP8_E5M2, pk.KV_FP16) + BLOCK


def f32(x):
    return np.asarray(x, np.float64).astype(np.float32).astype(np.float64)


# E4M3 values of the 256 codes from the format's definition (bias 7)
_c = np.arange(256)
_e, _m = (_c >> 3) & 15, _c & 7
E4M3 = np.where(_e == 0, _m * 2.0 ** -9, (8 + _m) * 2.0 ** (_e.astype(float) - 10))
E4M3 = np.where((_c & 127) == 127, np.nan, E4M3) * np.where(_c & 128, -1, 1)
_pos = E4M3[:127]                                    # 0 .. 448, ascending


def e4m3_encode(x):
    """Nearest code, ties to the even code, clamped to +-448; the sign is kept."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(_pos, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _pos[lo], _pos[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def encode(fmt, x):
    if fmt == pk.KV_INT8_BLOCK:
        return np.clip(np.rint(x), -127, 127).astype(np.int8).view(np.uint8)
    return e4m3_encode(x)


def numbers(fmt, codes):
    """Stored bytes [..., 128 * elem bytes] -> the numbers they hold, unscaled."""
    if fmt == pk.KV_FP16:
        return codes.view(np.float16).astype(np.float64)
    if fmt in (pk.KV_INT8, pk.KV_INT8_BLOCK):
        return codes.view(np.int8).astype(np.float64)
    if fmt == pk.KV_FP8_E5M2:
        return (codes.astype(np.uint16) << 8).view(np.float16).astype(np.float64)
    return E4M3[codes]


class Host:
    """Host copy of a cache's memory."""

    def __init__(self, cache):
        self.fmt, self.bs, self.hkv = cache.dtype, cache.block_size, cache.num_kv_heads
        self.k, self.v = cache.k_cache.cpu().numpy().copy(), cache.v_cache.cpu().numpy().copy()
        self.ks = self.vs = None
        src = {pk.KV_INT8: ("k_scale_tok", "v_scale_tok"), pk.KV_FP8_E4M3: ("k_scale", "v_scale"),
               pk.KV_FP8_E5M2: ("k_scale", "v_scale")}.get(self.fmt)
        if self.fmt in BLOCK:
            src = ("k_scale_blk", "v_scale_blk")
        if src:
            self.ks, self.vs = (getattr(cache, n).cpu().numpy().copy() for n in src)

    def rows(self, which, table, h, n):
        """The first n tokens' values of KV head h along one table row, float64 [n][128]."""
        c, s = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        nb = -(-n // self.bs)
        at = np.asarray(table)[:nb]
        y = numbers(self.fmt, c[at, h])
        if self.fmt in (pk.KV_FP8_E4M3, pk.KV_FP8_E5M2):
            y = y * float(s[h if s.size > 1 else 0])
        elif self.fmt == pk.KV_INT8:
            y = y * s[at, h].astype(np.float64)[..., None]
        elif s is not None:
            y = y * s[at, h].astype(np.float64)[:, None, None]
        return y.reshape(-1, D)[:n]


def write_block(host, k, v, cu, table, ctx):
    """The block write on a Host copy, block by block; k, v fp16 numpy [T][H][128]."""
    bs, fmt = host.bs, host.fmt
    for b in range(len(ctx)):
        n, c = int(cu[b + 1] - cu[b]), int(ctx[b])
        start = c - n
        lo = max(start, 0)
        if n <= 0:
            continue
        for i in range(lo // bs, -(-c // bs)):
            phys = int(table[b][i])
            p0, p1 = max(lo, i * bs), min(c, (i + 1) * bs)
            old = p0 - i * bs if i * bs < lo else 0
            for x, codes, scales in ((k, host.k, host.ks), (v, host.v, host.vs)):
                new = x[int(cu[b]) + p0 - start:int(cu[b]) + p1 - start].astype(np.float64)
                new = np.nan_to_num(new, nan=0.0, posinf=65504.0, neginf=-65504.0)
                for h in range(host.hkv):
                    s = f32(np.abs(new[:, h]).max() / QMAX[fmt])
                    s_old = float(scales[phys, h])
                    if old and s_old >= s:
                        s = s_old
                    elif old:
                        vals = numbers(fmt, codes[phys, h, :old])
                        codes[phys, h, :old] = encode(fmt, f32(vals * f32(s_old / s)))
                    q = f32(new[:, h] / s) if s > 0 else np.zeros_like(new[:, h])
                    codes[phys, h, p0 - i * bs:p1 - i * bs] = encode(fmt, q)
                    scales[phys, h] = s


def attention(q, keys, vals, pos, scale, window=0):
    """q [R][128], pos [R] (last visible key of each row) -> out, lse, weights
    [R][n], A = sum_j P_j |v_j| and the largest sum_d |q_d k_jd| * scale."""
    n = keys.shape[0]
    s = (q @ keys.T) * scale
    j = np.arange(n)
    seen = j[None] <= np.asarray(pos)[:, None]
    if window:
        seen &= j[None] > np.asarray(pos)[:, None] - window
    s = np.where(seen, s, -np.inf)
    m = s.max(1, initial=-np.inf)
    mu = np.where(np.isfinite(m), m, 0.0)
    p = np.exp(s - mu[:, None])
    l = p.sum(1)
    with np.errstate(divide="ignore"):
        lse = np.where(l > 0, mu + np.log(l), -np.inf)
    w = p / np.where(l > 0, l, 1.0)[:, None]
    sabs = float((np.abs(q) @ np.abs(keys).T).max(initial=0.0)) * scale
    return w @ vals, lse, w, w @ np.abs(vals), sabs


def half_step(x, t=torch.float16):
    """Half the spacing of t's numbers at |x|."""
    fi = torch.finfo(t)
    e = np.floor(np.log2(np.maximum(np.abs(x), fi.tiny)))
    return np.exp2(e) * fi.eps / 2


def out_bound(ref, a_abs, n, vmax, sabs, t=torch.float16, p_bits=11):
    """Per element: the output's rounding, and on A = sum P |v| the weights' own
    rounding (half a step, 2^-p_bits) and the scores' fp32 error: 128 products
    accumulated with truncation, 129 * 2^-23 * sabs, in the weight and its
    normaliser.  Weights below 2^-14 of the largest lose at most 2^-25 each in
    fp16, times the largest value (bf16 has no such range)."""
    es = 2 * 129 * 2.0 ** -23 * sabs + 2.0 ** -18
    sub = n * 2.0 ** -25 * vmax if t == torch.float16 else 0.0
    return half_step(ref, t) * 1.01 + (2.0 ** -p_bits + es) * a_abs + sub


def lse_bound(sabs):
    """Scores' fp32 error, and the fp32 log / maximum."""
    return 129 * 2.0 ** -23 * sabs + 2.0 ** -18 * (1 + sabs)


def evict(host, w, table, ctx, dst, budget, sink, recent, w_out_len):
    """keep [B][H][budget], weights_out, lens; moves the tokens on the Host copy."""
    B, H = w.shape[:2]
    keep = np.full((B, H, budget), -1, np.int32)
    wout = np.zeros((B, H, w_out_len), np.float32)
    lens = np.zeros(B, np.int32)
    bs, fmt = host.bs, host.fmt
    src = [a.copy() if a is not None else None for a in (host.k, host.v, host.ks, host.vs)]
    for b in range(B):
        n = int(ctx[b])
        m = lens[b] = min(n, budget)
        for h in range(H):
            x = w[b, h, :n]
            if n <= budget:
                pick = list(range(n))
            else:
                mid = range(sink, n - recent)
                # heaviest first, NaN last, equal ones by position
                best = sorted(mid, key=lambda j: (1, 0.0, j) if np.isnan(x[j]) else (0, -float(x[j]), j))
                pick = sorted(list(range(sink)) + best[:budget - sink - recent] + list(range(n - recent, n)))
            keep[b, h, :m] = pick
            wout[b, h, :m] = x[pick]
            for i in range(-(-int(m) // bs)):
                rows = pick[i * bs:min((i + 1) * bs, m)]
                d = int(dst[b][i])
                sb = [int(table[b][j // bs]) for j in rows]
                for codes, scales, c0, s0 in ((host.k, host.ks, src[0], src[2]), (host.v, host.vs, src[1], src[3])):
                    top = max(float(s0[q, h]) for q in sb) if fmt in BLOCK else 0.0
                    for r, (j, q) in enumerate(zip(rows, sb)):
                        row = c0[q, h, j % bs]
                        if fmt in BLOCK and s0[q, h] < top:
                            row = encode(fmt, f32(numbers(fmt, row) * f32(float(s0[q, h]) / top)))
                        codes[d, h, r] = row
                        if fmt == pk.KV_INT8:
                            scales[d, h, r] = s0[q, h, j % bs]
                    if fmt in BLOCK:
                        scales[d, h] = top
    return keep, wout, lens


# ------------------------------------------------------------ small cases --

def lay_out(ctx, bs, seed, spare=0, extra_cols=2):
    """Scattered blocks for sequences of ctx tokens (and `spare` more blocks
    each): (num_blocks, table int32 [B][cols], dst int32 [B][spare]).  Table
    entries behind a sequence are -1: nothing may read them."""
    nb = [-(-c // bs) for c in ctx]
    total = sum(nb) + spare * len(ctx)
    r = np.random.default_rng(seed)
    blocks = total + 3
    perm = r.permutation(blocks).astype(np.int32)
    table = np.full((len(ctx), max(nb + [1]) + extra_cols), -1, np.int32)
    at = 0
    for b, n in enumerate(nb):
        table[b, :n] = perm[at:at + n]
        at += n
    return blocks, table, perm[at:at + spare * len(ctx)].reshape(len(ctx), spare)


def random_cache(fmt, blocks, bs, hkv, seed, device="cuda"):
    """A cache of random codes (no NaN codes) and scales that differ from block
    to block by up to 2^6."""
    r = np.random.default_rng(seed)
    kw = {}
    if fmt in (pk.KV_FP8_E4M3, pk.KV_FP8_E5M2):
        kw = dict(k_scale=torch.tensor(r.uniform(0.5, 2, hkv) / 448, dtype=torch.float32),
                  v_scale=torch.tensor(r.uniform(0.5, 2, hkv) / 448, dtype=torch.float32))
        if fmt == pk.KV_FP8_E5M2:
            kw = {n: t * 448 for n, t in kw.items()}
    c = pk.PagedKVCache.allocate(fmt, blocks, bs, hkv, device=device, **kw)
    for name in ("k_cache", "v_cache"):
        t = getattr(c, name)
        x = r.standard_normal((blocks, hkv, bs, D))
        if fmt == pk.KV_FP16:
            raw = x.astype(np.float16).view(np.uint8)
        elif fmt in (pk.KV_INT8, pk.KV_INT8_BLOCK):
            raw = np.clip(np.rint(x * 35), -127, 127).astype(np.int8).view(np.uint8)
        elif fmt == pk.KV_FP8_E5M2:
            raw = (x.astype(np.float16).view(np.uint16) >> 8).astype(np.uint8)
        else:
            raw = e4m3_encode(x * 120)
        t.copy_(torch.from_numpy(raw.reshape(t.shape)))
    if fmt == pk.KV_INT8:
        for t in (c.k_scale_tok, c.v_scale_tok):
            t.copy_(torch.from_numpy((r.uniform(0.5, 2, t.shape) / 35).astype(np.float16)))
    if fmt in BLOCK:
        for t in (c.k_scale_blk, c.v_scale_blk):
            t.copy_(torch.from_numpy((np.exp2(r.uniform(-3, 3, t.shape)) / QMAX[fmt] * 3).astype(np.float32)))
    return c
