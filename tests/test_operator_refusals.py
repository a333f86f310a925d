"""Host-side refusals of the block-scaled, weight and eviction entry points
(CPU only: nothing is launched, the pointers are never dereferenced)."""
import ctypes

import pytest
import torch

import paged_quantized_kv_quant_b200 as pk
from paged_quantized_kv_quant_b200 import build as pkbuild

OK, INVALID, UNSUPPORTED, MISALIGNED, SMALL = 0, 1, 2, 3, 4
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    pkbuild.build()
    return pk.load_library()


def cache(**kw):
    base = dict(dtype=pk.KV_INT8_BLOCK, num_blocks=64, block_size=16, num_kv_heads=2, head_dim=128,
                k_cache=0x1000, v_cache=0x2000, k_scale_blk=0x3000, v_scale_blk=0x4000)
    base.update(kw)
    return pk.CacheStruct(**base)


def write(lib, c, **kw):
    a = dict(k=0x10000, v=0x20000, T=8, cu=0x30000, bt=0x40000, maxb=8, ctx=0x50000, B=2, n=4)
    a.update(kw)
    return lib.pkvq_kv_write_block_quant(ctypes.byref(c), P(a["k"]), P(a["v"]), a["T"], P(a["cu"]), P(a["bt"]),
                                         a["maxb"], P(a["ctx"]), a["B"], a["n"], None)


def test_block_write_refusals(lib):
    assert write(lib, cache(dtype=pk.KV_FP8_E4M3, k_scale=0x3000, v_scale=0x4000)) == UNSUPPORTED
    assert write(lib, cache(k_scale_blk=None)) == INVALID
    assert write(lib, cache(v_scale_blk=None)) == INVALID
    assert write(lib, cache(v_scale_blk=0x4004)) == MISALIGNED
    assert write(lib, cache(dtype=6)) == UNSUPPORTED
    assert write(lib, cache(head_dim=64)) == UNSUPPORTED
    for name in ("k", "v", "cu", "bt", "ctx"):
        assert write(lib, cache(), **{name: None}) == INVALID
    assert write(lib, cache(), k=0x10008) == MISALIGNED
    assert write(lib, cache(), B=-1) == INVALID
    assert write(lib, cache(), n=-1) == INVALID
    assert write(lib, cache(), B=1 << 20, n=1 << 20) == UNSUPPORTED    # the launch grid
    assert write(lib, cache(), n=(1 << 31) - 1, B=16) == UNSUPPORTED
    assert write(lib, cache(num_kv_heads=65536, num_blocks=1)) == UNSUPPORTED
    assert write(lib, cache(), T=-1) == INVALID
    assert write(lib, cache(), T=0, k=None) == OK
    assert write(lib, cache(), B=0, k=None) == OK
    assert write(lib, cache(), n=0, k=None) == OK


def test_slot_write_refuses_block_scaled_caches(lib):
    c = cache()
    assert lib.pkvq_kv_write_quant(ctypes.byref(c), P(16), P(16), P(16), 1, None) == UNSUPPORTED


def weights(lib, c, **kw):
    a = dict(q=0x10000, out=0x20000, bt=0x30000, maxb=64, ctx=0x40000, B=2, ql=1, Hq=8, maxctx=1024,
             scale=0.088, w=0x50000, stride=1024, ws=None, wsb=0, opts=None)
    a.update(kw)
    return lib.pkvq_paged_attn_decode_weights(
        ctypes.byref(c), P(a["q"]), P(a["out"]), None, P(a["bt"]), a["maxb"], P(a["ctx"]), a["B"], a["ql"],
        a["Hq"], a["maxctx"], ctypes.c_float(a["scale"]), a["opts"], P(a["w"]), a["stride"], P(a["ws"]),
        a["wsb"], None)


def test_weights_refusals(lib):
    c = cache()
    assert weights(lib, c, w=None) == INVALID
    assert weights(lib, c, stride=1023) == INVALID
    assert weights(lib, c, ql=17) == INVALID
    assert weights(lib, c, Hq=7) == INVALID
    assert weights(lib, c, Hq=34) == UNSUPPORTED
    assert weights(lib, c, q=None) == INVALID
    assert weights(lib, c, q=0x10008) == MISALIGNED
    assert weights(lib, c, scale=float("nan")) == INVALID
    assert weights(lib, c, maxb=63) == INVALID
    assert weights(lib, c, B=65536) == UNSUPPORTED
    assert weights(lib, c, opts=ctypes.byref(pk.AttnOpts(-1, None))) == INVALID
    need = lib.pkvq_decode_weights_workspace_bytes(2, 1, 8, 1024, ctypes.byref(c))
    # at least the scores: 2 sequences x 2 heads x 1024 keys x 4 rows, fp32
    assert need > 2 * 2 * 1024 * 4 * 4
    assert weights(lib, c) == SMALL
    assert weights(lib, c, ws=0x60000, wsb=need - 1) == SMALL
    assert weights(lib, c, ws=0x60008, wsb=need) == MISALIGNED
    assert weights(lib, c, B=0, w=None) == OK
    assert lib.pkvq_decode_weights_workspace_bytes(2, 1, 7, 1024, ctypes.byref(c)) == 0
    assert lib.pkvq_decode_weights_workspace_bytes(2, 1, 34, 1024, ctypes.byref(c)) == 0
    assert lib.pkvq_decode_weights_workspace_bytes(2, 1, 8, 1024, None) == 0


def evict(lib, c, **kw):
    a = dict(w=0x10000, ws=500, bt=0x20000, maxb=32, ctx=0x30000, B=2, budget=64, sink=4, recent=8,
             dst=0x40000, dstb=4, keep=0x50000, lens=0x60000, wo=0x70000, wos=500)
    a.update(kw)
    return lib.pkvq_kv_evict(ctypes.byref(c), P(a["w"]), a["ws"], P(a["bt"]), a["maxb"], P(a["ctx"]), a["B"],
                             a["budget"], a["sink"], a["recent"], P(a["dst"]), a["dstb"], P(a["keep"]),
                             P(a["lens"]), P(a["wo"]), a["wos"], None)


def test_evict_refusals(lib):
    c = cache()
    assert evict(lib, c, budget=0) == INVALID
    assert evict(lib, c, sink=-1) == INVALID
    assert evict(lib, c, recent=-1) == INVALID
    assert evict(lib, c, sink=60, recent=5) == INVALID
    assert evict(lib, c, sink=(1 << 31) - 1, recent=(1 << 31) - 1) == INVALID
    assert evict(lib, c, dstb=3) == INVALID           # 3 * 16 < 64
    assert evict(lib, c, wos=63) == INVALID
    assert evict(lib, c, wo=0x10000) == INVALID       # in place
    assert evict(lib, c, wo=0x10000 + 4 * (4 * 500 - 1)) == INVALID   # the last weight
    assert evict(lib, c, wo=0x10000 - 4 * (4 * 500 - 1)) == INVALID
    assert evict(lib, c, lens=0x30000) == INVALID     # in place
    for name in ("w", "bt", "ctx", "dst", "keep", "lens"):
        assert evict(lib, c, **{name: None}) == INVALID
    assert evict(lib, c, B=65536) == UNSUPPORTED
    assert evict(lib, c, budget=(1 << 30) + 1, dstb=(1 << 27), wos=1 << 31) == UNSUPPORTED
    assert evict(lib, cache(block_size=24)) == UNSUPPORTED
    assert evict(lib, c, B=0, w=None) == OK


def test_copy_refuses_mixed_formats(lib):
    a, b = cache(), cache(dtype=pk.KV_E4M3_BLOCK)
    assert lib.pkvq_kv_copy_blocks(ctypes.byref(a), ctypes.byref(b), P(16), 1, None) == INVALID


def test_python_checks_before_any_call():
    """Shapes, types and devices that the binding refuses itself."""
    c = pk.PagedKVCache(pk.KV_INT8_BLOCK, *(torch.zeros((4, 2, 16, 128), dtype=torch.uint8) for _ in "kv"),
                        k_scale_blk=torch.zeros((4, 2)), v_scale_blk=torch.zeros((4, 2)))
    with pytest.raises(ValueError, match="CUDA"):
        c.struct()
    i32 = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        pk.kv_write_block_quant(c, torch.zeros((1, 2, 128)), torch.zeros((1, 2, 128)), i32, i32[None], i32[:1], 1)
    with pytest.raises(ValueError):
        pk.kv_evict(c, torch.zeros((1, 2, 16)), i32[None], i32[:1], i32[None], 4)


def prompt(lib, out=0x40000, cu=0x50000, B=2, mx=64, scale=0.088, window=0, **kw):
    a = dict(dtype=0, head_dim=128, num_q_heads=8, num_kv_heads=2, total=100, q=0x10000, k=0x20000, v=0x30000,
             q_token_stride=1024, q_head_stride=128, k_token_stride=256, k_head_stride=128,
             v_token_stride=256, v_head_stride=128)
    a.update(kw)
    s = pk.PromptStruct(**a)
    return lib.pkvq_prompt_attn(ctypes.byref(s), P(out), None, P(cu), B, mx, ctypes.c_float(scale), window, None)


def test_prompt_refusals(lib):
    assert lib.pkvq_prompt_attn(None, P(16), None, P(16), 1, 1, ctypes.c_float(1), 0, None) == INVALID
    assert prompt(lib, dtype=2) == UNSUPPORTED
    assert prompt(lib, head_dim=64) == UNSUPPORTED
    assert prompt(lib, num_q_heads=7) == INVALID
    assert prompt(lib, num_q_heads=258) == UNSUPPORTED           # group 129
    assert prompt(lib, B=65536) == UNSUPPORTED
    assert prompt(lib, B=-1) == INVALID
    assert prompt(lib, mx=-1) == INVALID
    assert prompt(lib, total=-1) == INVALID
    assert prompt(lib, window=-1) == INVALID
    assert prompt(lib, scale=float("inf")) == INVALID
    for name in ("q", "k", "v"):
        assert prompt(lib, **{name: None}) == INVALID
        assert prompt(lib, **{name: 0x10008}) == MISALIGNED
        assert prompt(lib, **{name + "_token_stride": 1028}) == MISALIGNED
        assert prompt(lib, **{name + "_head_stride": 132}) == MISALIGNED
        assert prompt(lib, **{name + "_head_stride": 0}) == INVALID
        assert prompt(lib, **{name + "_token_stride": 1 << 40}) == INVALID
    assert prompt(lib, out=None) == INVALID
    assert prompt(lib, out=0x40008) == MISALIGNED
    assert prompt(lib, cu=None) == INVALID
    for kw in (dict(B=0), dict(mx=0), dict(total=0)):
        assert prompt(lib, **kw) == OK
