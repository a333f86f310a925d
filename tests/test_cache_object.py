"""The cache object and the C struct that it keeps between calls: copies, pickles, freed
tensors, and changes in place.  CPU: host tensors stand in (only the check that they
are on a GPU is lifted; nothing is launched)."""
import copy
import dataclasses
import gc
import pickle
import weakref

import numpy as np
import pytest
import torch

import paged_quantized_kv_quant_b200 as pk


@pytest.fixture
def host_tensors(monkeypatch):
    def need(t, dtype, name, ndim=None, host_ok=False):
        if not isinstance(t, torch.Tensor) or t.dtype != dtype:
            raise TypeError(name)
        if not t.is_contiguous() or (ndim is not None and t.dim() != ndim):
            raise ValueError(name)
    monkeypatch.setattr(pk, "_need", need)


def used(fmt=pk.KV_INT8_BLOCK, **kw):
    """A cache after a call's look at its struct."""
    c = pk.PagedKVCache.allocate(fmt, 8, 16, 2, device="cpu", **kw)
    c._c()
    return c


@pytest.mark.parametrize("fmt", [pk.KV_FP8_E4M3, pk.KV_INT8, pk.KV_FP16, pk.KV_E4M3_BLOCK])
def test_a_used_cache_copies_and_pickles(host_tensors, fmt):
    c = used(fmt, **(dict(k_scale=[1.0, 2.0], v_scale=[3.0, 4.0]) if fmt == pk.KV_FP8_E4M3 else {}))
    c.k_cache.random_(0, 100)
    assert set(vars(c)) == {f.name for f in dataclasses.fields(c)}
    again = pk.PagedKVCache(**vars(c))
    assert again._c().k_cache == c.k_cache.data_ptr()
    for d in (copy.deepcopy(c), pickle.loads(pickle.dumps(c))):
        assert d.dtype == fmt and torch.equal(d.k_cache, c.k_cache)
        assert d._c().k_cache == d.k_cache.data_ptr() != c.k_cache.data_ptr()
    s = copy.copy(c)
    s.k_cache = s.k_cache.clone()
    assert s._c().k_cache == s.k_cache.data_ptr() and c._c().k_cache == c.k_cache.data_ptr()


def test_a_replaced_tensor_is_freed(host_tensors):
    c = used()
    gone = weakref.ref(c.k_cache.untyped_storage())
    old = weakref.ref(c.k_cache)
    c.k_cache = None
    gc.collect()
    assert old() is None and gone() is None
    with pytest.raises(TypeError):
        c._c()


def test_changes_in_place_are_noticed(host_tensors):
    c = used(pk.KV_FP8_E4M3, k_scale=[1.0, 2.0], v_scale=[3.0, 4.0])
    at = c.k_cache.data_ptr()
    for t in (c.k_cache, c.v_cache):            # another block size in the same memory
        t.data = t.data.view(4, 2, 32, 128)
    cs = c._c()
    assert (cs.k_cache, cs.num_blocks, cs.block_size) == (at, 4, 32)
    for t in (c.k_cache, c.v_cache):
        t.resize_(2, 2, 32, 128)                # fewer blocks
    assert c._c().num_blocks == 2 and c.k_cache.data_ptr() == at
    c.k_cache.transpose_(1, 2)
    with pytest.raises(ValueError):
        c._c()
    c.k_cache.transpose_(1, 2)
    assert c._c().num_blocks == 2
    c.v_cache.resize_(1, 2, 32, 128)
    with pytest.raises(ValueError):
        c._c()
    b = used()
    b.v_scale_blk.data = b.v_scale_blk.data.view(torch.int32)
    with pytest.raises(TypeError):
        b._c()
    b = used()
    b.k_scale_blk.resize_(4, 2)
    with pytest.raises(ValueError):
        b._c()


def test_a_callers_struct_is_its_own(host_tensors):
    c = used()
    cs = c.struct()
    cs.num_blocks = 1
    assert c._c().num_blocks == 8 and c.struct().num_blocks == 8


@pytest.mark.gpu
def test_copies_give_the_same_results():
    from pkvq_ref64 import D, random_cache
    c = random_cache(pk.KV_INT8_BLOCK, 8, 16, 2, 131)
    t = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    n = torch.tensor([50], dtype=torch.int32, device="cuda")
    q = torch.from_numpy(np.random.default_rng(132).standard_normal((1, 1, 4, D))).half().cuda()
    out = pk.paged_attn_decode(c, q, t, n, 50, 0.1)
    for d in (copy.deepcopy(c), pickle.loads(pickle.dumps(c))):
        c.k_cache.zero_()
        assert torch.equal(pk.paged_attn_decode(d, q, t, n, 50, 0.1), out)
