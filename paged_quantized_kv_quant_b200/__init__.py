"""pkvq: attention over a paged, 8-bit-quantized KV cache on B200 (sm_100a).

Thin Python binding of ``libpkvq.so`` (C ABI declared in include/pkvq.h).
This module only marshals arguments: it checks tensor dtypes/devices/shapes,
passes raw device pointers and the current CUDA stream, and turns status codes
into exceptions.  Every step of the computation runs in the library's CUDA
kernels; there is no CPU or PyTorch fallback, and loading fails loudly when
the library has not been built.

Entry points (same names as the C ABI, without the ``pkvq_`` prefix):
  kv_write_quant, kv_write_block_quant (block-scaled formats),
  decode_workspace_bytes, paged_attn_decode (with the _ex options as keyword
  arguments: sliding_window, query_pos), paged_attn_decode_append,
  prompt_attn (whole packed prompts, K and V as projected),
  paged_attn_decode_weights and decode_weights_workspace_bytes (decode that
  accumulates every key's attention weight), kv_evict (eviction by those
  weights), paged_attn_prefill (sliding_window), merge_attn_states,
  kv_copy_blocks, device_status, status_string, version.  ``dcp`` adds the all-gather step
  of sequence-sharded decode (torch.distributed plumbing).

The paged calls take the batch from q (decode) or context_lens (the others).  Block
tables, context lengths and cu_seqlens may be longer than the batch needs, and out and
lse larger than the results, which are written from their start.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpkvq.so")
LIB_CHECKED_PATH = os.path.join(_HERE, "libpkvq_checked.so")

KV_FP8_E4M3 = 0
KV_INT8 = 1
KV_FP8_E5M2 = 2
KV_FP16 = 3
KV_INT8_BLOCK = 4
KV_E4M3_BLOCK = 5
_BLOCK_FORMATS = (KV_INT8_BLOCK, KV_E4M3_BLOCK)
_FP8_FORMATS = (KV_FP8_E4M3, KV_FP8_E5M2)

EXPORTED = (
    "pkvq_kv_write_quant",
    "pkvq_kv_write_block_quant",
    "pkvq_decode_weights_workspace_bytes",
    "pkvq_paged_attn_decode_weights",
    "pkvq_kv_evict",
    "pkvq_prompt_attn",
    "pkvq_decode_workspace_bytes",
    "pkvq_paged_attn_decode_append",
    "pkvq_paged_attn_decode",
    "pkvq_paged_attn_decode_ex",
    "pkvq_paged_attn_decode_noalloc",
    "pkvq_paged_attn_prefill",
    "pkvq_paged_attn_prefill_ex",
    "pkvq_merge_attn_states",
    "pkvq_kv_copy_blocks",
    "pkvq_status_string",
    "pkvq_device_status",
    "pkvq_version",
    "pkvq_last_error",
)


def elem_bytes(dtype: int) -> int:
    """Bytes per stored cache element of a format (2 for FP16, else 1)."""
    return 2 if dtype == KV_FP16 else 1


class PkvqError(RuntimeError):
    def __init__(self, status: int, what: str):
        detail = ""
        if status == 6:
            detail = ": " + _lib().pkvq_last_error().decode()
        super().__init__(f"{what}: {status_string(status)} (status {status}){detail}")
        self.status = status


class CacheStruct(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int32),
        ("num_blocks", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("k_cache", ctypes.c_void_p),
        ("v_cache", ctypes.c_void_p),
        ("k_scale", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p),
        ("k_scale_tok", ctypes.c_void_p),
        ("v_scale_tok", ctypes.c_void_p),
        ("scale_per_layer", ctypes.c_int32),
        ("k_scale_blk", ctypes.c_void_p),
        ("v_scale_blk", ctypes.c_void_p),
    ]


class PromptStruct(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("num_q_heads", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("total", ctypes.c_int64),
        ("q", ctypes.c_void_p),
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("q_token_stride", ctypes.c_int64),
        ("q_head_stride", ctypes.c_int64),
        ("k_token_stride", ctypes.c_int64),
        ("k_head_stride", ctypes.c_int64),
        ("v_token_stride", ctypes.c_int64),
        ("v_head_stride", ctypes.c_int64),
    ]


class AttnOpts(ctypes.Structure):
    _fields_ = [
        ("sliding_window", ctypes.c_int32),
        ("query_pos", ctypes.c_void_p),
    ]


_libs = {}


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Loads libpkvq.so (or another build of it); raises if it is missing."""
    path = path or os.environ.get("PKVQ_LIBRARY", LIB_PATH)
    if path in _libs:
        return _libs[path]
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} not found: build the CUDA library first "
            "(python -m paged_quantized_kv_quant_b200.build)")
    lib = ctypes.CDLL(path)
    P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    lib.pkvq_kv_write_quant.restype = I32
    lib.pkvq_kv_write_quant.argtypes = [P, P, P, P, I32, P]
    lib.pkvq_kv_write_block_quant.restype = I32
    lib.pkvq_kv_write_block_quant.argtypes = [P, P, P, ctypes.c_int64, P, P, I32, P, I32, I32, P]
    lib.pkvq_decode_weights_workspace_bytes.restype = SZ
    lib.pkvq_decode_weights_workspace_bytes.argtypes = [I32, I32, I32, I32, P]
    lib.pkvq_paged_attn_decode_weights.restype = I32
    lib.pkvq_paged_attn_decode_weights.argtypes = [P, P, P, P, P, I32, P, I32, I32, I32, I32,
                                                   ctypes.c_float, P, P, ctypes.c_int64, P, SZ,
                                                   P]
    lib.pkvq_kv_evict.restype = I32
    lib.pkvq_kv_evict.argtypes = [P, P, ctypes.c_int64, P, I32, P, I32, I32, I32, I32, P, I32,
                                  P, P, P, ctypes.c_int64, P]
    lib.pkvq_prompt_attn.restype = I32
    lib.pkvq_prompt_attn.argtypes = [P, P, P, P, I32, I32, ctypes.c_float, I32, P]
    lib.pkvq_decode_workspace_bytes.restype = SZ
    lib.pkvq_decode_workspace_bytes.argtypes = [I32, I32, I32, I32, P]
    lib.pkvq_paged_attn_decode.restype = I32
    lib.pkvq_paged_attn_decode.argtypes = [P, P, P, P, P, I32, P, I32, I32, I32, I32,
                                           ctypes.c_float, P, SZ, P]
    lib.pkvq_paged_attn_decode_noalloc.restype = I32
    lib.pkvq_paged_attn_decode_noalloc.argtypes = [P, P, P, P, P, I32, P, I32, I32, I32, I32,
                                                   ctypes.c_float, P]
    lib.pkvq_paged_attn_decode_ex.restype = I32
    lib.pkvq_paged_attn_decode_ex.argtypes = [P, P, P, P, P, I32, P, I32, I32, I32, I32,
                                              ctypes.c_float, P, P, SZ, P]
    lib.pkvq_paged_attn_decode_append.restype = I32
    lib.pkvq_paged_attn_decode_append.argtypes = [P, P, P, P, P, P, P, I32, P, I32, I32, I32,
                                                  I32, ctypes.c_float, P, P, SZ, P]
    lib.pkvq_paged_attn_prefill.restype = I32
    lib.pkvq_paged_attn_prefill.argtypes = [P, P, P, P, P, P, I32, P, I32, I32, I32,
                                            ctypes.c_float, P, SZ, P]
    lib.pkvq_paged_attn_prefill_ex.restype = I32
    lib.pkvq_paged_attn_prefill_ex.argtypes = [P, P, P, P, P, P, I32, P, I32, I32, I32,
                                               ctypes.c_float, P, P, SZ, P]
    lib.pkvq_merge_attn_states.restype = I32
    lib.pkvq_merge_attn_states.argtypes = [P, P, I32, ctypes.c_int64, I32, P, P, P]
    lib.pkvq_kv_copy_blocks.restype = I32
    lib.pkvq_kv_copy_blocks.argtypes = [P, P, P, I32, P]
    lib.pkvq_status_string.restype = ctypes.c_char_p
    lib.pkvq_status_string.argtypes = [I32]
    lib.pkvq_device_status.restype = I32
    lib.pkvq_device_status.argtypes = [ctypes.POINTER(ctypes.c_uint32), I32]
    lib.pkvq_version.restype = ctypes.c_char_p
    lib.pkvq_version.argtypes = []
    lib.pkvq_last_error.restype = ctypes.c_char_p
    lib.pkvq_last_error.argtypes = []
    _libs[path] = lib
    return lib


_current = None


def _lib():
    return _current if _current is not None else load_library()


@contextlib.contextmanager
def use_library(path: str):
    """Routes every call of this module to another build of the library
    (e.g. libpkvq_checked.so, built with PKVQ_BOUNDS_CHECK) inside the block."""
    global _current
    prev, _current = _current, load_library(path)
    try:
        yield _current
    finally:
        _current = prev


def status_string(status: int) -> str:
    return _lib().pkvq_status_string(int(status)).decode()


def version() -> str:
    return _lib().pkvq_version().decode()


def _check(status: int, what: str) -> None:
    if status != 0:
        raise PkvqError(status, what)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(stream, device: Optional[int] = None) -> int:
    """Raw stream: the given one, or the current one of a CUDA device index."""
    if stream is not None:
        return stream.cuda_stream
    if device is None:
        device = torch._C._cuda_getDevice()
    return torch._C._cuda_getCurrentRawStream(device)


_SAME_DEVICE = contextlib.nullcontext()


def _on(t: torch.Tensor, stream=None):
    """Context in which `t`'s device and the call's stream are the current ones:
    launches go there, and what the call allocates belongs to that stream."""
    if stream is not None:
        if not isinstance(stream, torch.cuda.Stream):   # anything with a raw cuda_stream
            stream = torch.cuda.ExternalStream(stream.cuda_stream, device=t.device)
        elif stream.device_index != t.get_device():
            raise ValueError(f"stream must be on the tensors' device, {t.device}")
        return torch.cuda.stream(stream)
    if t.get_device() == torch._C._cuda_getDevice():
        return _SAME_DEVICE
    return torch.cuda.device(t.device)


def _arg(name: str, t, dtype, shape: tuple, device: int) -> Optional[int]:
    """Address of a tensor of exactly this dtype and shape, contiguous, on CUDA
    device `device`; None for None."""
    if t is None:
        return None
    try:
        if (t.dtype is dtype and t.shape == shape and t.get_device() == device
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    _need(t, dtype, name)
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be on cuda:{device}")


def _room(name: str, t, dtype, shape: tuple, device: int) -> Optional[int]:
    """As _arg, for a buffer that may be larger: as many dimensions, and at least
    as many elements, which the call uses from its start (preallocated tables,
    lengths and results for more sequences than the call has)."""
    if t is None:
        return None
    try:
        if (t.dtype is dtype and t.get_device() == device and t.is_contiguous()
                and (t.shape == shape
                     or (t.dim() == len(shape) and t.numel() >= math.prod(shape)))):
            return t.data_ptr()
    except AttributeError:
        pass
    _need(t, dtype, name)
    if t.dim() != len(shape) or t.numel() < math.prod(shape):
        raise ValueError(f"{name} must hold {shape}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be on cuda:{device}")


def _table(name: str, t, rows: int, device: int):
    """(address, columns) of a block table of at least `rows` rows."""
    try:
        shape = t.shape
        if (len(shape) == 2 and shape[0] >= rows and t.dtype is torch.int32
                and t.get_device() == device and t.is_contiguous()):
            return t.data_ptr(), shape[1]
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.shape[0] < rows:
        raise ValueError(f"{name} must be a 2-D tensor of at least {rows} rows")
    return _arg(name, t, torch.int32, tuple(t.shape), device), t.shape[1]


def _lens(name: str, t, device: int):
    """(address, entries) of an int32 vector whose length is the batch."""
    try:
        if (t.dtype is torch.int32 and t.dim() == 1 and t.get_device() == device
                and t.is_contiguous()):
            return t.data_ptr(), t.numel()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or t.dim() != 1:
        raise ValueError(f"{name} must be a 1-D tensor")
    return _arg(name, t, torch.int32, tuple(t.shape), device), t.numel()


def _scratch(workspace: Optional[torch.Tensor], device: int):
    """(address, bytes) of a caller's workspace."""
    if workspace is None:
        return None, 0
    if workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on cuda:{device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _need(t: torch.Tensor, dtype, name: str, ndim: Optional[int] = None,
          host_ok: bool = False):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not (t.is_cuda or (host_ok and (t.is_pinned() or t.dim() == 1))):
        raise ValueError(f"{name} must be a CUDA tensor" +
                         (" or pinned host memory" if host_ok else ""))
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")


@dataclass
class PagedKVCache:
    """Caller-owned paged cache: elements [num_blocks][Hkv][block_size][D x
    elem_bytes] uint8 (E4M3 / E5M2 bits, int8 two's complement, or fp16 bits),
    fp32 scales for the FP8 formats ([Hkv], or [1] with scale_per_layer),
    per-(block, head, token) fp16 scales for INT8, fp32 scales
    [num_blocks][Hkv] for the block-scaled formats."""
    dtype: int
    k_cache: torch.Tensor
    v_cache: torch.Tensor
    k_scale: Optional[torch.Tensor] = None
    v_scale: Optional[torch.Tensor] = None
    k_scale_tok: Optional[torch.Tensor] = None
    v_scale_tok: Optional[torch.Tensor] = None
    scale_per_layer: bool = False
    k_scale_blk: Optional[torch.Tensor] = None
    v_scale_blk: Optional[torch.Tensor] = None

    __slots__ = ("__dict__", "__weakref__", "_kept")

    @staticmethod
    def allocate(dtype: int, num_blocks: int, block_size: int, num_kv_heads: int,
                 head_dim: int = 128, device="cuda", k_scale=None, v_scale=None,
                 scale_per_layer: bool = False, pin_host: bool = False):
        """Zeroed cache on `device`; with device="cpu" and pin_host=True, in
        pinned host memory the GPU can address (a host tier for kv_copy_blocks)."""
        shape = (num_blocks, num_kv_heads, block_size, head_dim * elem_bytes(dtype))

        def zeros(shp, dt):
            t = torch.zeros(shp, dtype=dt, device=device)
            return t.pin_memory() if pin_host else t
        kc, vc = zeros(shape, torch.uint8), zeros(shape, torch.uint8)
        if dtype in _FP8_FORMATS:
            n = 1 if scale_per_layer else num_kv_heads
            ks = torch.as_tensor(k_scale, dtype=torch.float32).reshape(-1)[:n].to(device)
            vs = torch.as_tensor(v_scale, dtype=torch.float32).reshape(-1)[:n].to(device)
            if ks.numel() != n or vs.numel() != n:
                raise ValueError(f"need {n} K and V scales")
            return PagedKVCache(dtype, kc, vc, k_scale=ks.contiguous(), v_scale=vs.contiguous(),
                                scale_per_layer=scale_per_layer)
        if dtype == KV_FP16:
            return PagedKVCache(dtype, kc, vc)
        if dtype in _BLOCK_FORMATS:
            return PagedKVCache(dtype, kc, vc, k_scale_blk=zeros(shape[:2], torch.float32),
                                v_scale_blk=zeros(shape[:2], torch.float32))
        kst, vst = zeros(shape[:3], torch.float16), zeros(shape[:3], torch.float16)
        return PagedKVCache(dtype, kc, vc, k_scale_tok=kst, v_scale_tok=vst)

    @property
    def num_blocks(self):
        return self.k_cache.shape[0]

    @property
    def num_kv_heads(self):
        return self.k_cache.shape[1]

    @property
    def block_size(self):
        return self.k_cache.shape[2]

    @property
    def head_dim(self):
        return self.k_cache.shape[3] // elem_bytes(self.dtype)

    def struct(self, device_ok: bool = False) -> CacheStruct:
        """The cache as the C ABI sees it, checked now (the caller's own copy)."""
        if device_ok:
            return self._struct(True)
        return CacheStruct.from_buffer_copy(self._c())

    def _c(self) -> CacheStruct:
        """The C struct of a call.  Kept with the object, without its tensors: they
        are checked again when one has another address, shape, layout or type."""
        try:
            key = [None if t is None else (t.data_ptr(), t.shape, t.dtype, t.is_contiguous())
                   for t in (self.k_cache, self.v_cache, self.k_scale, self.v_scale,
                             self.k_scale_tok, self.v_scale_tok, self.k_scale_blk,
                             self.v_scale_blk)]
            key += (self.dtype, self.scale_per_layer)
        except AttributeError:   # not a tensor
            return self._struct(False)
        kept = getattr(self, "_kept", None)
        if kept is None or kept[0] != key:
            self._kept = kept = (key, self._struct(False))
        return kept[1]

    def __getstate__(self):   # copies and pickles hold the fields alone
        return dict(self.__dict__)

    def _struct(self, device_ok: bool) -> CacheStruct:
        for name in ("k_cache", "v_cache"):
            _need(getattr(self, name), torch.uint8, name, 4, host_ok=device_ok)
        if self.dtype in _FP8_FORMATS:
            # (a block copy reads no scale: a host tier may keep its own copy)
            _need(self.k_scale, torch.float32, "k_scale", 1, host_ok=device_ok)
            _need(self.v_scale, torch.float32, "v_scale", 1, host_ok=device_ok)
        elif self.dtype == KV_INT8:
            _need(self.k_scale_tok, torch.float16, "k_scale_tok", 3, host_ok=device_ok)
            _need(self.v_scale_tok, torch.float16, "v_scale_tok", 3, host_ok=device_ok)
        elif self.dtype in _BLOCK_FORMATS:
            for name in ("k_scale_blk", "v_scale_blk"):
                t = getattr(self, name)
                _need(t, torch.float32, name, 2, host_ok=device_ok)
                if t.shape != self.k_cache.shape[:2]:
                    raise ValueError(f"{name} must be [num_blocks][num_kv_heads]")
        if self.v_cache.shape != self.k_cache.shape:
            raise ValueError("k_cache and v_cache must have the same shape")
        if self.dtype == KV_INT8 and not (self.k_scale_tok.shape == self.v_scale_tok.shape ==
                                          self.k_cache.shape[:3]):
            raise ValueError("per-token scales must be [num_blocks][num_kv_heads][block_size]")
        if not device_ok and len({t.get_device() for t in (
                self.k_cache, self.v_cache, self.k_scale, self.v_scale, self.k_scale_tok,
                self.v_scale_tok, self.k_scale_blk, self.v_scale_blk) if t is not None}) > 1:
            raise ValueError("the cache's tensors must be on one device")
        nb, hkv, bs, rb = self.k_cache.shape
        return CacheStruct(self.dtype, nb, bs, hkv, rb // elem_bytes(self.dtype),
                           self.k_cache.data_ptr(), self.v_cache.data_ptr(),
                           self.k_scale.data_ptr() if self.k_scale is not None else None,
                           self.v_scale.data_ptr() if self.v_scale is not None else None,
                           self.k_scale_tok.data_ptr() if self.k_scale_tok is not None else None,
                           self.v_scale_tok.data_ptr() if self.v_scale_tok is not None else None,
                           1 if self.scale_per_layer else 0,
                           self.k_scale_blk.data_ptr() if self.k_scale_blk is not None else None,
                           self.v_scale_blk.data_ptr() if self.v_scale_blk is not None else None)


def kv_write_quant(cache: PagedKVCache, k: torch.Tensor, v: torch.Tensor,
                   slot_mapping: torch.Tensor, stream=None) -> None:
    """Quantizes fp16 K/V [T][Hkv][D] into the cache slots (negative = skip)."""
    _need(k, torch.float16, "k", 3)
    _need(v, torch.float16, "v", 3)
    _need(slot_mapping, torch.int32, "slot_mapping", 1)
    cs = cache._c()
    _check(_lib().pkvq_kv_write_quant(ctypes.byref(cs), _ptr(k), _ptr(v), _ptr(slot_mapping),
                                      int(slot_mapping.shape[0]), _stream(stream)),
           "kv_write_quant")


def kv_write_block_quant(cache: PagedKVCache, k: torch.Tensor, v: torch.Tensor,
                         cu_seqlens_new: torch.Tensor, block_table: torch.Tensor,
                         context_lens: torch.Tensor, max_new_len: int, stream=None) -> None:
    """Quantizes fp16 K/V [T][Hkv][D], the last cu[b + 1] - cu[b] positions of
    every sequence b (packed), into a block-scaled cache; context_lens counts
    them.  A block's scale covers the tokens written to it: it grows when a
    louder token arrives, and the block's older codes are rounded again."""
    cs = cache._c()
    dev = cache.k_cache.get_device()
    lens, B = _lens("context_lens", context_lens, dev)
    table, cols = _table("block_table", block_table, B, dev)
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("k must be [tokens][num_kv_heads][head_dim]")
    rows = (k.shape[0], cs.num_kv_heads, cs.head_dim)
    args = (_arg("k", k, torch.float16, rows, dev), _arg("v", v, torch.float16, rows, dev), rows[0],
            _room("cu_seqlens_new", cu_seqlens_new, torch.int32, (B + 1,), dev),
            table, cols, lens, B, int(max_new_len))
    with _on(k, stream):
        _check(_lib().pkvq_kv_write_block_quant(ctypes.byref(cs), *args, _stream(stream, dev)),
               "kv_write_block_quant")


def decode_workspace_bytes(cache: PagedKVCache, batch: int, q_len: int, num_q_heads: int,
                           max_context_len: int) -> int:
    cs = cache._c()
    return int(_lib().pkvq_decode_workspace_bytes(batch, q_len, num_q_heads, max_context_len,
                                                  ctypes.byref(cs)))


def _opts(sliding_window: int, query_pos: Optional[torch.Tensor]):
    if not sliding_window and query_pos is None:
        return None
    return AttnOpts(int(sliding_window), None if query_pos is None else query_pos.data_ptr())


def _queries(q: torch.Tensor, cs: CacheStruct, device: int):
    """(address, batch, q_len, query heads, shape) of decode queries for a cache."""
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError(f"q must be [batch][q_len][num_q_heads][{cs.head_dim}]")
    shape = tuple(q.shape)
    B, q_len, Hq, D = shape
    if D != cs.head_dim:
        raise ValueError(f"q must be [batch][q_len][num_q_heads][{cs.head_dim}]")
    if q.dtype is torch.float16 and q.get_device() == device and q.is_contiguous():
        return q.data_ptr(), B, q_len, Hq, shape
    return _arg("q", q, torch.float16, shape, device), B, q_len, Hq, shape


def paged_attn_decode(cache: PagedKVCache, q: torch.Tensor, block_table: torch.Tensor,
                      context_lens: torch.Tensor, max_context_len: int, softmax_scale: float,
                      out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None,
                      sliding_window: int = 0,
                      query_pos: Optional[torch.Tensor] = None) -> torch.Tensor:
    """q fp16 [B][q_len][Hq][D] -> out fp16 [B][q_len][Hq][D] (lse fp32 [B][q_len][Hq]).
    sliding_window > 0 limits every query to its last `sliding_window` keys;
    query_pos (int32 [B][q_len]) gives each query's position among the keys."""
    cs = cache._c()
    dev = cache.k_cache.get_device()
    q_ptr, B, q_len, Hq, shape = _queries(q, cs, dev)
    table, cols = _table("block_table", block_table, B, dev)
    with _on(q, stream):
        if out is None:
            out = torch.empty_like(q)
        if workspace is None and B:   # contents need not be initialised
            need = _lib().pkvq_decode_workspace_bytes(B, q_len, Hq, max_context_len,
                                                      ctypes.byref(cs))
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
        ws, wbytes = _scratch(workspace, dev)
        _arg("query_pos", query_pos, torch.int32, (B, q_len), dev)
        opts = _opts(sliding_window, query_pos)
        _check(_lib().pkvq_paged_attn_decode_ex(
            ctypes.byref(cs), q_ptr, _room("out", out, torch.float16, shape, dev),
            _room("lse", lse, torch.float32, shape[:3], dev),
            table, cols, _room("context_lens", context_lens, torch.int32, (B,), dev),
            B, q_len, Hq,
            int(max_context_len), float(softmax_scale),
            None if opts is None else ctypes.byref(opts), ws, wbytes, _stream(stream, dev)),
            "paged_attn_decode")
    return out


def decode_weights_workspace_bytes(cache: PagedKVCache, batch: int, q_len: int,
                                   num_q_heads: int, max_context_len: int) -> int:
    cs = cache._c()
    with _on(cache.k_cache):
        return int(_lib().pkvq_decode_weights_workspace_bytes(
            batch, q_len, num_q_heads, max_context_len, ctypes.byref(cs)))


def paged_attn_decode_weights(cache: PagedKVCache, q: torch.Tensor, block_table: torch.Tensor,
                              context_lens: torch.Tensor, max_context_len: int,
                              softmax_scale: float, weights: torch.Tensor,
                              out: Optional[torch.Tensor] = None,
                              lse: Optional[torch.Tensor] = None,
                              workspace: Optional[torch.Tensor] = None, stream=None,
                              sliding_window: int = 0,
                              query_pos: Optional[torch.Tensor] = None) -> torch.Tensor:
    """paged_attn_decode that also adds every key's softmax weight, summed over
    the query rows of its KV head, to weights fp32 [B][Hkv][>= max_context_len]
    (zero the entries of new tokens).  Input of kv_evict."""
    cs = cache._c()
    dev = cache.k_cache.get_device()
    q_ptr, B, q_len, Hq, shape = _queries(q, cs, dev)
    table, cols = _table("block_table", block_table, B, dev)
    if not isinstance(weights, torch.Tensor) or weights.dim() != 3:
        raise ValueError("weights must be [batch][num_kv_heads][positions]")
    W = weights.shape[2]
    with _on(q, stream):
        if out is None:
            out = torch.empty_like(q)
        if workspace is None and B:   # contents need not be initialised
            need = _lib().pkvq_decode_weights_workspace_bytes(B, q_len, Hq, max_context_len,
                                                              ctypes.byref(cs))
            workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
        ws, wbytes = _scratch(workspace, dev)
        _arg("query_pos", query_pos, torch.int32, (B, q_len), dev)
        opts = _opts(sliding_window, query_pos)
        _check(_lib().pkvq_paged_attn_decode_weights(
            ctypes.byref(cs), q_ptr, _room("out", out, torch.float16, shape, dev),
            _room("lse", lse, torch.float32, shape[:3], dev),
            table, cols, _room("context_lens", context_lens, torch.int32, (B,), dev),
            B, q_len, Hq,
            int(max_context_len), float(softmax_scale),
            None if opts is None else ctypes.byref(opts),
            _arg("weights", weights, torch.float32, (B, cs.num_kv_heads, W), dev), W, ws, wbytes,
            _stream(stream, dev)), "paged_attn_decode_weights")
    return out


def kv_evict(cache: PagedKVCache, weights: torch.Tensor, block_table: torch.Tensor,
             context_lens: torch.Tensor, dst_block_table: torch.Tensor, budget: int,
             num_sink: int = 0, num_recent: int = 0,
             weights_out: Optional[torch.Tensor] = None, keep: Optional[torch.Tensor] = None,
             new_context_lens: Optional[torch.Tensor] = None, stream=None):
    """Keeps at most `budget` tokens of every (sequence, KV head) -- the first
    num_sink, the last num_recent and the heaviest others by weights fp32
    [B][Hkv][W] -- and moves them, in order, to the blocks of dst_block_table
    (distinct blocks that hold no token of these sequences).
    Returns (new_context_lens int32 [B], weights_out fp32 [B][Hkv][W'], keep
    int32 [B][Hkv][budget]: the kept positions, -1 behind the last)."""
    cs = cache._c()
    dev = cache.k_cache.get_device()
    lens, B = _lens("context_lens", context_lens, dev)
    H, budget = cs.num_kv_heads, int(budget)
    table, cols = _table("block_table", block_table, B, dev)
    dst_table, dst_cols = _table("dst_block_table", dst_block_table, B, dev)
    if budget < 1:
        raise ValueError("budget must be at least 1")
    if not isinstance(weights, torch.Tensor) or weights.dim() != 3:
        raise ValueError("weights must be [batch][num_kv_heads][positions]")
    W = weights.shape[2]
    with _on(weights, stream):
        if weights_out is None:
            weights_out = torch.empty((B, H, max(W, budget)), dtype=torch.float32,
                                      device=weights.device)
        if keep is None:
            keep = torch.empty((B, H, budget), dtype=torch.int32, device=weights.device)
        if new_context_lens is None:
            new_context_lens = torch.empty_like(context_lens)
        w_out = weights_out.shape[-1]
        _check(_lib().pkvq_kv_evict(
            ctypes.byref(cs), _arg("weights", weights, torch.float32, (B, H, W), dev), W,
            table, cols, lens, B, budget,
            int(num_sink), int(num_recent),
            dst_table, dst_cols,
            _arg("keep", keep, torch.int32, (B, H, budget), dev),
            _arg("new_context_lens", new_context_lens, torch.int32, (B,), dev),
            _arg("weights_out", weights_out, torch.float32, (B, H, w_out), dev), w_out,
            _stream(stream, dev)), "kv_evict")
    return new_context_lens, weights_out, keep


def paged_attn_decode_append(cache: PagedKVCache, k_new: torch.Tensor, v_new: torch.Tensor,
                             q: torch.Tensor, block_table: torch.Tensor,
                             context_lens: torch.Tensor, max_context_len: int,
                             softmax_scale: float, out: Optional[torch.Tensor] = None,
                             lse: Optional[torch.Tensor] = None,
                             workspace: Optional[torch.Tensor] = None, stream=None,
                             sliding_window: int = 0) -> torch.Tensor:
    """One decode step with its KV write: k_new / v_new fp16 [B][q_len][Hkv][D]
    are the keys and values of each sequence's last q_len positions; they are
    quantised into the cache (as kv_write_quant) and attention runs as
    paged_attn_decode."""
    cs = cache._c()
    dev = cache.k_cache.get_device()
    q_ptr, B, q_len, Hq, shape = _queries(q, cs, dev)
    table, cols = _table("block_table", block_table, B, dev)
    new = (B, q_len, cs.num_kv_heads, cs.head_dim)
    with _on(q, stream):
        if out is None:
            out = torch.empty_like(q)
        if workspace is None and B:   # contents need not be initialised
            need = _lib().pkvq_decode_workspace_bytes(B, q_len, Hq, max_context_len,
                                                      ctypes.byref(cs))
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
        ws, wbytes = _scratch(workspace, dev)
        opts = _opts(sliding_window, None)
        _check(_lib().pkvq_paged_attn_decode_append(
            ctypes.byref(cs), _arg("k_new", k_new, torch.float16, new, dev),
            _arg("v_new", v_new, torch.float16, new, dev),
            q_ptr, _room("out", out, torch.float16, shape, dev),
            _room("lse", lse, torch.float32, shape[:3], dev),
            table, cols, _room("context_lens", context_lens, torch.int32, (B,), dev),
            B, q_len, Hq,
            int(max_context_len), float(softmax_scale),
            None if opts is None else ctypes.byref(opts), ws, wbytes, _stream(stream, dev)),
            "paged_attn_decode_append")
    return out


def paged_attn_prefill(cache: PagedKVCache, q: torch.Tensor, cu_seqlens_q: torch.Tensor,
                       block_table: torch.Tensor, context_lens: torch.Tensor, max_q_len: int,
                       softmax_scale: float, out: Optional[torch.Tensor] = None,
                       lse: Optional[torch.Tensor] = None, stream=None,
                       sliding_window: int = 0) -> torch.Tensor:
    """q fp16 [total_q][Hq][D] (packed varlen) -> out fp16 [total_q][Hq][D]."""
    cs = cache._c()
    dev = cache.k_cache.get_device()
    if not isinstance(q, torch.Tensor) or q.dim() != 3 or q.shape[2] != cs.head_dim:
        raise ValueError(f"q must be [total_q][num_q_heads][{cs.head_dim}]")
    shape = tuple(q.shape)
    q_ptr = _arg("q", q, torch.float16, shape, dev)
    lens, B = _lens("context_lens", context_lens, dev)
    table, cols = _table("block_table", block_table, B, dev)
    with _on(q, stream):
        if out is None:
            out = torch.empty_like(q)
        opts = _opts(sliding_window, None)
        _check(_lib().pkvq_paged_attn_prefill_ex(
            ctypes.byref(cs), q_ptr, _room("out", out, torch.float16, shape, dev),
            _room("lse", lse, torch.float32, shape[:2], dev),
            _room("cu_seqlens_q", cu_seqlens_q, torch.int32, (B + 1,), dev),
            table, cols, lens, B, int(max_q_len),
            shape[1], float(softmax_scale), None if opts is None else ctypes.byref(opts), None,
            0, _stream(stream, dev)), "paged_attn_prefill")
    return out


_PROMPT_DTYPES = {torch.float16: 0, torch.bfloat16: 1}


def prompt_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                max_len: int, softmax_scale: float, out: Optional[torch.Tensor] = None,
                lse: Optional[torch.Tensor] = None, stream=None,
                sliding_window: int = 0) -> torch.Tensor:
    """Causal attention over packed whole prompts: q [T][Hq][D], k and v
    [T][Hkv][D], fp16 or bf16, the rows of sequence b from cu_seqlens[b] to
    cu_seqlens[b + 1] (int32 [B + 1]) -> out [T][Hq][D] (lse fp32 [T][Hq]).  The
    last dimension is contiguous; token and head strides may be those of
    slices of one fused projection (multiples of 8 elements)."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    dtype = _PROMPT_DTYPES.get(q.dtype)
    if dtype is None:
        raise TypeError(f"q must be fp16 or bf16, got {q.dtype}")
    dev = q.get_device()
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dtype != q.dtype or t.get_device() != dev:
            raise TypeError(f"{name} must be {q.dtype} on cuda:{dev}")
        if t.dim() != 3 or t.stride(2) != 1:
            raise ValueError(f"{name} must have 3 dims, the last one contiguous")
        if t.shape[0] != q.shape[0] or t.shape[2] != q.shape[2]:
            raise ValueError(f"{name} must have q's tokens and head_dim")
    if k.shape != v.shape:
        raise ValueError("k and v must have the same shape")
    T, Hq, D = q.shape
    _need(cu_seqlens, torch.int32, "cu_seqlens", 1)
    if cu_seqlens.shape[0] < 1 or cu_seqlens.get_device() != dev:
        raise ValueError(f"cu_seqlens must hold batch + 1 entries on cuda:{dev}")
    (qt, qh, _), (kt, kh, _), (vt, vh, _) = q.stride(), k.stride(), v.stride()
    # (a dimension of one element may carry any stride)
    if Hq == 1:
        qh = D
    if k.shape[1] == 1:
        kh = vh = D
    if T == 1:
        qt, kt, vt = Hq * D, k.shape[1] * D, k.shape[1] * D
    ps = PromptStruct(dtype, D, Hq, k.shape[1], T, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                      qt, qh, kt, kh, vt, vh)
    with _on(q, stream):
        if out is None:
            out = torch.empty((T, Hq, D), dtype=q.dtype, device=q.device)
        _check(_lib().pkvq_prompt_attn(
            ctypes.byref(ps), _arg("out", out, q.dtype, (T, Hq, D), dev),
            _arg("lse", lse, torch.float32, (T, Hq), dev), cu_seqlens.data_ptr(),
            cu_seqlens.shape[0] - 1, int(max_len), float(softmax_scale), int(sliding_window),
            _stream(stream, dev)), "prompt_attn")
    return out


def merge_attn_states(parts_out: torch.Tensor, parts_lse: torch.Tensor,
                      out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                      stream=None):
    """parts_out fp16 [R][..., D], parts_lse fp32 [R][...] (results of the same
    queries over disjoint key sets) -> (out fp16 [..., D], lse fp32 [...])."""
    _need(parts_out, torch.float16, "parts_out")
    _need(parts_lse, torch.float32, "parts_lse")
    R, D = int(parts_out.shape[0]), int(parts_out.shape[-1])
    if tuple(parts_lse.shape) != tuple(parts_out.shape[:-1]):
        raise ValueError("parts_lse must match parts_out without its last dimension")
    n = parts_lse.numel() // max(R, 1)
    if out is None:
        out = torch.empty(parts_out.shape[1:], dtype=torch.float16, device=parts_out.device)
    if lse is None:
        lse = torch.empty(parts_lse.shape[1:], dtype=torch.float32, device=parts_out.device)
    _need(out, torch.float16, "out")
    _need(lse, torch.float32, "lse")
    _check(_lib().pkvq_merge_attn_states(_ptr(parts_out), _ptr(parts_lse), R, n, D, _ptr(out),
                                         _ptr(lse), _stream(stream)), "merge_attn_states")
    return out, lse


def kv_copy_blocks(dst: PagedKVCache, src: PagedKVCache, pairs: torch.Tensor,
                   stream=None) -> None:
    """Block pairs[i][0] of src -> block pairs[i][1] of dst (either cache on the
    GPU or in pinned host memory; pairs int32 [n][2] on the GPU)."""
    _need(pairs, torch.int32, "pairs", 2)
    sd, ss = dst.struct(device_ok=True), src.struct(device_ok=True)
    _check(_lib().pkvq_kv_copy_blocks(ctypes.byref(sd), ctypes.byref(ss), _ptr(pairs),
                                      int(pairs.shape[0]), _stream(stream)), "kv_copy_blocks")


def device_status(clear: bool = True) -> int:
    """Device status word (0 = no device-side check fired); synchronizes."""
    v = ctypes.c_uint32(0)
    _check(_lib().pkvq_device_status(ctypes.byref(v), 1 if clear else 0), "device_status")
    return int(v.value)
