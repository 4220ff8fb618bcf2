"""ctypes binding of the attention calls of libmoe_gb300.so: packed prompts (attn_prefill), the
paged key-value cache (KvCache, kv_append) and one new token per sequence over it (attn_decode).

As in the rest of the package, bf16 tensors are int16 bit patterns, calls are asynchronous on the
current torch stream, and PyTorch supplies device memory only. All tensors of a call lie on the
current device (ValueError otherwise): that is where the library launches.
"""
from __future__ import annotations

import ctypes
import math

import torch

from .binding import MoeError, _check, _check_dev, c_int32, c_size_t, c_void_p, lib

KV_BF16, KV_E4M3 = 0, 1


class AttnDims(ctypes.Structure):
    """n_q_heads query heads over n_kv_heads key-value heads of head_dim values."""
    _fields_ = [(n, c_int32) for n in ("n_q_heads", "n_kv_heads", "head_dim")]


class HeadsView(ctypes.Structure):
    _fields_ = [("p", c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class KvCacheC(ctypes.Structure):
    _fields_ = [("dims", AttnDims), ("format", c_int32), ("page_size", c_int32), ("n_pages", c_int32),
                ("k", c_void_p), ("v", c_void_p), ("k_scale", c_void_p), ("v_scale", c_void_p)]


_FN = {}


def _fn(name: str):
    """The library's function, its argument types declared on first use."""
    f = _FN.get(name)
    if f is None:
        P, i32, vp = ctypes.POINTER, c_int32, c_void_p
        types = {
            "moe_attn_workspace_bytes": [P(AttnDims)],
            "moe_attn_prefill": [P(AttnDims), HeadsView, HeadsView, HeadsView, vp, vp, i32, i32, i32, ctypes.c_float,
                                 i32, vp, vp, vp, c_size_t, vp],
            "moe_kv_append": [P(KvCacheC), HeadsView, HeadsView, vp, vp, vp, i32, i32, i32, vp, c_size_t, vp],
            "moe_attn_decode": [P(KvCacheC), HeadsView, vp, vp, i32, i32, ctypes.c_float, vp, vp, vp, c_size_t, vp],
        }[name]
        f = getattr(lib(), name)
        f.argtypes = types
        f.restype = c_size_t if name == "moe_attn_workspace_bytes" else ctypes.c_int
        _FN[name] = f
    return f


def _device(t: torch.Tensor, name: str) -> int:
    """The current device, on which t has to lie."""
    dev = t.get_device()  # -1 on the host
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise ValueError(f"{name} must be on the current CUDA device")
    return dev


def _stream(dev: int) -> int:
    """The current stream of a device, as a handle (without building a torch.cuda.Stream, which
    costs as much as a kernel launch)."""
    return torch._C._cuda_getCurrentRawStream(dev)


def attn_workspace_bytes(dims: AttnDims) -> int:
    return int(_fn("moe_attn_workspace_bytes")(ctypes.byref(dims)))


def attn_workspace(dims: AttnDims, device="cuda") -> torch.Tensor:
    """A zero-filled workspace for the attention calls of one head layout."""
    n = attn_workspace_bytes(dims)
    if n == 0:
        raise MoeError(2, "attn_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


# What follows checks that a tensor lies on device `dev`, the current one.
def _view(t: torch.Tensor, heads: int, d: int, name: str, dev: int) -> HeadsView:
    shape = t.shape
    if t.dtype is not torch.int16 or t.get_device() != dev or len(shape) != 3 or shape[1] != heads or shape[2] != d:
        raise ValueError(f"{name} must be an int16 tensor [tokens, {heads}, {d}] on the current CUDA device")
    s = t.stride()
    if s[2] != 1:
        raise ValueError(f"{name}: the values of one head must be contiguous")
    # the stride of an axis of length one is never used, and torch may give any
    return HeadsView(t.data_ptr(), s[0] if shape[0] > 1 else d, s[1] if heads > 1 else d)


def _ints(t: torch.Tensor, n: int | None, name: str, dev: int) -> int:
    if t.dtype is not torch.int32 or t.get_device() != dev or not t.is_contiguous() or (n is not None and t.numel() != n):
        raise ValueError(f"{name} must be a contiguous int32 tensor" + ("" if n is None else f" of {n}") +
                         " on the current CUDA device")
    return t.data_ptr()


def _ws(ws: torch.Tensor, dev: int) -> int:
    if ws.dtype is not torch.uint8 or ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous uint8 tensor on the current CUDA device (attn_workspace)")
    return ws.data_ptr()


def _lse(lse: torch.Tensor | None, rows: int, heads: int, dev: int) -> int | None:
    if lse is None:
        return None
    if lse.dtype is not torch.float32 or lse.get_device() != dev or not lse.is_contiguous() or lse.shape != (rows, heads):
        raise ValueError(f"lse must be a contiguous float32 tensor [{rows}, {heads}] on the current CUDA device")
    return lse.data_ptr()


def _out(o: torch.Tensor | None, q: torch.Tensor, dev: int) -> torch.Tensor:
    if o is None:
        return torch.empty_like(q, memory_format=torch.contiguous_format)
    rows, heads, d = q.shape
    if o.dtype is not torch.int16 or o.get_device() != dev or not o.is_contiguous() or o.shape != (rows, heads, d):
        raise ValueError(f"o must be a contiguous int16 tensor [{rows}, {heads}, {d}] on the current CUDA device")
    return o


def attn_prefill(dims: AttnDims, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor,
                 cu_k: torch.Tensor, ws: torch.Tensor, *, causal: bool = True, scale: float | None = None,
                 o: torch.Tensor | None = None, lse: torch.Tensor | None = None) -> torch.Tensor:
    """moe_attn_prefill: attention over packed prompts. q [total_q, n_q_heads, head_dim], k and v
    [total_k, n_kv_heads, head_dim] (strided views of a fused projection are fine), cu_q and cu_k
    int32 [n_seqs + 1] on the device. scale defaults to 1 / sqrt(head_dim). Returns o; lse, if
    given, receives the rows' log sums [total_q, n_q_heads]."""
    hq, hkv, d = dims.n_q_heads, dims.n_kv_heads, dims.head_dim
    dev = _device(q, "q")
    qv, kv, vv = _view(q, hq, d, "q", dev), _view(k, hkv, d, "k", dev), _view(v, hkv, d, "v", dev)
    tq, tk, n = q.shape[0], k.shape[0], cu_q.numel() - 1
    if v.shape[0] != tk:
        raise ValueError("k and v must have the same number of rows")
    o = _out(o, q, dev)
    _check(_fn("moe_attn_prefill")(ctypes.byref(dims), qv, kv, vv, _ints(cu_q, None, "cu_q", dev),
                                   _ints(cu_k, n + 1, "cu_k", dev), n, tq, tk,
                                   1.0 / math.sqrt(d) if scale is None else scale, 1 if causal else 0, o.data_ptr(),
                                   _lse(lse, tq, hq, dev), _ws(ws, dev), ws.numel(), _stream(dev)), "moe_attn_prefill")
    return o


class KvCache:
    """A paged key-value cache over the caller's tensors k and v [n_pages, n_kv_heads, page_size,
    head_dim]: int16 (bf16 bits), or uint8 (e4m3 codes) with k_scale and v_scale float32
    [n_kv_heads]. The tensors are kept and written in place."""

    def __init__(self, dims: AttnDims, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor | None = None,
                 v_scale: torch.Tensor | None = None):
        if k.dtype not in (torch.int16, torch.uint8):
            raise ValueError("a cache is int16 (bf16 bits) or uint8 (e4m3 codes)")
        _check_dev(k, k.dtype, "k")
        _check_dev(v, k.dtype, "v")
        if k.dim() != 4 or k.shape != v.shape or k.shape[1] != dims.n_kv_heads or k.shape[3] != dims.head_dim:
            raise ValueError(f"k and v must be [n_pages, {dims.n_kv_heads}, page_size, {dims.head_dim}]")
        fp8 = k.dtype == torch.uint8
        if fp8 != (k_scale is not None) or fp8 != (v_scale is not None):
            raise ValueError("an e4m3 cache has k_scale and v_scale, a bf16 cache has neither")
        for name, s in (("k_scale", k_scale), ("v_scale", v_scale)) if fp8 else ():
            _check_dev(s, torch.float32, name)
            if s.shape != (dims.n_kv_heads,):
                raise ValueError(f"{name} must have {dims.n_kv_heads} values")
        if any(t.get_device() != k.get_device() for t in ((v, k_scale, v_scale) if fp8 else (v,))):
            raise ValueError("a cache's tensors must be on one device")
        self.dims, self.k, self.v, self.k_scale, self.v_scale = dims, k, v, k_scale, v_scale
        self._c = KvCacheC(dims, KV_E4M3 if fp8 else KV_BF16, k.shape[2], k.shape[0], k.data_ptr(), v.data_ptr(),
                           k_scale.data_ptr() if fp8 else None, v_scale.data_ptr() if fp8 else None)

    @classmethod
    def empty(cls, dims: AttnDims, n_pages: int, page_size: int, k_scale=None, v_scale=None, device="cuda"):
        """A new cache; e4m3 if scales are given. Its rows are uninitialised: no call reads a row
        before it has been appended."""
        t = torch.int16 if k_scale is None else torch.uint8
        k, v = (torch.empty((n_pages, dims.n_kv_heads, page_size, dims.head_dim), dtype=t, device=device)
                for _ in range(2))
        return cls(dims, k, v, k_scale, v_scale)

    @property
    def page_size(self) -> int:
        return self._c.page_size

    @property
    def c(self) -> KvCacheC:
        return self._c


def _cache(cache: KvCache, dev: int):
    if cache.k.get_device() != dev:
        raise ValueError("the cache must be on the current CUDA device")
    return ctypes.byref(cache._c)


def _table(page_table: torch.Tensor, n: int, dev: int) -> int:
    if page_table.dim() != 2 or page_table.shape[0] != n:
        raise ValueError(f"page_table must be [{n}, pages per sequence]")
    return _ints(page_table, None, "page_table", dev)


def kv_append(cache: KvCache, k: torch.Tensor, v: torch.Tensor, cu: torch.Tensor, start: torch.Tensor,
              page_table: torch.Tensor, ws: torch.Tensor) -> None:
    """moe_kv_append: row i of sequence b (rows cu[b] .. cu[b + 1] - 1 of k and v [total,
    n_kv_heads, head_dim]) is written at position start[b] + i of the cache."""
    dims = cache.dims
    dev = _device(k, "k")
    kv, vv = (_view(t, dims.n_kv_heads, dims.head_dim, name, dev) for t, name in ((k, "k"), (v, "v")))
    total, n = k.shape[0], start.numel()
    if v.shape[0] != total:
        raise ValueError("k and v must have the same number of rows")
    _check(_fn("moe_kv_append")(_cache(cache, dev), kv, vv, _ints(cu, n + 1, "cu", dev), _ints(start, n, "start", dev),
                                _table(page_table, n, dev), page_table.shape[1], n, total, _ws(ws, dev), ws.numel(),
                                _stream(dev)), "moe_kv_append")


def attn_decode(cache: KvCache, q: torch.Tensor, lens: torch.Tensor, page_table: torch.Tensor, ws: torch.Tensor, *,
                scale: float | None = None, o: torch.Tensor | None = None,
                lse: torch.Tensor | None = None) -> torch.Tensor:
    """moe_attn_decode: row b of q [n_seqs, n_q_heads, head_dim] attends to positions 0 .. lens[b] - 1
    of sequence b. Returns o; lse, if given, receives the rows' log sums [n_seqs, n_q_heads]."""
    dims = cache.dims
    hq, d, n = dims.n_q_heads, dims.head_dim, q.shape[0]
    dev = _device(q, "q")
    qv = _view(q, hq, d, "q", dev)
    o = _out(o, q, dev)
    _check(_fn("moe_attn_decode")(_cache(cache, dev), qv, _ints(lens, n, "lens", dev), _table(page_table, n, dev),
                                  page_table.shape[1], n, 1.0 / math.sqrt(d) if scale is None else scale,
                                  o.data_ptr(), _lse(lse, n, hq, dev), _ws(ws, dev), ws.numel(), _stream(dev)),
           "moe_attn_decode")
    return o
