"""ctypes binding of the 8-bit expert calls of libmoe_gb300.so: tokens sorted by expert (sort_tokens,
dispatch) and brought back (combine), grouped products of e4m3 rows and weights (gemm_e4m3), the
activation between them (swiglu), and the gradients of all of these.

As in the rest of the package, bf16 tensors are int16 bit patterns, calls are asynchronous on the
current torch stream, and PyTorch supplies device memory only. All tensors of a call lie on the
current device (ValueError otherwise). Rows may be strided views; the values of one row are
contiguous.
"""
from __future__ import annotations

import ctypes

import torch

from .attention import _device, _ints, _stream
from .binding import MoeError, _check, _check_dev, c_int32, c_size_t, c_void_p, lib

ROWS_BF16, ROWS_E4M3 = 0, 1


class RowsC(ctypes.Structure):
    _fields_ = [("format", c_int32), ("p", c_void_p), ("stride", ctypes.c_int64), ("scale", c_void_p),
                ("scale_stride", ctypes.c_int64)]


class WeightsC(ctypes.Structure):
    _fields_ = [("q", c_void_p), ("scale", c_void_p), ("n_experts", c_int32), ("n", c_int32), ("k", c_int32)]


_FN = {}


def _fn(name: str):
    """The library's function, its argument types declared on first use."""
    f = _FN.get(name)
    if f is None:
        i32, vp, rows, weights = c_int32, c_void_p, ctypes.POINTER(RowsC), ctypes.POINTER(WeightsC)
        end = [vp, c_size_t, vp]  # workspace, its size, stream
        types = {
            "moe_expert_workspace_bytes": [i32],
            "moe_sort_tokens": [vp, i32, i32, vp, vp, vp] + end,
            "moe_dispatch": [rows, vp, i32, i32, i32, rows, i32] + end,
            "moe_combine": [rows, i32, vp, vp, i32, i32, i32, rows, rows] + end,
            "moe_combine_grad": [rows, rows, i32, vp, vp, i32, i32, i32, rows, vp] + end,
            "moe_quant_weights": [vp, i32, i32, i32, vp, vp, vp],
            "moe_gemm_e4m3": [rows, i32, weights, vp, i32, rows] + end,
            "moe_swiglu": [rows, i32, i32, vp, rows] + end,
            "moe_swiglu_grad": [rows, rows, i32, i32, vp, rows] + end,
        }[name]
        f = getattr(lib(), name)
        f.argtypes = types
        f.restype = c_size_t if name == "moe_expert_workspace_bytes" else ctypes.c_int
        _FN[name] = f
    return f


def expert_workspace_bytes(n_experts: int) -> int:
    return int(_fn("moe_expert_workspace_bytes")(n_experts))


def expert_workspace(n_experts: int, device="cuda") -> torch.Tensor:
    """A zero-filled workspace for the 8-bit expert calls; its size does not depend on the rows."""
    n = expert_workspace_bytes(n_experts)
    if n == 0:
        raise MoeError(2, "expert_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def _blocks(n: int) -> int:
    return (n + 127) // 128


class E4m3Rows:
    """Rows in 8 bits over the caller's tensors: codes q uint8 [rows, columns], scale float32
    [rows, ceil(columns / 128)]; a code c of column j stands for scale[row, j // 128] * c."""

    def __init__(self, q: torch.Tensor, scale: torch.Tensor):
        if q.dtype is not torch.uint8 or q.dim() != 2 or not q.is_cuda or (q.numel() and q.stride(1) != 1):
            raise ValueError("q must be a CUDA tensor of uint8 [rows, columns], the values of a row contiguous")
        rows, cols = q.shape
        if rows >= _MANY or cols >= _MANY:
            raise ValueError("rows and columns must be fewer than 2^31")
        if (scale.dtype is not torch.float32 or scale.shape != (rows, _blocks(cols)) or not scale.is_cuda
                or scale.get_device() != q.get_device() or (scale.shape[1] > 1 and rows and scale.stride(1) != 1)):
            raise ValueError(f"scale must be a float32 tensor [{rows}, {_blocks(cols)}] on q's device, the values of "
                             "a row contiguous")
        self.q, self.scale, self.shape = q, scale, q.shape
        # the stride of an axis of length one is never used, and torch may give any
        self._c = RowsC(ROWS_E4M3, q.data_ptr(), q.stride(0) if rows > 1 else _blocks(cols) * 128, scale.data_ptr(),
                        scale.stride(0) if rows > 1 else _blocks(cols))

    @classmethod
    def empty(cls, rows: int, cols: int, device="cuda"):
        return cls(torch.empty((rows, cols), dtype=torch.uint8, device=device),
                   torch.empty((rows, _blocks(cols)), dtype=torch.float32, device=device))

    def values(self) -> torch.Tensor:
        """What the codes stand for, in float32."""
        s = self.scale.repeat_interleave(128, 1)[:, :self.shape[1]]
        return self.q.view(torch.float8_e4m3fn).float() * s

    def get_device(self) -> int:
        return self.q.get_device()


class E4m3Weights:
    """Expert matrices in 8 bits over the caller's tensors, contiguous: codes q uint8
    [n_experts, n, k], scale float32 [n_experts, ceil(n / 128), ceil(k / 128)]."""

    def __init__(self, q: torch.Tensor, scale: torch.Tensor):
        _check_dev(q, torch.uint8, "q")
        _check_dev(scale, torch.float32, "scale")
        if q.dim() != 3 or max(q.shape) >= _MANY or scale.shape != (q.shape[0], _blocks(q.shape[1]), _blocks(q.shape[2])):
            raise ValueError("q must be [n_experts, n, k] and scale [n_experts, ceil(n / 128), ceil(k / 128)]")
        if q.get_device() != scale.get_device():
            raise ValueError("the weights' tensors must be on one device")
        self.q, self.scale, self.shape = q, scale, q.shape
        self._c = WeightsC(q.data_ptr(), scale.data_ptr(), *q.shape)

    @classmethod
    def quantise(cls, w: torch.Tensor) -> "E4m3Weights":
        """moe_quant_weights: bf16 matrices int16 [n_experts, n, k] in blocks of 128 x 128."""
        dev = _device(w, "w")
        if w.dtype is not torch.int16 or w.dim() != 3 or not w.is_contiguous() or max(w.shape) >= _MANY:
            raise ValueError("w must be a contiguous int16 tensor [n_experts, n, k]")
        E, n, k = w.shape
        q = torch.empty(w.shape, dtype=torch.uint8, device=w.device)
        scale = torch.empty((E, _blocks(n), _blocks(k)), dtype=torch.float32, device=w.device)
        _check(_fn("moe_quant_weights")(w.data_ptr(), E, n, k, q.data_ptr(), scale.data_ptr(), _stream(dev)),
               "moe_quant_weights")
        return cls(q, scale)


_I16, _I32, _F32, _U8 = torch.int16, torch.int32, torch.float32, torch.uint8
_MANY = 1 << 31  # sizes from here on do not fit the library's integers; it refuses smaller ones itself

# The checks below take as few calls into torch as they can: a call on small rows is bound by its host time.


def _bf16(t: torch.Tensor, rows: int | None, cols: int | None, name: str, dev: int) -> RowsC:
    """A view of bf16 rows; rows and cols None: any."""
    shape = t.shape
    if t.dtype is _I16 and t.get_device() == dev and len(shape) == 2:
        r, c = shape
        if (rows is None or r == rows) and (cols is None or c == cols) and r < _MANY and c < _MANY:
            stride, inner = t.stride()
            if inner == 1 or r * c == 0:
                # the stride of an axis of length one is never used, and torch may give any
                return RowsC(ROWS_BF16, t.data_ptr(), stride if r > 1 else (c + 7) // 8 * 8, None, 0)
    want = f"[{'rows' if rows is None else rows}, {'columns' if cols is None else cols}]"
    raise ValueError(f"{name} must be an int16 tensor {want} on the current CUDA device, the values of a row contiguous")


def _e4m3(r: E4m3Rows, rows: int | None, cols: int, name: str, dev: int) -> RowsC:
    if not isinstance(r, E4m3Rows) or r.get_device() != dev or rows not in (None, r.shape[0]) or r.shape[1] != cols:
        raise ValueError(f"{name} must be E4m3Rows [{'rows' if rows is None else rows}, {cols}] on the current CUDA device")
    return r._c


def _out(out, e4m3: bool, rows: int | None, cols: int, dev: int, like: torch.Tensor):
    """The output rows and their description; if none are given, `rows` new ones on the device of `like`."""
    if out is None:
        if not e4m3:
            out = torch.empty((rows, cols), dtype=_I16, device=like.device)
            return out, RowsC(ROWS_BF16, out.data_ptr(), cols if rows > 1 else (cols + 7) // 8 * 8, None, 0)
        out = E4m3Rows.empty(rows, cols, like.device)
    if isinstance(out, E4m3Rows):
        return out, _e4m3(out, rows, cols, "out", dev)
    return out, _bf16(out, rows, cols, "out", dev)


def _space(ws: torch.Tensor, dev: int) -> int:
    if ws.dtype is not _U8 or ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous uint8 tensor on the current CUDA device (expert_workspace)")
    return ws.data_ptr()


def _floats(t: torch.Tensor, shape, name: str, dev: int) -> int:
    if t.dtype is not _F32 or t.get_device() != dev or not t.is_contiguous() or t.shape != shape:
        raise ValueError(f"{name} must be a contiguous float32 tensor {list(shape)} on the current CUDA device")
    return t.data_ptr()


def _places(inv: torch.Tensor, T: int, dev: int) -> tuple[int, int]:
    """The pointer of inv [T, top_k], and top_k."""
    shape = inv.shape
    if len(shape) != 2 or shape[0] != T or shape[1] >= _MANY:
        raise ValueError(f"inv must be [{T}, top_k]")
    return _ints(inv, None, "inv", dev), shape[1]


def sort_tokens(ids: torch.Tensor, n_experts: int, ws: torch.Tensor):
    """moe_sort_tokens: ids int32 [T, top_k], negative for none. Returns offsets [n_experts + 1],
    perm [T * top_k] (place -> assignment) and inv [T, top_k] (assignment -> place), int32."""
    dev = _device(ids, "ids")
    p, n, device = _ints(ids, None, "ids", dev), ids.numel(), ids.device
    if n >= _MANY:
        raise ValueError("ids must have fewer than 2^31 entries")
    offsets = torch.empty(max(n_experts, 0) + 1, dtype=_I32, device=device)
    perm = torch.empty(n, dtype=_I32, device=device)
    inv = torch.empty_like(ids)
    _check(_fn("moe_sort_tokens")(p, n, n_experts, offsets.data_ptr(), perm.data_ptr(), inv.data_ptr(), _space(ws, dev),
                                  ws.numel(), _stream(dev)), "moe_sort_tokens")
    return offsets, perm, inv


def dispatch(x: torch.Tensor, inv: torch.Tensor | None, ws: torch.Tensor, *, e4m3: bool = False, out=None):
    """moe_dispatch: row t of x [T, d] goes to the places inv[t]; inv None: to row t. Returns the rows,
    int16 or (e4m3=True) E4m3Rows, one for each assignment; `out` gives them (of either kind). Rows without
    an assignment are left as they were: uninitialised, where the call made them."""
    dev = _device(x, "x")
    xv = _bf16(x, None, None, "x", dev)
    T, d = x.shape
    iv, k = (None, 1) if inv is None else _places(inv, T, dev)
    out, ov = _out(out, e4m3, T * k if out is None else None, d, dev, x)
    _check(_fn("moe_dispatch")(ctypes.byref(xv), iv, T, k, d, ctypes.byref(ov), out.shape[0], _space(ws, dev),
                               ws.numel(), _stream(dev)), "moe_dispatch")
    return out


def combine(ys: torch.Tensor, inv: torch.Tensor, w: torch.Tensor | None, ws: torch.Tensor, *,
            add: torch.Tensor | None = None, y: torch.Tensor | None = None) -> torch.Tensor:
    """moe_combine: y[t] = add[t] + sum_j w[t, j] * ys[inv[t, j]]; w float32 [T, top_k], None for ones
    (dispatch_grad). y may be add."""
    dev = _device(ys, "ys")
    yv = _bf16(ys, None, None, "ys", dev)
    rows, d = ys.shape
    T = inv.shape[0]
    iv, k = _places(inv, T, dev)
    av = None if add is None else _bf16(add, T, d, "add", dev)
    y, ov = _out(y, False, T, d, dev, ys)
    _check(_fn("moe_combine")(ctypes.byref(yv), rows, iv, None if w is None else _floats(w, (T, k), "w", dev), T, k, d,
                              None if av is None else ctypes.byref(av), ctypes.byref(ov), _space(ws, dev), ws.numel(),
                              _stream(dev)), "moe_combine")
    return y


def dispatch_grad(dxs: torch.Tensor, inv: torch.Tensor, ws: torch.Tensor, *, add: torch.Tensor | None = None,
                  dx: torch.Tensor | None = None) -> torch.Tensor:
    """The gradient of dispatch: dx[t] = add[t] + sum_j dxs[inv[t, j]] (moe_combine without weights)."""
    return combine(dxs, inv, None, ws, add=add, y=dx)


def combine_grad(dy: torch.Tensor, ys: torch.Tensor, inv: torch.Tensor, w: torch.Tensor, ws: torch.Tensor, *,
                 e4m3: bool = False, out=None, dw: torch.Tensor | None = None):
    """moe_combine_grad: the gradients (dys, dw) of combine's rows and weights; dys int16 or (e4m3=True)
    E4m3Rows, as many as ys; `out` gives them. The gradient of combine's `add` is dy itself."""
    dev = _device(dy, "dy")
    dv = _bf16(dy, None, None, "dy", dev)
    T, d = dy.shape
    yv, rows = _bf16(ys, None, d, "ys", dev), ys.shape[0]
    iv, k = _places(inv, T, dev)
    out, ov = _out(out, e4m3, rows, d, dev, dy)
    dw = torch.empty((T, k), dtype=torch.float32, device=dy.device) if dw is None else dw
    _check(_fn("moe_combine_grad")(ctypes.byref(dv), ctypes.byref(yv), rows, iv, _floats(w, (T, k), "w", dev), T,
                                   k, d, ctypes.byref(ov), _floats(dw, (T, k), "dw", dev), _space(ws, dev), ws.numel(),
                                   _stream(dev)), "moe_combine_grad")
    return out, dw


def gemm_e4m3(a: E4m3Rows, w: E4m3Weights, offsets: torch.Tensor | None, ws: torch.Tensor, *, transposed: bool = False,
              out: torch.Tensor | None = None) -> torch.Tensor:
    """moe_gemm_e4m3: rows offsets[e] .. offsets[e + 1] - 1 of a times expert e's matrix (int32
    [n_experts + 1] on the device; None: one expert, all rows). a has k columns and the result n;
    transposed: n columns and the result k, the products with the matrices' transposes."""
    if not isinstance(a, E4m3Rows) or not isinstance(w, E4m3Weights):
        raise ValueError("a must be E4m3Rows and w E4m3Weights")
    dev = _device(a.q, "a")
    if w.q.get_device() != dev:
        raise ValueError("w must be on the current CUDA device")
    E, n, k = w.shape
    av = _e4m3(a, None, n if transposed else k, "a", dev)
    out, ov = _out(out, False, a.shape[0], k if transposed else n, dev, a.q)
    _check(_fn("moe_gemm_e4m3")(ctypes.byref(av), a.shape[0], ctypes.byref(w._c),
                                None if offsets is None else _ints(offsets, E + 1, "offsets", dev),
                                1 if transposed else 0, ctypes.byref(ov), _space(ws, dev), ws.numel(), _stream(dev)),
           "moe_gemm_e4m3")
    return out


def _total(total: torch.Tensor | None, dev: int) -> int | None:
    return None if total is None else _ints(total, 1, "total", dev)


def swiglu(gu: torch.Tensor, ws: torch.Tensor, *, total: torch.Tensor | None = None, e4m3: bool = False, out=None):
    """moe_swiglu: silu(g) * u for rows gu = g | u [rows, 2 * inter]; total: int32 [1] on the device, the
    number of rows that count (offsets[-1:]). Returns int16 or (e4m3=True) E4m3Rows; `out` gives them."""
    dev = _device(gu, "gu")
    gv = _bf16(gu, None, None, "gu", dev)
    rows, cols = gu.shape
    inter = cols // 2
    if cols % 2:
        raise ValueError("gu must have an even number of columns")
    out, ov = _out(out, e4m3, rows, inter, dev, gu)
    _check(_fn("moe_swiglu")(ctypes.byref(gv), rows, inter, _total(total, dev), ctypes.byref(ov), _space(ws, dev),
                             ws.numel(), _stream(dev)), "moe_swiglu")
    return out


def swiglu_grad(gu: torch.Tensor, dh: torch.Tensor, ws: torch.Tensor, *, total: torch.Tensor | None = None,
                e4m3: bool = False, out=None):
    """moe_swiglu_grad: the gradient of swiglu's rows, dg | du [rows, 2 * inter], from that of its
    result, dh [rows, inter]."""
    dev = _device(gu, "gu")
    gv = _bf16(gu, None, None, "gu", dev)
    rows, cols = gu.shape
    inter = cols // 2
    if cols % 2:
        raise ValueError("gu must have an even number of columns")
    hv = _bf16(dh, rows, inter, "dh", dev)
    out, ov = _out(out, e4m3, rows, 2 * inter, dev, gu)
    _check(_fn("moe_swiglu_grad")(ctypes.byref(gv), ctypes.byref(hv), rows, inter, _total(total, dev), ctypes.byref(ov),
                                  _space(ws, dev), ws.numel(), _stream(dev)), "moe_swiglu_grad")
    return out
