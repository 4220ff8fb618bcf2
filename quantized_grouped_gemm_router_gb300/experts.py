"""Binding of the 8-bit expert calls of libmoe_gb300.so: tokens sorted by expert (sort_tokens, dispatch) and
brought back (combine), grouped products of e4m3 rows and weights (gemm_e4m3), the activation between them
(swiglu), and the gradients of all of these.

As in the rest of the package, bf16 tensors are int16 bit patterns, calls are asynchronous on the
current torch stream, and PyTorch supplies device memory only. All tensors of a call lie on the
current device (ValueError otherwise). Rows may be strided views; the values of one row are
contiguous. Outputs that are not given are made.

The arguments' checks and the calls themselves are in C (csrc/py_experts.c, built beside the library as the module
_experts): a call on a few rows is bound by its host time.
"""
from __future__ import annotations

import importlib

import torch

from .binding import MoeError, lib


class _Unloaded:
    """Stands for the module until its first use."""

    def __getattr__(self, name):
        global _native
        lib()  # says what to do where nothing is built
        try:
            module = importlib.import_module("._experts", __package__)
        except ModuleNotFoundError as e:
            raise ImportError("the 8-bit expert calls are not built: build() needs a C compiler and Python's headers for them") from e
        _native = module
        _native.setup(MoeError, E4m3Rows, E4m3Weights)
        return getattr(_native, name)


_native = _Unloaded()


def expert_workspace_bytes(n_experts: int) -> int:
    return _native.workspace_bytes(n_experts)


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
    [rows, ceil(columns / 128)]; a code c of column j stands for scale[row, j // 128] * c.

    Every call reads the two tensors, and checks them, as they are then: others may be put in their place, and a copy
    of the object (copy.deepcopy, pickle) has tensors of its own."""

    def __init__(self, q: torch.Tensor, scale: torch.Tensor):
        _native.check_rows(q, scale)
        self.q, self.scale = q, scale

    @property
    def shape(self) -> torch.Size:
        return self.q.shape

    @classmethod
    def empty(cls, rows: int, cols: int, device="cuda"):
        return cls(torch.empty((rows, cols), dtype=torch.uint8, device=device),
                   torch.empty((rows, _blocks(cols)), dtype=torch.float32, device=device))

    def values(self) -> torch.Tensor:
        """What the codes stand for, in float32."""
        s = self.scale.repeat_interleave(128, 1)[:, :self.shape[1]]
        return self.q.view(torch.float8_e4m3fn).float() * s


class E4m3Weights:
    """Expert matrices in 8 bits over the caller's tensors, contiguous: codes q uint8
    [n_experts, n, k], scale float32 [n_experts, ceil(n / 128), ceil(k / 128)]. Read at every call, as E4m3Rows."""

    def __init__(self, q: torch.Tensor, scale: torch.Tensor):
        _native.check_weights(q, scale)
        self.q, self.scale = q, scale

    @property
    def shape(self) -> torch.Size:
        return self.q.shape

    @classmethod
    def quantise(cls, w: torch.Tensor) -> "E4m3Weights":
        """moe_quant_weights: bf16 matrices int16 [n_experts, n, k] in blocks of 128 x 128."""
        if w.dim() != 3:
            raise ValueError("w must be a contiguous int16 tensor [n_experts, n, k]")
        E, n, k = w.shape
        q = torch.empty(w.shape, dtype=torch.uint8, device=w.device)
        scale = torch.empty((E, _blocks(n), _blocks(k)), dtype=torch.float32, device=w.device)
        _native.quant_weights(w, q, scale)
        return cls(q, scale)


def sort_tokens(ids: torch.Tensor, n_experts: int, ws: torch.Tensor):
    """moe_sort_tokens: ids int32 [T, top_k], negative for none. Returns offsets [n_experts + 1],
    perm [T * top_k] (place -> assignment) and inv [T, top_k] (assignment -> place), int32."""
    return _native.sort_tokens(ids, n_experts, ws)


def dispatch(x: torch.Tensor, inv: torch.Tensor | None, ws: torch.Tensor, *, e4m3: bool = False, out=None):
    """moe_dispatch: row t of x [T, d] goes to the places inv[t]; inv None: to row t. Returns the rows,
    int16 or (e4m3=True) E4m3Rows, one for each assignment; `out` gives them (of either kind). Rows without
    an assignment are left as they were: uninitialised, where the call made them."""
    return _native.dispatch(x, inv, ws, e4m3, out)


def combine(ys: torch.Tensor, inv: torch.Tensor, w: torch.Tensor | None, ws: torch.Tensor, *,
            add: torch.Tensor | None = None, y: torch.Tensor | None = None) -> torch.Tensor:
    """moe_combine: y[t] = add[t] + sum_j w[t, j] * ys[inv[t, j]]; w float32 [T, top_k], None for ones
    (dispatch_grad). y may be add."""
    return _native.combine(ys, inv, w, ws, add, y)


def dispatch_grad(dxs: torch.Tensor, inv: torch.Tensor, ws: torch.Tensor, *, add: torch.Tensor | None = None,
                  dx: torch.Tensor | None = None) -> torch.Tensor:
    """The gradient of dispatch: dx[t] = add[t] + sum_j dxs[inv[t, j]] (moe_combine without weights)."""
    return _native.combine(dxs, inv, None, ws, add, dx)


def combine_grad(dy: torch.Tensor, ys: torch.Tensor, inv: torch.Tensor, w: torch.Tensor, ws: torch.Tensor, *,
                 e4m3: bool = False, out=None, dw: torch.Tensor | None = None):
    """moe_combine_grad: the gradients (dys, dw) of combine's rows and weights; dys int16 or (e4m3=True)
    E4m3Rows, as many as ys; `out` gives them. The gradient of combine's `add` is dy itself."""
    return _native.combine_grad(dy, ys, inv, w, ws, e4m3, out, dw)


def gemm_e4m3(a: E4m3Rows, w: E4m3Weights, offsets: torch.Tensor | None, ws: torch.Tensor, *, transposed: bool = False,
              out: torch.Tensor | None = None) -> torch.Tensor:
    """moe_gemm_e4m3: rows offsets[e] .. offsets[e + 1] - 1 of a times expert e's matrix (int32
    [n_experts + 1] on the device; None: one expert, all rows). a has k columns and the result n;
    transposed: n columns and the result k, the products with the matrices' transposes."""
    return _native.gemm_e4m3(a, w, offsets, ws, transposed, out)


def swiglu(gu: torch.Tensor, ws: torch.Tensor, *, total: torch.Tensor | None = None, e4m3: bool = False, out=None):
    """moe_swiglu: silu(g) * u for rows gu = g | u [rows, 2 * inter]; total: int32 [1] on the device, the
    number of rows that count (offsets[-1:]). Returns int16 or (e4m3=True) E4m3Rows; `out` gives them."""
    return _native.swiglu(gu, ws, total, e4m3, out)


def swiglu_grad(gu: torch.Tensor, dh: torch.Tensor, ws: torch.Tensor, *, total: torch.Tensor | None = None,
                e4m3: bool = False, out=None):
    """moe_swiglu_grad: the gradient of swiglu's rows, dg | du [rows, 2 * inter], from that of its
    result, dh [rows, inter]."""
    return _native.swiglu_grad(gu, dh, ws, total, e4m3, out)
