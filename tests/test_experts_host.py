"""Argument checks of the 8-bit expert calls (CPU only): every call below fails validation or has
nothing to do, so nothing is launched and no pointer is followed."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from quantized_grouped_gemm_router_gb300 import build as B  # noqa: E402

A = 1 << 20  # a fake, aligned pointer
BIG = 1 << 30


@pytest.fixture(scope="module")
def m():
    B.build()
    import quantized_grouped_gemm_router_gb300 as mod
    return mod


class RowsC(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("p", ctypes.c_void_p), ("stride", ctypes.c_int64), ("scale", ctypes.c_void_p),
                ("scale_stride", ctypes.c_int64)]


class WeightsC(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("n_experts", ctypes.c_int32), ("n", ctypes.c_int32),
                ("k", ctypes.c_int32)]


@pytest.fixture(scope="module")
def fn(m):
    """The C entry points, with their argument types."""
    i32, vp, rows, weights = ctypes.c_int32, ctypes.c_void_p, ctypes.POINTER(RowsC), ctypes.POINTER(WeightsC)
    end = [vp, ctypes.c_size_t, vp]  # workspace, its size, stream
    types = {
        "moe_sort_tokens": [vp, i32, i32, vp, vp, vp] + end,
        "moe_dispatch": [rows, vp, i32, i32, i32, rows, i32] + end,
        "moe_combine": [rows, i32, vp, vp, i32, i32, i32, rows, rows] + end,
        "moe_combine_grad": [rows, rows, i32, vp, vp, i32, i32, i32, rows, vp] + end,
        "moe_quant_weights": [vp, i32, i32, i32, vp, vp, vp],
        "moe_gemm_e4m3": [rows, i32, weights, vp, i32, rows] + end,
        "moe_swiglu": [rows, i32, i32, vp, rows] + end,
        "moe_swiglu_grad": [rows, rows, i32, i32, vp, rows] + end,
    }

    def get(name):
        f = getattr(m.lib(), name)
        f.argtypes, f.restype = types[name], ctypes.c_int
        return f
    return get


def bf16(p=A, stride=64, **kw):
    return RowsC(kw.get("format", 0), p, stride, None, 0)


def e4m3(p=A, stride=64, scale=A, scale_stride=1):
    return RowsC(1, p, stride, scale, scale_stride)


def ref(x):
    return None if x is None else ctypes.byref(x)


def bad_bf16(call):
    """Rows of 64 columns that every call refuses, `call` given them."""
    assert call(None) == 1 and call(bf16(None)) == 1 and call(bf16(A + 8)) == 3
    assert call(bf16(stride=56)) == 1 and call(bf16(stride=68)) == 1 and call(bf16(stride=1 << 38)) == 1
    assert call(bf16(format=2)) == 1 and call(bf16(format=-1)) == 1


def bad_e4m3(call):
    assert call(e4m3(None)) == 1 and call(e4m3(A + 8)) == 3 and call(e4m3(stride=72)) == 1
    assert call(e4m3(scale=None)) == 1 and call(e4m3(scale=A + 2)) == 3 and call(e4m3(scale_stride=0)) == 1
    assert call(e4m3(scale_stride=1 << 38)) == 1


def bad_space(call, need):
    assert call(None, need) == 1 and call(A + 64, need) == 3 and call(A, need - 1) == 4 and call(A, 0) == 4


def test_workspace(m):
    sizes = [m.expert_workspace_bytes(E) for E in (1, 16, 256, 1024)]
    assert all(a < b for a, b in zip(sizes, sizes[1:])) and sizes[0] > 256
    for bad in (0, -1, 1025):
        assert m.expert_workspace_bytes(bad) == 0
        with pytest.raises(m.MoeError):
            m.expert_workspace(bad, device="cpu")


def test_sort_refusals(m, fn):
    need = m.expert_workspace_bytes(8)

    def call(ids=A, n=10, E=8, offsets=A, perm=A, inv=A, ws=A, size=need):
        return fn("moe_sort_tokens")(ids, n, E, offsets, perm, inv, ws, size, None)

    assert call(E=0) == 2 and call(E=1025) == 2 and call(n=-1) == 1 and call(n=1 << 26) == 2
    for name in ("ids", "offsets", "perm", "inv"):
        assert call(**{name: None}) == 1 and call(**{name: A + 2}) == 3, name
    bad_space(lambda ws, size: call(ws=ws, size=size), need)


def test_dispatch_refusals(m, fn):
    need = m.expert_workspace_bytes(1)

    def call(x=bf16(), inv=A, T=5, k=2, d=64, out=bf16(), rows=10, ws=A, size=need):
        return fn("moe_dispatch")(ref(x), inv, T, k, d, ref(out), rows, ws, size, None)

    bad_bf16(lambda r: call(x=r))
    bad_bf16(lambda r: call(out=r))
    bad_e4m3(lambda r: call(out=r))
    assert call(x=e4m3()) == 1
    assert call(T=-1) == 1 and call(rows=-1) == 1 and call(inv=A + 1) == 3
    assert call(inv=None) == 1 and call(inv=None, k=1, rows=4) == 1           # no places: a row each
    for kw in (dict(k=0), dict(k=17), dict(d=0), dict(d=24), dict(d=65552), dict(T=1 << 26), dict(T=BIG, k=16),
               dict(rows=1 << 26)):
        assert call(**kw) == 2, kw
    bad_space(lambda ws, size: call(ws=ws, size=size), need)
    assert call(T=0, x=None, out=None, inv=None, k=1) == 0


def test_combine_refusals(m, fn):
    need = m.expert_workspace_bytes(1)

    def call(ys=bf16(), rows=10, inv=A, w=A, T=5, k=2, d=64, add=None, y=bf16(), ws=A, size=need):
        return fn("moe_combine")(ref(ys), rows, inv, w, T, k, d, ref(add), ref(y), ws, size, None)

    def grad(dy=bf16(), ys=bf16(), rows=10, inv=A, w=A, T=5, k=2, d=64, dys=bf16(), dw=A, ws=A, size=need):
        return fn("moe_combine_grad")(ref(dy), ref(ys), rows, inv, w, T, k, d, ref(dys), dw, ws, size, None)

    bad_bf16(lambda r: call(ys=r))
    bad_bf16(lambda r: call(y=r))
    bad_bf16(lambda r: call(add=r) if r is not None else 1)
    for name in ("dy", "ys", "dys"):
        bad_bf16(lambda r: grad(**{name: r}))
    bad_e4m3(lambda r: grad(dys=r))
    assert call(ys=e4m3()) == 1 and call(y=e4m3()) == 1 and call(add=e4m3()) == 1
    assert grad(dy=e4m3()) == 1 and grad(ys=e4m3()) == 1
    assert call(w=A + 2) == 3 and grad(w=None) == 1 and grad(dw=None) == 1 and grad(dw=A + 1) == 3
    for f in (call, grad):
        assert f(T=-1) == 1 and f(rows=-1) == 1 and f(inv=None) == 1 and f(inv=A + 2) == 3
        for kw in (dict(k=0), dict(k=17), dict(d=8), dict(d=40), dict(T=1 << 26), dict(rows=1 << 26)):
            assert f(**kw) == 2, kw
        bad_space(lambda ws, size: f(ws=ws, size=size), need)
        assert f(T=0, ys=None, inv=None) == 0


def test_weights_refusals(m, fn):
    def call(w=A, E=2, n=64, k=64, q=A, scale=A):
        return fn("moe_quant_weights")(w, E, n, k, q, scale, None)

    assert call(E=0) == 2 and call(E=1025) == 2 and call(n=8) == 2 and call(k=100) == 2 and call(k=1 << 17) == 2
    for name in ("w", "q", "scale"):
        assert call(**{name: None}) == 1
    assert call(w=A + 8) == 3 and call(q=A + 8) == 3 and call(scale=A + 2) == 3


def test_product_refusals(m, fn):
    need = m.expert_workspace_bytes(4)

    def call(a=e4m3(), rows=9, w=None, offsets=A, transposed=0, out=bf16(), ws=A, size=need, **kw):
        c = dict(q=A, scale=A, n_experts=4, n=64, k=64)
        c.update(kw)
        return fn("moe_gemm_e4m3")(ref(a), rows, ref(w or WeightsC(*c.values())), offsets, transposed, ref(out), ws,
                                   size, None)

    bad_e4m3(lambda r: call(a=r))
    bad_bf16(lambda r: call(out=r))
    assert call(a=bf16()) == 1 and call(a=None) == 1 and call(out=e4m3()) == 1
    assert fn("moe_gemm_e4m3")(ref(e4m3()), 9, None, A, 0, ref(bf16()), A, need, None) == 1
    assert call(offsets=None) == 1 and call(offsets=A + 2) == 3               # four experts need offsets
    assert call(q=None) == 1 and call(q=A + 8) == 3 and call(scale=None) == 1 and call(scale=A + 1) == 3
    for kw in (dict(n_experts=0), dict(n_experts=1025), dict(n=72), dict(k=8), dict(rows=1 << 26)):
        assert call(**kw) == 2, kw
    assert call(rows=-1) == 1 and call(rows=0, a=None, out=None) == 0
    # the columns follow the direction
    assert call(k=80) == 1 and call(n=80, transposed=1) == 1
    assert call(n=80) == 1 and call(k=80, transposed=1) == 1
    bad_space(lambda ws, size: call(ws=ws, size=size), need)


def test_swiglu_refusals(m, fn):
    need = m.expert_workspace_bytes(1)

    def call(gu=bf16(stride=128), rows=5, inter=64, total=None, h=bf16(), ws=A, size=need):
        return fn("moe_swiglu")(ref(gu), rows, inter, total, ref(h), ws, size, None)

    def grad(gu=bf16(stride=128), dh=bf16(), rows=5, inter=64, total=None, dgu=bf16(stride=128), ws=A, size=need):
        return fn("moe_swiglu_grad")(ref(gu), ref(dh), rows, inter, total, ref(dgu), ws, size, None)

    bad_bf16(lambda r: call(h=r))
    bad_e4m3(lambda r: call(h=r))
    bad_bf16(lambda r: grad(dh=r))
    for f in (call, grad):
        assert f(gu=bf16(stride=120)) == 1 and f(gu=None) == 1 and f(gu=e4m3(stride=128)) == 1
        assert f(rows=-1) == 1 and f(rows=1 << 26) == 2 and f(inter=8) == 2 and f(inter=32784) == 2
        assert f(total=A + 2) == 3 and f(rows=0, gu=None) == 0
        bad_space(lambda ws, size: f(ws=ws, size=size), need)
    assert grad(dgu=bf16(stride=120)) == 1 and grad(dgu=e4m3(stride=128, scale_stride=0)) == 1 and grad(dh=e4m3()) == 1


class Placed(torch.Tensor):
    """A host tensor that says it lies on CUDA device `place`."""
    place = 0
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.place


def place(t, dev):
    t = t.as_subclass(Placed)
    t.place = dev
    return t


def calls(m):
    """(name, call, its tensors). Every workspace is too small, so that the library refuses what reaches it."""
    i16, i32, u8, f32 = torch.int16, torch.int32, torch.uint8, torch.float32

    def z(*shape, dtype=i16):
        return torch.zeros(*shape, dtype=dtype)

    ws, inv, w = z(16, dtype=u8), z(3, 2, dtype=i32), z(3, 2, dtype=f32)
    rows = lambda n: dict(q=z(n, 32, dtype=u8), s=z(n, 1, dtype=f32))  # noqa: E731
    e = lambda t: m.E4m3Rows(t["q"], t["s"])  # noqa: E731
    wt = dict(wq=z(2, 32, 32, dtype=u8), wsc=z(2, 1, 1, dtype=f32))
    return [
        ("sort", lambda t: m.sort_tokens(t["ids"], 4, t["ws"]), dict(ids=z(3, 2, dtype=i32), ws=ws)),
        ("dispatch", lambda t: m.dispatch(t["x"], t["inv"], t["ws"], out=t["out"]), dict(x=z(3, 32), inv=inv, ws=ws, out=z(6, 32))),
        ("dispatch", lambda t: m.dispatch(t["x"], t["inv"], t["ws"], out=e(t)), dict(x=z(3, 32), inv=inv, ws=ws, **rows(6))),
        ("combine", lambda t: m.combine(t["ys"], t["inv"], t["w"], t["ws"], add=t["add"], y=t["y"]),
         dict(ys=z(6, 32), inv=inv, w=w, ws=ws, add=z(3, 32), y=z(3, 32))),
        ("dispatch_grad", lambda t: m.dispatch_grad(t["ys"], t["inv"], t["ws"], add=t["add"], dx=t["y"]),
         dict(ys=z(6, 32), inv=inv, ws=ws, add=z(3, 32), y=z(3, 32))),
        ("combine_grad", lambda t: m.combine_grad(t["dy"], t["ys"], t["inv"], t["w"], t["ws"], out=t["out"], dw=t["dw"]),
         dict(dy=z(3, 32), ys=z(6, 32), inv=inv, w=w, ws=ws, out=z(6, 32), dw=w.clone())),
        ("gemm", lambda t: m.gemm_e4m3(e(t), m.E4m3Weights(t["wq"], t["wsc"]), t["offsets"], t["ws"], out=t["out"]),
         dict(offsets=z(3, dtype=i32), ws=ws, out=z(6, 32), **rows(6), **wt)),
        ("swiglu", lambda t: m.swiglu(t["gu"], t["ws"], total=t["total"], out=t["out"]),
         dict(gu=z(3, 64), ws=ws, total=z(1, dtype=i32), out=z(3, 32))),
        ("swiglu_grad", lambda t: m.swiglu_grad(t["gu"], t["dh"], t["ws"], total=t["total"], out=t["out"]),
         dict(gu=z(3, 64), dh=z(3, 32), ws=ws, total=z(1, dtype=i32), out=z(3, 64))),
    ]


@pytest.fixture
def on_device(monkeypatch):
    """Sets the device that torch says is current."""
    at = {}
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: at["device"], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    made, like = torch.empty, torch.empty_like
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **kw: place(made(*a, **kw), at["device"]))
    monkeypatch.setattr(torch, "empty_like", lambda t: place(like(t.as_subclass(torch.Tensor)), at["device"]))

    def set_device(dev):
        at["device"] = dev
    return set_device


def reaches(m, call, tensors):
    """The binding accepts the call: the library refuses its workspace, which is too small or not aligned."""
    with pytest.raises(m.MoeError) as e:
        call(tensors)
    return e.value.code in (3, 4)


def test_binding_refuses_other_devices(m, on_device):
    """Every tensor of a call lies on the current device; else nothing reaches the library."""
    for name, call, tensors in calls(m):
        for current in (0, 1):
            on_device(current)
            assert reaches(m, call, {n: place(t, current) for n, t in tensors.items()}), name
            for odd in tensors:
                with pytest.raises(ValueError):
                    call({n: place(t, 1 - current if n == odd else current) for n, t in tensors.items()})
            with pytest.raises(ValueError):
                call({n: place(t, 1 - current) for n, t in tensors.items()})


def test_binding_refuses_wrong_tensors(m, on_device):
    """Types, shapes and layouts that the library could not tell."""
    on_device(0)
    for name, call, tensors in calls(m):
        for n, t in tensors.items():
            wrong = [t.to(torch.float64), "rows", 3]
            if n not in ("ids", "offsets", "total"):  # these count, whatever their axes
                wrong += [t[None]]
            if t.dim() == 2 and n not in ("x", "gu", "ids") and (name, n) not in (("dispatch", "out"), ("combine", "ys"),
                                                                                  ("dispatch_grad", "ys")):
                wrong += [torch.zeros(t.shape[0] + 1, t.shape[1], dtype=t.dtype)]
            if t.dim() == 2 and t.shape[1] > 1:
                wrong += [torch.zeros(t.shape[1], t.shape[0], dtype=t.dtype).t()]
            if n in ("offsets", "total"):
                wrong += [torch.zeros(t.numel() + 1, dtype=t.dtype)]
            for x in wrong:
                bad = {k: place(x if k == n else v, 0) if isinstance(x if k == n else v, torch.Tensor) else x
                       for k, v in tensors.items()}
                with pytest.raises(ValueError):
                    call(bad)
        for n in ("inv", "ws", "ids", "gu", "dh", "dy", "ys", "x"):  # what has no default
            if n in tensors:
                if name == "dispatch" and n == "inv":
                    continue  # no places: a row each
                with pytest.raises(ValueError):
                    call({k: None if k == n else place(v, 0) for k, v in tensors.items()})


def test_binding_makes_outputs(m, on_device):
    """Outputs that are not given are made, of the right kind, before the library is called."""
    on_device(0)
    p = lambda *shape, dtype=torch.int16: place(torch.zeros(*shape, dtype=dtype), 0)  # noqa: E731
    ws, inv, w = p(16, dtype=torch.uint8), p(3, 2, dtype=torch.int32), p(3, 2, dtype=torch.float32)
    for e in (False, True):
        for call in (lambda: m.dispatch(p(3, 32), inv, ws, e4m3=e), lambda: m.dispatch(p(3, 32), None, ws, e4m3=e),
                     lambda: m.combine_grad(p(3, 32), p(6, 32), inv, w, ws, e4m3=e), lambda: m.swiglu(p(3, 64), ws, e4m3=e),
                     lambda: m.swiglu_grad(p(3, 64), p(3, 32), ws, e4m3=e)):
            assert reaches(m, lambda _: call(), None)
    assert reaches(m, lambda _: m.combine(p(6, 32), inv, None, ws), None)
    with pytest.raises(m.MoeError):  # k = 8 is not a multiple of 16
        m.E4m3Weights.quantise(p(1, 16, 8))
    for n_experts in (-1, 1 << 31, 1 << 40):
        with pytest.raises(m.MoeError):
            m.sort_tokens(inv, n_experts, ws)


def test_binding_refuses_host_tensors(m):
    x, inv, ws = torch.zeros(3, 32, dtype=torch.int16), torch.zeros(3, 2, dtype=torch.int32), torch.zeros(256, dtype=torch.uint8)
    for call in (lambda: m.sort_tokens(inv, 4, ws), lambda: m.dispatch(x, inv, ws), lambda: m.combine(x, inv, None, ws),
                 lambda: m.swiglu(x, ws), lambda: m.swiglu_grad(x, x, ws), lambda: m.combine_grad(x, x, inv, None, ws),
                 lambda: m.E4m3Rows(torch.zeros(3, 32, dtype=torch.uint8), torch.zeros(3, 1)),
                 lambda: m.E4m3Weights(torch.zeros(1, 32, 32, dtype=torch.uint8), torch.zeros(1, 1, 1)),
                 lambda: m.E4m3Weights.quantise(torch.zeros(1, 32, 32, dtype=torch.int16)),
                 lambda: m.gemm_e4m3(x, x, None, ws), lambda: m.E4m3Rows(x, x), lambda: m.E4m3Weights(None, None)):
        with pytest.raises(ValueError):
            call()
