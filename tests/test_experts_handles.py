"""Which memory the 8-bit expert calls hand to the library, where E4m3Rows and E4m3Weights were copied, pickled, or given
other tensors (CPU only): the binding is compiled against a stand-in library that notes its arguments and launches nothing."""
import copy
import ctypes
import importlib.util
import io
import os
import pickle
import shutil
import subprocess
import sysconfig

import pytest

torch = pytest.importorskip("torch")

from quantized_grouped_gemm_router_gb300 import build as B  # noqa: E402
from tests.test_experts_host import Placed, on_device  # noqa: E402, F401

STAND_IN = r"""
#include "moe_gb300.h"
moe_rows noted_rows[3];   /* the call's rows, its weights and its sizes */
moe_e4m3_weights noted_weights;
int32_t noted_sizes[2];
size_t moe_expert_workspace_bytes(int32_t n) { return 256; }
int moe_sort_tokens(const int32_t* a, int32_t b, int32_t c, int32_t* d, int32_t* e, int32_t* f, void* g, size_t h, moe_stream_t i) { return 0; }
int moe_dispatch(const moe_rows* x, const int32_t* inv, int32_t T, int32_t k, int32_t d, const moe_rows* out, int32_t rows, void* w, size_t n,
                 moe_stream_t s) {
  noted_rows[0] = *x, noted_rows[1] = *out, noted_sizes[0] = rows, noted_sizes[1] = d;
  return 0;
}
int moe_combine(const moe_rows* a, int32_t b, const int32_t* c, const float* d, int32_t e, int32_t f, int32_t g, const moe_rows* h,
                const moe_rows* i, void* j, size_t k, moe_stream_t l) { return 0; }
int moe_combine_grad(const moe_rows* dy, const moe_rows* ys, int32_t rows, const int32_t* inv, const float* w, int32_t T, int32_t k, int32_t d,
                     const moe_rows* dys, float* dw, void* ws, size_t n, moe_stream_t s) {
  noted_rows[1] = *dys;
  return 0;
}
int moe_quant_weights(const uint16_t* a, int32_t b, int32_t c, int32_t d, uint8_t* e, float* f, moe_stream_t g) { return 0; }
int moe_gemm_e4m3(const moe_rows* a, int32_t rows, const moe_e4m3_weights* w, const int32_t* o, int32_t t, const moe_rows* out, void* ws, size_t n,
                  moe_stream_t s) {
  noted_rows[0] = *a, noted_rows[1] = *out, noted_weights = *w, noted_sizes[0] = rows;
  return 0;
}
int moe_swiglu(const moe_rows* gu, int32_t rows, int32_t inter, const int32_t* total, const moe_rows* h, void* ws, size_t n, moe_stream_t s) {
  noted_rows[1] = *h;
  return 0;
}
int moe_swiglu_grad(const moe_rows* gu, const moe_rows* dh, int32_t rows, int32_t inter, const int32_t* total, const moe_rows* dgu, void* ws,
                    size_t n, moe_stream_t s) {
  noted_rows[1] = *dgu;
  return 0;
}
"""


class RowsC(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("p", ctypes.c_void_p), ("stride", ctypes.c_int64), ("scale", ctypes.c_void_p),
                ("scale_stride", ctypes.c_int64)]


class WeightsC(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("n_experts", ctypes.c_int32), ("n", ctypes.c_int32),
                ("k", ctypes.c_int32)]


@pytest.fixture(scope="module")
def stand_in(tmp_path_factory):
    """The binding's module on the stand-in library, as (module, library)."""
    headers, cc = sysconfig.get_paths()["include"], shutil.which("cc") or shutil.which("gcc")
    if not cc or not os.path.exists(os.path.join(headers, "Python.h")):
        pytest.skip("needs a C compiler and Python's headers")
    B.build()
    at = tmp_path_factory.mktemp("stand_in")
    (at / "library.c").write_text(STAND_IN)
    path = str(at / ("_experts" + sysconfig.get_config_var("EXT_SUFFIX")))
    subprocess.run([cc, "-O1", "-shared", "-fPIC", f"-I{headers}", f"-I{B.INCLUDE}", B.MODULE_SOURCE, str(at / "library.c"), "-o", path], check=True)
    spec = importlib.util.spec_from_file_location("_experts", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module, ctypes.CDLL(path)


@pytest.fixture
def m(stand_in, on_device, monkeypatch):  # noqa: F811
    import quantized_grouped_gemm_router_gb300 as mod
    from quantized_grouped_gemm_router_gb300 import experts
    stand_in[0].setup(mod.MoeError, mod.E4m3Rows, mod.E4m3Weights)
    monkeypatch.setattr(experts, "_native", stand_in[0])
    on_device(0)
    return mod


class Here(Placed):
    """A host tensor that says it lies on CUDA device 0, and so do its copies."""

    def __deepcopy__(self, memo):
        return here(copy.deepcopy(self.as_subclass(torch.Tensor), memo))


def here(t):
    return t.as_subclass(Here)


def noted(stand_in, i):
    return (RowsC * 3).in_dll(stand_in[1], "noted_rows")[i]


def z(*shape, dtype=torch.int16):
    return here(torch.zeros(*shape, dtype=dtype))


def rows(m, n=6, cols=32):
    return m.E4m3Rows(z(n, cols, dtype=torch.uint8), z(n, (cols + 127) // 128, dtype=torch.float32))


def weights(m, n=48, k=32):
    return m.E4m3Weights(z(2, n, k, dtype=torch.uint8), z(2, (n + 127) // 128, (k + 127) // 128, dtype=torch.float32))


def check(m, stand_in, r, w):
    """A product from r, and rows written to r: the addresses, strides and sizes are those of the objects' tensors now."""
    ws, n = z(16, dtype=torch.uint8), r.q.shape[0]

    def same(c):
        assert (c.p, c.scale) == (r.q.data_ptr(), r.scale.data_ptr())
        assert n < 2 or (c.stride, c.scale_stride) == (r.q.stride(0), r.scale.stride(0))

    m.gemm_e4m3(r, w, z(3, dtype=torch.int32), ws)
    same(noted(stand_in, 0))
    v = WeightsC.in_dll(stand_in[1], "noted_weights")
    assert (v.q, v.scale, v.n_experts, v.n, v.k) == (w.q.data_ptr(), w.scale.data_ptr(), *w.q.shape)
    assert r.shape == r.q.shape and w.shape == w.q.shape
    cols = r.q.shape[1]
    for call in (lambda: m.dispatch(z(n, cols), None, ws, out=r),
                 lambda: m.combine_grad(z(n, cols), z(n, cols), z(n, 1, dtype=torch.int32), z(n, 1, dtype=torch.float32), ws, out=r),
                 lambda: m.swiglu(z(n, 2 * cols), ws, out=r), lambda: m.swiglu_grad(z(n, cols), z(n, cols // 2), ws, out=r)):
        call()
        same(noted(stand_in, 1))


def pickled(x):
    return pickle.loads(pickle.dumps(x))


def saved(x):
    f = io.BytesIO()
    torch.save(x, f)
    f.seek(0)
    return torch.load(f, weights_only=False)


def test_as_made(m, stand_in):
    check(m, stand_in, rows(m), weights(m))


@pytest.mark.parametrize("again", [copy.deepcopy, pickled, saved], ids=["deepcopy", "pickle", "save"])
def test_copies_own_their_memory(m, stand_in, again):
    r, w = rows(m), weights(m)
    r2, w2 = again(r), again(w)
    for old, new in ((r, r2), (w, w2)):
        assert old.q.data_ptr() != new.q.data_ptr() and old.scale.data_ptr() != new.scale.data_ptr()
    del old, new, r, w
    check(m, stand_in, r2, w2)


def test_shallow_copies_share(m, stand_in):
    r, w = rows(m), weights(m)
    r2, w2 = copy.copy(r), copy.copy(w)
    assert r2.q is r.q and w2.scale is w.scale
    check(m, stand_in, r2, w2)


def test_a_model_is_copied(m, stand_in):
    """As a second replica or a moving average of a layer is made."""
    class Layer(torch.nn.Module):
        def __init__(self):
            super().__init__()
            self.down = weights(m)
    a = Layer()
    b = copy.deepcopy(a)
    assert b.down.q.data_ptr() != a.down.q.data_ptr()
    check(m, stand_in, rows(m), b.down)


def test_other_tensors(m, stand_in):
    """q and scale may be exchanged, or made to look elsewhere."""
    r, w = rows(m), weights(m)
    r.q, r.scale, w.q, w.scale = rows(m).q, rows(m).scale, weights(m).q, weights(m).scale
    check(m, stand_in, r, w)
    r, w = rows(m), weights(m)
    for x in (r.q, r.scale, w.q, w.scale):
        x.data = torch.zeros(x.shape, dtype=x.dtype)
    check(m, stand_in, r, w)
    r, w = rows(m), weights(m)
    for x in (r.q, r.scale, w.q, w.scale):
        x.set_(torch.zeros(x.shape, dtype=x.dtype))
    check(m, stand_in, r, w)
    r = rows(m)
    for x in (r.q, r.scale):
        x.resize_(4096, x.shape[1])
    check(m, stand_in, r, w)
    r.q, r.scale = z(9, 64, dtype=torch.uint8)[:, 16:48], z(9, 3, dtype=torch.float32)[:, 1:2]  # strided, with other rows
    check(m, stand_in, r, w)


def test_unfit_tensors_are_refused(m, stand_in):
    """What the constructor refuses a call refuses, too, and the library is not reached."""
    ws, off = z(16, dtype=torch.uint8), z(3, dtype=torch.int32)
    elsewhere = z(6, 32, dtype=torch.uint8)
    elsewhere.place = 1
    bad_rows = dict(q=[z(6, 32), z(6, 32, 1, dtype=torch.uint8), z(32, 6, dtype=torch.uint8).t(), torch.zeros(6, 32, dtype=torch.uint8),
                       elsewhere, None, 3],
                    scale=[z(5, 1, dtype=torch.float32), z(6, 2, dtype=torch.float32), z(6, 1), torch.zeros(6, 1), None])
    bad_weights = dict(q=[z(2, 48, 32), z(48, 32, dtype=torch.uint8), z(2, 32, 48, dtype=torch.uint8).transpose(1, 2),
                          torch.zeros(2, 48, 32, dtype=torch.uint8), None],
                       scale=[z(2, 1, 2, dtype=torch.float32), z(1, 1, 1, dtype=torch.float32), z(2, 1, 1), None])
    for name, values in bad_rows.items():
        for x in values:
            r = rows(m)
            setattr(r, name, x)
            for call in (lambda: m.gemm_e4m3(r, weights(m), off, ws), lambda: m.dispatch(z(6, 32), None, ws, out=r)):
                noted(stand_in, 0).p = None
                with pytest.raises(ValueError):
                    call()
                assert noted(stand_in, 0).p is None
    for name, values in bad_weights.items():
        for x in values:
            w = weights(m)
            setattr(w, name, x)
            noted(stand_in, 0).p = None
            with pytest.raises(ValueError):
                m.gemm_e4m3(rows(m), w, off, ws)
            assert noted(stand_in, 0).p is None
    r, w = rows(m), weights(m)
    del r.q, w.scale
    with pytest.raises(ValueError):
        m.gemm_e4m3(r, weights(m), off, ws)
    with pytest.raises(ValueError):
        m.gemm_e4m3(rows(m), w, off, ws)


class Undecided:
    """Neither true nor false, as an array of several values is."""

    def __bool__(self):
        raise ValueError("truth value of several values")


def test_an_undecided_format(m, stand_in):
    """What cannot say whether it is true is an error, not `False`."""
    ws = z(16, dtype=torch.uint8)
    inv, w = z(6, 1, dtype=torch.int32), z(6, 1, dtype=torch.float32)
    for call in (lambda e: m.dispatch(z(6, 32), None, ws, e4m3=e), lambda e: m.swiglu(z(6, 64), ws, e4m3=e),
                 lambda e: m.swiglu_grad(z(6, 64), z(6, 32), ws, e4m3=e), lambda e: m.combine_grad(z(6, 32), z(6, 32), inv, w, ws, e4m3=e)):
        with pytest.raises(ValueError, match="truth value"):
            call(Undecided())
        call(True), call(False)
