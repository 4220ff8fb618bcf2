"""Which form of the product's kernel a call takes (CPU only): a GB300 has 152 SMs and runs 76 pairs of CTAs at once. The sizes
are those whose results tests/test_gpu_experts*.py check, so that a change of the choice that leaves a form untested shows."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from quantized_grouped_gemm_router_gb300 import build as B  # noqa: E402
from tests.product_forms import COLUMNS_128, COLUMNS_256, FEW_ROWS, FORM_CASES, PAIRS  # noqa: E402

SMS, N_PAIRS = 152, 76


@pytest.fixture(scope="module")
def form():
    B.build()
    import quantized_grouped_gemm_router_gb300 as m
    f = m.lib().moe_gemm_e4m3_form
    f.argtypes, f.restype = [ctypes.c_int32] * 5 + [ctypes.c_int64] + [ctypes.c_int32] * 2, ctypes.c_int32

    def get(rows, E, out, cols, transposed, pad=0, sms=SMS, pairs=N_PAIRS):
        n, k = (cols, out) if transposed else (out, cols)
        return f(rows, E, n, k, int(transposed), cols + pad, sms, pairs)
    return get


@pytest.mark.parametrize("want,counts,out,cols,pad,transposed", FORM_CASES)
def test_form_cases(form, want, counts, out, cols, pad, transposed):
    assert form(sum(counts), len(counts), out, cols, transposed, pad) == want


def test_every_form_is_covered():
    """Each form in each direction that it has, on rows on and off 128-byte lines."""
    def off(case):
        _, _, out, cols, pad, transposed = case
        return (out if transposed else cols) % 128 != 0 or (cols + pad) % 128 != 0
    seen = {(c[0], c[5], off(c)) for c in FORM_CASES}
    assert seen >= {(f, t, o) for f in (COLUMNS_128, COLUMNS_256, PAIRS) for t in (False, True) for o in (False, True)}
    assert seen >= {(FEW_ROWS, False, o) for o in (False, True)}
    assert any(c[0] == PAIRS and len(c[1]) > 1 for c in FORM_CASES)


def test_no_pairs(form):
    """A device that runs none takes single CTAs, and few experts with few rows never ask."""
    for want, counts, out, cols, pad, transposed in FORM_CASES:
        got = form(sum(counts), len(counts), out, cols, transposed, pad, pairs=0)
        assert got == want if want != PAIRS else got in (COLUMNS_128, COLUMNS_256)


def test_forms_of_the_wide_tests(form):
    """tests/test_gpu_experts.py's sizes with more items than SMs: two of the first three are pairs'."""
    for t in (False, True):
        assert [form(6001, 3, 2064, 144, t), form(5400, 1, 2064, 1296, t), form(5126, 5, 4112, 80, t)] == [COLUMNS_256, PAIRS, PAIRS]
        assert [form(5012, 40, 1040, 144, t), form(1400, 200, 400, 272, t), form(7760, 160, 272, 528, t)] == [COLUMNS_256, COLUMNS_256, COLUMNS_128]


def test_refusals(form):
    for bad in (dict(rows=0), dict(rows=1 << 26), dict(E=0), dict(E=1025), dict(out=8), dict(cols=65552), dict(pad=-256), dict(sms=0), dict(pairs=-1)):
        assert form(**{**dict(rows=5, E=2, out=128, cols=256, transposed=False), **bad}) == -1, bad
