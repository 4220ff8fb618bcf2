"""The 8-bit expert calls on a GB300 where their arguments are unusual: gates far below zero, copied handles, each form of the product's
kernel, weights of more than 2^31 codes."""
import copy
import ctypes

import pytest

torch = pytest.importorskip("torch")

from tests import expert_check as C  # noqa: E402
from tests.product_forms import FORM_CASES  # noqa: E402
from tests.test_gpu_experts import dev, guarded, make_product, m, rand, untouched, ws  # noqa: E402, F401

pytestmark = pytest.mark.gpu


def far_values():
    """g from -30 down to where no result is left, u and dh over bf16's range; only results below 2^126."""
    g, u, h = [], [], []
    for x in (-30.0, -32.0, -32.25, -46.0, -64.0, -87.0, -87.5, -88.0, -88.5, -89.0, -96.0, -104.0, -120.0, -150.0, -174.0, -175.0, -200.0,
              -250.0, -300.0, -348.0, -350.0, -1000.0, -2.0 ** 127):
        for y in (1.0, -3.0, 2.0 ** -60, 2.0 ** 40, 1.5 * 2.0 ** 100, -1.75 * 2.0 ** 126):
            for z in (1.0, -2.0 ** -30, 2.0 ** 60, 1.25 * 2.0 ** 120):
                g.append(x), u.append(y), h.append(z)
    return (torch.tensor(v, dtype=torch.float64) for v in (g, u, h))


def as_rows(x, cols):
    """Values as bf16 rows of `cols`, the last row filled up with -40."""
    assert torch.equal(x.to(torch.bfloat16).double(), x)
    n = (len(x) + cols - 1) // cols * cols
    return torch.cat([x, torch.full((n - len(x),), -40.0, dtype=torch.float64)]).view(-1, cols)


@pytest.mark.parametrize("inter", [48, 128, 528])
def test_swiglu_far_below(m, ws, inter):  # noqa: F811
    """Where s = 1 / (1 + e^-g) is no normal fp32 number, a large u or dh brings its products back into range. The bounds
    are those of expert_check without its allowance of 2^-126 in s: fp32 results below 2^-126 are off by 2^-150, and the
    rest by (|g| + 8) 2^-23 of themselves (1 + g (1 - s) is 1 + g there to 2^-46, exact in 64 bits)."""
    g, u, h = far_values()
    s = torch.sigmoid(g)
    for name, ref in (("h", g * s * u), ("du", h * g * s), ("dg", h * u * s * (1 + g * torch.sigmoid(-g)))):
        keep = ref.abs() < 2.0 ** 126
        if name == "dg":  # both halves of the gradient
            keep &= (h * g * s).abs() < 2.0 ** 126
        G, U, H = (as_rows(v[keep], inter) for v in (g, u, h))
        S = torch.sigmoid(G)
        e = (G.abs() + 8) * 2.0 ** -23
        gu = torch.cat([G, U], 1).to(torch.bfloat16)
        if name == "h":
            ref = G * S * U
            got = m.swiglu(dev(gu), ws)
            err = ref.abs() * e + 2.0 ** -149
        else:
            dg, du = H * U * S * (1 + G * torch.sigmoid(-G)), H * G * S
            if name == "du":  # dg may be out of range: its u is left out
                gu[:, inter:] = 0
                dg = torch.zeros_like(dg)
            ref = torch.cat([dg, du], 1)
            got = m.swiglu_grad(dev(gu), dev(H.to(torch.bfloat16)), ws)
            err = ref.abs() * torch.cat([e, e], 1) + 2.0 ** -149
        C.check_rows(got, ref, err, name)
        assert (ref.abs() > 2.0 ** -100).any() and (ref[ref.abs() < 2.0 ** -100].abs() > 2.0 ** -126).any()


def test_swiglu_far_below_in_8_bits(m, ws):  # noqa: F811
    g = torch.tensor([-88.0, -90.0, -100.0, -120.0]).double().repeat(2, 64)
    u = torch.full_like(g, 2.0 ** 100)
    u[1] = -1.5 * 2.0 ** 120
    h = torch.full_like(g, 2.0 ** 20)
    s = torch.sigmoid(g)
    e = (g.abs() + 8) * 2.0 ** -23
    gu = torch.cat([g, u], 1).to(torch.bfloat16)
    ref = g * s * u
    C.check_rows(m.swiglu(dev(gu), ws, e4m3=True), ref, ref.abs() * e)
    ref = torch.cat([h * u * s * (1 + g * torch.sigmoid(-g)), h * g * s], 1)
    C.check_rows(m.swiglu_grad(dev(gu), dev(h.to(torch.bfloat16)), ws, e4m3=True), ref, ref.abs() * torch.cat([e, e], 1) + 2.0 ** -149)


def test_copied_handles(m, ws):  # noqa: F811
    """A copy computes with its own memory: the original may change, and go."""
    a, w, offsets, _ = make_product(m, 5, [40, 0, 91], 272, 400, False)
    want = m.gemm_e4m3(a, w, offsets, ws)
    a2, w2 = copy.deepcopy(a), copy.deepcopy(w)
    for x in (a.q, w.q):
        x.fill_(0x7F)
    assert torch.equal(m.gemm_e4m3(a2, w2, offsets, ws), want)
    assert not torch.equal(m.gemm_e4m3(a, w, offsets, ws), want)
    out, x = copy.deepcopy(a2), dev(rand(1, 131, 400))
    m.dispatch(x, None, ws, out=out)
    assert torch.equal(m.gemm_e4m3(a2, w2, offsets, ws), want)  # what was written to a copy of it
    a.q, a.scale, w.q.data, w.scale.data = a2.q, a2.scale, w2.q, w2.scale
    del a2, w2
    assert torch.equal(m.gemm_e4m3(a, w, offsets, ws), want)


@pytest.mark.parametrize("form,counts,out,cols,pad,transposed", FORM_CASES)
def test_product_forms(m, ws, form, counts, out, cols, pad, transposed):  # noqa: F811
    """Each form of the kernel, on rows on and off 128-byte lines (on a GPU of other SMs the sizes may take other forms)."""
    n, k = (cols, out) if transposed else (out, cols)
    a, w, offsets, (ref, size) = make_product(m, out + cols, counts, n, k, transposed)
    rows = sum(counts)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    if sms == 152:
        got = m.lib().moe_gemm_e4m3_form(rows, len(counts), n, k, int(transposed), ctypes.c_int64(cols + pad), sms, sms // 2)
        assert got == form
    if pad:
        wide = torch.full((rows, cols + pad), 0x7F, dtype=torch.uint8, device="cuda")
        wide[:, :cols] = a.q
        a = m.E4m3Rows(wide[:, :cols], a.scale)
    whole, got = guarded(rows, out, 0x7FC0)
    for _ in range(2):
        m.gemm_e4m3(a, w, offsets, ws, transposed=transposed, out=got)
    C.check_product(got, ref, size, C.blocks(cols))
    assert untouched(whole, rows, out, 0x7FC0)


def test_more_weights_than_31_bits(m, ws):  # noqa: F811
    """The last of 33 experts of 8192 x 8192 lies behind 2^31 codes (and 2^32 bytes of bf16): the same bits as alone."""
    E, n = 33, 8192
    g = torch.Generator(device="cuda").manual_seed(1)
    w16 = torch.zeros(E, n, n, dtype=torch.int16, device="cuda")
    w16[-1] = (torch.randn(n, n, generator=g, device="cuda") / 90).to(torch.bfloat16).view(torch.int16)
    w = m.E4m3Weights.quantise(w16)
    one = m.E4m3Weights.quantise(w16[-1:])
    assert w.q.numel() > 2 ** 31 and torch.equal(w.q[-1:], one.q) and torch.equal(w.scale[-1:], one.scale) and one.q.any()
    assert not w.q[:-1].any()
    for rows in (1, 300):
        a = m.dispatch(torch.randn(rows, n, generator=g, device="cuda").to(torch.bfloat16).view(torch.int16), None, ws, e4m3=True)
        offsets = torch.tensor([0] * E + [rows], dtype=torch.int32, device="cuda")
        for transposed in (False, True):
            want = m.gemm_e4m3(a, one, None, ws, transposed=transposed)
            assert torch.equal(m.gemm_e4m3(a, w, offsets, ws, transposed=transposed), want) and want.any()
