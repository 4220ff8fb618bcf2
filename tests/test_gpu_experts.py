"""The 8-bit expert calls on a GB300 against plain 64-bit arithmetic (tests/expert_check.py)."""
import pytest

torch = pytest.importorskip("torch")

from tests import expert_check as C  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    from quantized_grouped_gemm_router_gb300 import build as B
    B.build()
    import quantized_grouped_gemm_router_gb300 as mod
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return mod


@pytest.fixture(scope="module")
def ws(m):
    w = m.expert_workspace(1024)
    yield w
    assert m.read_device_status(w) == 0  # no test below leaves an unread error


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rand(seed, *shape, gain=1.0):
    """bf16 normal values on the host."""
    return (torch.randn(*shape, generator=gen(seed)) * gain).to(torch.bfloat16)


def dev(x):
    """To the device; bf16 as bits."""
    return (x.view(torch.int16) if x.dtype == torch.bfloat16 else x).cuda()


def some_ids(seed, T, k, E, absent=0.1):
    g = gen(seed)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]) if T else torch.zeros(0, k)
    ids = ids.to(torch.int32)
    ids[torch.rand(ids.shape, generator=g) < absent] = -1
    return ids


def guarded(rows, cols, fill):
    """Rows inside a wider buffer, as (whole, view): what lies around them has to stay."""
    whole = torch.full((rows + 2, cols + 32), fill, dtype=torch.int16 if fill == 0x7FC0 else torch.uint8, device="cuda")
    return whole, whole[1:rows + 1, 16:16 + cols]


def untouched(whole, rows, cols, fill):
    whole = whole.clone()
    whole[1:rows + 1, 16:16 + cols] = fill
    return bool((whole == fill).all())


def guarded_e4m3(m, rows, cols):
    whole, q = guarded(rows, cols, 0x55)
    ws_ = torch.full((rows + 2, C.blocks(cols) + 5), -7.0, device="cuda")
    return whole, ws_, m.E4m3Rows(q, ws_[1:rows + 1, 2:2 + C.blocks(cols)])


def untouched_e4m3(whole, ws_, rows, cols):
    s = ws_.clone()
    s[1:rows + 1, 2:2 + C.blocks(cols)] = -7.0
    return untouched(whole, rows, cols, 0x55) and bool((s == -7.0).all())


# ------------------------------------------------------------------------------------ sorting
@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 256), (5, 2, 3), (33, 4, 1024), (129, 3, 60), (512, 8, 256),
                                   (513, 8, 256), (700, 16, 17), (2100, 2, 2), (1500, 6, 1024)])
def test_sort(m, ws, T, k, E):
    k = min(k, E)
    ids = some_ids(T, T, k, E)
    got = m.sort_tokens(ids.cuda(), E, ws)
    for g, want in zip(got, C.sort(ids, E)):
        assert torch.equal(g.cpu(), want)


def test_sort_large(m, ws):
    """Chunks of more than a thousand assignments, every expert, and one expert alone."""
    for T, k, E, seed in ((40000, 8, 256, 0), (200001, 1, 64, 1)):
        ids = torch.randint(-1, E, (T, k), generator=gen(seed)).to(torch.int32)
        if seed:
            ids[:] = 63
        offsets, perm, inv = (x.cpu() for x in m.sort_tokens(ids.cuda(), E, ws))
        flat = ids.reshape(-1)
        order = torch.argsort(torch.where(flat < 0, E, flat), stable=True)
        total = int((flat >= 0).sum())
        assert torch.equal(offsets.long(), torch.tensor([int((flat < e).sum()) for e in range(E + 1)]) - int((flat < 0).sum()))
        assert torch.equal(perm[:total].long(), order[:total]) and (perm[total:] == -1).all()
        assert torch.equal(inv.reshape(-1)[order[:total]].long(), torch.arange(total))
        assert (inv.reshape(-1)[flat < 0] == -1).all()


def test_sort_edges(m, ws):
    for ids in (torch.zeros(0, 4), torch.full((7, 3), -1), torch.full((5000, 1), -5), torch.full((9, 2), 4)):
        ids = ids.to(torch.int32)
        for g, want in zip(m.sort_tokens(ids.cuda(), 5, ws), C.sort(ids, 5)):
            assert torch.equal(g.cpu(), want)


@pytest.mark.parametrize("T", [3, 5000])
def test_sort_bad_ids(m, ws, T):
    """Ids past the experts count as none and are reported."""
    ids = torch.randint(0, 7, (T, 2), generator=gen(3)).to(torch.int32)
    ids[1, 1], ids[T - 1, 0] = 7, 2 ** 31 - 1
    got = m.sort_tokens(ids.cuda(), 7, ws)
    assert m.read_device_status(ws) == 9
    for g, want in zip(got, C.sort(torch.where(ids > 6, -1, ids), 7)):
        assert torch.equal(g.cpu(), want)


def test_sort_like_route(m, ws):
    """The same places as moe_route's for the ids that it picked."""
    from synthetic import TINY, make_layer, make_tokens
    layer = m.upload_layer(make_layer(TINY, seed=0))
    x = torch.from_numpy(make_tokens(300, TINY.d, seed=0).view("int16")).cuda()
    r = m.route(layer, x, 300, m.workspace(layer.dims, 300))
    offsets, perm, inv = m.sort_tokens(r["topk_idx"], TINY.n_experts, ws)
    assert torch.equal(offsets, r["offsets"]) and torch.equal(perm, r["perm"])
    assert torch.equal(inv.reshape(-1), r["inv_perm"])


# ------------------------------------------------------------------------------------ dispatch
SHAPES = [(1, 1, 16), (3, 2, 48), (7, 8, 128), (65, 3, 144), (33, 5, 528), (9, 16, 1040), (40, 4, 2048), (5, 1, 8208)]


@pytest.mark.parametrize("T,k,d", SHAPES)
def test_dispatch(m, ws, T, k, d):
    x = rand(T, T, d, gain=3.0)
    x[0, :16] = 0
    ids = some_ids(d, T, k, 16)
    _, perm, inv = C.sort(ids, 16)
    total = int((inv >= 0).sum())
    want = x[(perm[:total] // k).long()]
    whole, out = guarded(T * k, d, 0x7FC0)
    assert m.dispatch(dev(x), inv.cuda(), ws, out=out) is out
    assert torch.equal(out[:total].cpu(), want.view(torch.int16)) and (out[total:] == 0x7FC0).all()
    assert untouched(whole, T * k, d, 0x7FC0)
    whole, ws_, rows = guarded_e4m3(m, T * k, d)
    m.dispatch(dev(x), inv.cuda(), ws, out=rows)
    q, scale = C.quantise(want.float())
    assert C.same_codes(rows.q[:total], q) and torch.equal(rows.scale[:total].cpu(), scale)
    assert (rows.q[total:] == 0x55).all() and (rows.scale[total:] == -7.0).all()
    assert untouched_e4m3(whole, ws_, T * k, d)
    # strided rows, and outputs that the call makes
    wide = torch.zeros(T, d + 24, dtype=torch.int16, device="cuda")
    wide[:, 8:8 + d] = dev(x)
    assert torch.equal(m.dispatch(wide[:, 8:8 + d], inv.cuda(), ws)[:total].cpu(), want.view(torch.int16))
    made = m.dispatch(wide[:, 8:8 + d], inv.cuda(), ws, e4m3=True)
    assert made.shape == (T * k, d) and torch.equal(made.q[:total], rows.q[:total])


@pytest.mark.parametrize("d", [16, 128, 272, 4096])
def test_quantise_rows(m, ws, d):
    """No inv: rows in place. Extreme values: zeros, subnormals, the largest, values that are not finite."""
    x = rand(1, 23, d)
    x[1] = 0
    x[2] *= 1e-38
    x[3] = 2.0 ** -133
    x[4] = torch.finfo(torch.bfloat16).max
    x[5, 3], x[5, 9] = float("inf"), float("-inf")
    x[6, 0] = float("nan")
    x[7] = float("inf")
    x[8] *= 2.0 ** -99
    got = m.dispatch(dev(x), None, ws, e4m3=True)
    q, scale = C.quantise(x.float())
    assert C.same_codes(got.q, q) and torch.equal(got.scale.cpu(), scale)
    assert torch.equal(m.dispatch(dev(x), None, ws).cpu(), x.view(torch.int16))
    assert C.same_codes(got.q[5:6], q[5:6]) and int((got.q[5] == 0x7F).sum()) == 2


def test_dispatch_bad_places(m, ws):
    """Places past the rows are skipped and reported; nothing outside is written."""
    x, inv = rand(2, 4, 64), torch.tensor([[0, 9], [1, 2 ** 31 - 1], [2, 8], [3, -1]], dtype=torch.int32)
    for e4m3 in (False, True):
        if e4m3:
            whole, ws_, out = guarded_e4m3(m, 8, 64)
        else:
            whole, out = guarded(8, 64, 0x7FC0)
        m.dispatch(dev(x), inv.cuda(), ws, out=out)
        assert m.read_device_status(ws) == 9
        if e4m3:
            assert (out.q[4:] == 0x55).all() and untouched_e4m3(whole, ws_, 8, 64)
            assert C.same_codes(out.q[:4], C.quantise(x.float())[0])
        else:
            assert (out[4:] == 0x7FC0).all() and untouched(whole, 8, 64, 0x7FC0)
            assert torch.equal(out[:4].cpu(), x.view(torch.int16))


# ------------------------------------------------------------------------------------ combine
@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("T,k,d", SHAPES)
def test_combine(m, ws, T, k, d, add):
    inv = C.sort(some_ids(d + 1, T, k, 16, absent=0.2), 16)[2]
    ys, w = rand(T, T * k, d), torch.rand(T, k, generator=gen(T)) * 2 - 1
    res = rand(T + 1, T, d) if add else None
    dead = torch.ones(T * k, dtype=torch.bool)
    dead[inv[inv >= 0].long()] = False
    ys[dead] = float("nan")                       # rows that no token names
    w[inv < 0] = float("nan")                     # weights of assignments without a place
    whole, y = guarded(T, d, 0x7FC0)
    r = m.combine(dev(ys), inv.cuda(), w.cuda(), ws, add=dev(res) if add else None, y=y)
    assert r is y and untouched(whole, T, d, 0x7FC0)
    ref, size = C.combine(ys.double(), inv, w.double(), res.double() if add else None)
    C.check_combine(y, ref, size, k)
    # without weights: the gradient of dispatch; the output may be the added rows
    ref, size = C.combine(ys.double(), inv, None, res.double() if add else None)
    buf = dev(res) if add else None
    got = m.dispatch_grad(dev(ys), inv.cuda(), ws, add=buf, dx=buf)
    assert not add or got is buf
    C.check_combine(got, ref, size, k)


def test_combine_empty_and_bad(m, ws):
    ys, inv = dev(rand(0, 3, 32)), torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    w = torch.ones(2, 4, device="cuda")
    assert (m.combine(ys, inv, w, ws) == 0).all()
    assert torch.equal(m.combine(ys, inv, w, ws, add=ys[:2]), ys[:2])
    assert (m.combine(ys[:0], inv, w, ws) == 0).all()
    inv[0, 1], inv[1, 3] = 3, 1
    got = m.combine(ys, inv, w, ws)
    assert m.read_device_status(ws) == 9
    assert torch.equal(got[1], ys[1])
    _, dw = m.combine_grad(ys[:2], ys, inv, w, ws)
    assert m.read_device_status(ws) == 9
    assert (dw[0] == 0).all() and (dw[1, :3] == 0).all()


@pytest.mark.parametrize("T,k,d", SHAPES)
def test_combine_grad(m, ws, T, k, d):
    inv = C.sort(some_ids(d + 2, T, k, 16, absent=0.2), 16)[2]
    ys, dy, w = rand(T, T * k, d), rand(T + 3, T, d, gain=0.01), torch.rand(T, k, generator=gen(T)) * 2 - 1
    there = inv >= 0
    place, of = inv[there].long(), there.nonzero()[:, 0]
    x = dy.float()[of] * w[there][:, None]                              # IEEE: what the call rounds or quantises
    want_dw, size = torch.zeros(T, k).double(), torch.zeros(T, k).double()
    want_dw[there] = (dy.double()[of] * ys.double()[place]).sum(-1)
    size[there] = (dy.double()[of] * ys.double()[place]).abs().sum(-1)
    tol = ((d + 511) // 512 * 16 + 8) * 2.0 ** -24 * size
    whole, out = guarded(T * k, d, 0x7FC0)
    dw = torch.full((T, k), float("nan"), device="cuda")
    r = m.combine_grad(dev(dy), dev(ys), inv.cuda(), w.cuda(), ws, out=out, dw=dw)
    assert r[0] is out and r[1] is dw
    C.close(dw, want_dw, tol)
    assert torch.equal(out[place].cpu(), C.bits(x)) and untouched(whole, T * k, d, 0x7FC0)
    dead = torch.ones(T * k, dtype=torch.bool)
    dead[place] = False
    assert (out[dead.cuda()] == 0x7FC0).all()
    whole, ws_, rows = guarded_e4m3(m, T * k, d)
    _, dw = m.combine_grad(dev(dy), dev(ys), inv.cuda(), w.cuda(), ws, out=rows)
    C.close(dw, want_dw, tol)
    q, scale = C.quantise(x)
    assert C.same_codes(rows.q[place], q) and torch.equal(rows.scale[place].cpu(), scale)
    assert (rows.q[dead.cuda()] == 0x55).all() and untouched_e4m3(whole, ws_, T * k, d)


def test_combine_grad_against_differences(m, ws):
    """dw and dys are the slopes of combine: y is linear in either."""
    T, k, d = 6, 3, 96
    inv = C.sort(some_ids(5, T, k, 8, absent=0.0), 8)[2]
    ys, dy, w = rand(1, T * k, d).double(), rand(2, T, d).double(), torch.rand(T, k, generator=gen(3)).double()
    dys, dw = m.combine_grad(dev(dy.to(torch.bfloat16)), dev(ys.to(torch.bfloat16)), inv.cuda(), w.float().cuda(), ws)

    def loss(ys, w):
        return (C.combine(ys, inv, w, None)[0] * dy).sum()

    w = w.float().double()
    for t, j in ((0, 0), (3, 2), (5, 1)):
        step = torch.zeros_like(w)
        step[t, j] = 0.5
        slope = loss(ys, w + step) - loss(ys, w - step)
        assert abs(dw[t, j].item() - slope) <= 2.0 ** -18 * (dy[t] * ys[inv[t, j]]).abs().sum() + 1e-9
        step = torch.zeros_like(ys)
        step[inv[t, j], 17] = 0.5
        slope = loss(ys + step, w) - loss(ys - step, w)
        assert abs(C.values(dys)[inv[t, j], 17] - slope) <= 2.0 ** -8 * abs(slope) + 1e-9


# ------------------------------------------------------------------------------------ SwiGLU
ROWS = [(1, 16), (3, 48), (17, 128), (5, 208), (9, 512), (6, 1040), (2, 4352), (70, 256)]


@pytest.mark.parametrize("grad", [False, True], ids=["forward", "grad"])
@pytest.mark.parametrize("rows,inter", ROWS)
def test_swiglu(m, ws, rows, inter, grad):
    gu, dh = rand(rows, rows, 2 * inter, gain=3.0), rand(rows + 1, rows, inter, gain=0.1)
    gu[0, :8] = torch.tensor([0.0, -0.0, 30.0, -30.0, 88.0, -88.0, 100.0, -100.0])
    cols = 2 * inter if grad else inter
    ref, err = C.swiglu_grad(gu.double(), dh.double()) if grad else C.swiglu(gu.double())

    def call(**kw):
        return m.swiglu_grad(dev(gu), dev(dh), ws, **kw) if grad else m.swiglu(dev(gu), ws, **kw)

    C.check_rows(call(), ref, err)
    C.check_rows(call(e4m3=True), ref, err)
    n = rows - rows // 3
    total = torch.tensor([n], dtype=torch.int32, device="cuda")
    whole, out = guarded(rows, cols, 0x7FC0)
    assert call(total=total, out=out) is out
    C.check_rows(out[:n], ref[:n], err[:n])
    assert (out[n:] == 0x7FC0).all() and untouched(whole, rows, cols, 0x7FC0)
    whole, ws_, out = guarded_e4m3(m, rows, cols)
    call(total=total, out=out)
    C.check_rows(m.E4m3Rows(out.q[:n], out.scale[:n]), ref[:n], err[:n])
    assert (out.q[n:] == 0x55).all() and (out.scale[n:] == -7.0).all() and untouched_e4m3(whole, ws_, rows, cols)


def test_swiglu_strided_and_totals(m, ws):
    rows, inter = 7, 80
    gu, dh = rand(1, rows, 2 * inter), rand(2, rows, inter)
    wide = torch.zeros(rows, 2 * inter + 40, dtype=torch.int16, device="cuda")
    wide[:, 24:24 + 2 * inter] = dev(gu)
    view = wide[:, 24:24 + 2 * inter]
    assert torch.equal(m.swiglu(view, ws), m.swiglu(dev(gu), ws))
    assert torch.equal(m.swiglu_grad(view, dev(dh), ws), m.swiglu_grad(dev(gu), dev(dh), ws))
    for total, kept in ((0, 0), (-3, 0), (8, 7)):
        out = torch.full((rows, inter), 0x7FC0, dtype=torch.int16, device="cuda")
        m.swiglu(dev(gu), ws, total=torch.tensor([total], dtype=torch.int32, device="cuda"), out=out)
        assert m.read_device_status(ws) == (0 if total == 0 else 9)
        assert (out[kept:] == 0x7FC0).all() and torch.equal(out[:kept], m.swiglu(dev(gu), ws)[:kept])
    assert m.swiglu(dev(gu)[:0], ws).shape == (0, inter)


def test_swiglu_not_finite(m, ws):
    """A value that is not finite spoils its own result, not its neighbours'."""
    gu = rand(3, 4, 256)
    want = m.swiglu(dev(gu), ws, e4m3=True)
    bad = gu.clone()
    bad[1, 5], bad[2, 128 + 9], bad[3, 7] = float("nan"), float("inf"), float("-inf")
    got = m.swiglu(dev(bad), ws, e4m3=True)
    assert torch.equal(got.q[0], want.q[0])
    for r, c in ((1, 5), (2, 9), (3, 7)):
        assert got.q[r, c] == 0x7F or got.q[r, c] == 0xFF
        rest = torch.arange(128) != c
        finite = gu.float()[r, :128] * torch.sigmoid(gu.float()[r, :128]) * gu.float()[r, 128:]
        if finite.abs().argmax() != c:
            assert torch.equal(got.q[r].cpu()[rest], want.q[r].cpu()[rest])


def test_swiglu_grad_against_differences(m, ws):
    gu, dh = rand(4, 3, 64).double(), rand(5, 3, 32).double()
    got = C.values(m.swiglu_grad(dev(gu.to(torch.bfloat16)), dev(dh.to(torch.bfloat16)), ws))
    h = 1e-4
    for r in range(3):
        for c in range(64):
            step = torch.zeros_like(gu)
            step[r, c] = h
            slope = ((C.swiglu(gu + step)[0] - C.swiglu(gu - step)[0]) * dh).sum() / (2 * h)
            assert abs(got[r, c] - slope) <= 2.0 ** -8 * abs(slope) + 1e-6


# ------------------------------------------------------------------------------------ weights
@pytest.mark.parametrize("shape", [(1, 16, 16), (2, 128, 128), (3, 144, 272), (1, 400, 48)])
def test_quantise_weights(m, shape):
    E, n, k = shape
    w = rand(n, *shape, gain=0.1)
    w[0, 3, 5], w[0, 7, 7] = float("nan"), float("inf")
    w[-1, -16:, -16:] = 0
    got = m.E4m3Weights.quantise(dev(w))
    assert got.scale.shape == (E, C.blocks(n), C.blocks(k))
    for e in range(E):
        for i in range(0, n, 128):
            for j in range(0, k, 128):
                b = w[e, i:i + 128, j:j + 128].float()
                fine = torch.isfinite(b)
                a = torch.where(fine, b.abs(), torch.zeros(())).max().clamp_min(2.0 ** -100)
                q = (torch.where(fine, b, torch.zeros(())) * (torch.tensor(448.0) / a)).clamp(-448, 448)
                q = torch.where(fine, q.to(torch.float8_e4m3fn).view(torch.uint8), torch.tensor(0x7F, dtype=torch.uint8))
                assert C.same_codes(got.q[e, i:i + 128, j:j + 128], q)
                assert got.scale[e, i // 128, j // 128].item() == (a / torch.tensor(448.0)).item()


# ------------------------------------------------------------------------------------ products
def codes(seed, *shape, gain=100.0):
    return (torch.randn(*shape, generator=gen(seed)) * gain).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def make_product(m, seed, counts, n, k, transposed, spare=0):
    """Rows (spare ones of NaN codes behind the last), weights and offsets on the device, the result in 64 bits."""
    rows, cols, E = sum(counts), n if transposed else k, len(counts)
    aq, a_s = codes(seed, rows + spare, cols), torch.rand(rows + spare, C.blocks(cols), generator=gen(seed + 1)) + 0.25
    if spare:
        aq[rows:] = 0x7F
    wq, w_s = codes(seed + 2, E, n, k), (torch.rand(E, C.blocks(n), C.blocks(k), generator=gen(seed + 3)) + 0.25) * 1e-3
    ref = C.product(C.code_values(aq[:rows], a_s[:rows]), C.weight_values(wq, w_s), counts, transposed)
    offsets = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    return m.E4m3Rows(aq.cuda(), a_s.cuda()), m.E4m3Weights(wq.cuda(), w_s.cuda()), offsets, ref


COUNTS = {
    "one_row": [1],
    "token": [0, 1, 0, 0, 1, 1, 0, 1],
    "few": [3, 0, 9, 1, 0, 17],
    "ragged": [130, 0, 1, 127, 128, 33, 0, 260],
    "last_empty": [5, 70, 0, 0],
    "dense": [300],
}


@pytest.mark.parametrize("transposed", [False, True], ids=["plain", "transposed"])
@pytest.mark.parametrize("n,k", [(16, 16), (128, 128), (144, 272), (400, 1040), (256, 512), (1008, 80)])
@pytest.mark.parametrize("counts", COUNTS.values(), ids=COUNTS.keys())
def test_product(m, ws, counts, n, k, transposed):
    rows, spare = sum(counts), 3
    a, w, offsets, (ref, size) = make_product(m, n + k, counts, n, k, transposed, spare)
    cols, nb = (k, C.blocks(n)) if transposed else (n, C.blocks(k))
    whole, out = guarded(rows + spare, cols, 0x7FC0)
    assert m.gemm_e4m3(a, w, offsets, ws, transposed=transposed, out=out) is out
    assert m.read_device_status(ws) == 0
    C.check_product(out[:rows], ref, size, nb)
    assert (out[rows:] == 0x7FC0).all() and untouched(whole, rows + spare, cols, 0x7FC0)
    if len(counts) == 1:  # one expert needs no offsets
        b = m.E4m3Rows(a.q[:rows], a.scale[:rows])
        assert torch.equal(m.gemm_e4m3(b, w, None, ws, transposed=transposed), out[:rows])


@pytest.mark.parametrize("transposed", [False, True], ids=["plain", "transposed"])
@pytest.mark.parametrize("counts,n,k", [([2700], 528, 400), ([2200, 0, 1, 2500], 272, 144), ([5] * 60 + [0] * 900 + [3] * 64, 32, 48),
                                        ([37, 300], 160, 8336), ([130], 4112, 256), ([1, 700], 2064, 1040)])
def test_product_many_tiles(m, ws, counts, n, k, transposed):
    """More row tiles than run together, more items than SMs, many experts, many blocks of inputs."""
    a, w, offsets, (ref, size) = make_product(m, n + 7 * k, counts, n, k, transposed)
    got = m.gemm_e4m3(a, w, offsets, ws, transposed=transposed)
    C.check_product(got, ref, size, C.blocks(n if transposed else k))


@pytest.mark.parametrize("transposed", [False, True], ids=["plain", "transposed"])
@pytest.mark.parametrize("counts,out,cols", [
    ([2700, 0, 3301], 2064, 144), ([5400], 2064, 1296), ([129, 1, 256, 4700, 40], 4112, 80),        # pairs of CTAs
    ([130] * 30 + [0, 1, 128, 127, 300] * 2, 1040, 144), ([7] * 200, 400, 272), ([64, 32, 65, 33] * 40, 272, 528)])
def test_product_wide(m, ws, counts, out, cols, transposed):
    """More items than SMs: columns 256 at a time, by single CTAs or, where experts have many rows, by pairs."""
    n, k = (cols, out) if transposed else (out, cols)
    a, w, offsets, (ref, size) = make_product(m, out + 3 * cols, counts, n, k, transposed)
    rows = sum(counts)
    whole, got = guarded(rows, out, 0x7FC0)
    for _ in range(3):
        m.gemm_e4m3(a, w, offsets, ws, transposed=transposed, out=got)
    assert m.read_device_status(ws) == 0
    C.check_product(got, ref, size, C.blocks(cols))
    assert untouched(whole, rows, out, 0x7FC0)


@pytest.mark.parametrize("counts", [[1], [3, 5], [9], [40, 0, 91]], ids=str)
@pytest.mark.parametrize("n,k,transposed", [(144, 1040, False), (1040, 144, True), (512, 512, False), (512, 512, True)])
def test_product_strides(m, ws, counts, n, k, transposed):
    """Rows and scales inside wider buffers, on every alignment that the call takes: the same bits."""
    a, w, offsets, _ = make_product(m, 5, counts, n, k, transposed)
    want = m.gemm_e4m3(a, w, offsets, ws, transposed=transposed)
    rows, cols = a.shape
    nb = C.blocks(cols)
    for pad, spad, sat in ((16, 1, 0), (48, 3, 2), (128, 4, 1), (16, 4 - nb % 4, 0)):
        q = torch.full((rows, cols + pad), 0x7F, dtype=torch.uint8, device="cuda")
        s = torch.full((rows, nb + spad + sat), float("nan"), device="cuda")
        q[:, 16:16 + cols], s[:, sat:sat + nb] = a.q, a.scale
        b = m.E4m3Rows(q[:, 16:16 + cols], s[:, sat:sat + nb])
        whole, out = guarded(rows, want.shape[1], 0x7FC0)
        m.gemm_e4m3(b, w, offsets, ws, transposed=transposed, out=out)
        assert torch.equal(out, want) and untouched(whole, rows, want.shape[1], 0x7FC0)
    # the weights' scales on a 4-byte boundary
    flat = torch.full((w.scale.numel() + 1,), float("nan"), device="cuda")
    flat[1:] = w.scale.reshape(-1)
    v = m.E4m3Weights(w.q, flat[1:].view(w.scale.shape))
    assert torch.equal(m.gemm_e4m3(a, v, offsets, ws, transposed=transposed), want)


@pytest.mark.parametrize("transposed", [False, True], ids=["plain", "transposed"])
@pytest.mark.parametrize("counts", [[2, 3, 1], [70, 129, 40]], ids=str)
def test_product_not_finite(m, ws, counts, transposed):
    """A NaN in a row, a weight or a scale spoils what it belongs to and nothing else."""
    n, k = 272, 400
    a, w, offsets, _ = make_product(m, 9, counts, n, k, transposed)
    want = m.gemm_e4m3(a, w, offsets, ws, transposed=transposed).view(torch.bfloat16)
    first = counts[0]
    q, s = a.q.clone(), a.scale.clone()
    q[1, 17] = 0x7F
    s[first, -1] = float("inf")
    got = m.gemm_e4m3(m.E4m3Rows(q, s), w, offsets, ws, transposed=transposed).view(torch.bfloat16)
    fine = torch.ones(sum(counts), dtype=torch.bool, device="cuda")
    fine[1] = fine[first] = False
    assert torch.isnan(got[1]).all() and not torch.isfinite(got[first]).any() and torch.equal(got[fine], want[fine])
    wq, w_s = w.q.clone(), w.scale.clone()
    wq[1, 33, 44] = 0x7F
    w_s[0, 1, 0] = float("nan")
    got = m.gemm_e4m3(a, m.E4m3Weights(wq, w_s), offsets, ws, transposed=transposed).view(torch.bfloat16)
    bad = torch.isnan(got)
    expect = torch.zeros_like(bad)
    expect[first:first + counts[1], 44 if transposed else 33] = True   # the second expert's column
    expect[:first, slice(0, 128) if transposed else slice(128, 256)] = True  # the first expert's block of columns
    assert torch.equal(bad, expect) and torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("rows,k", [(7, 256), (300, 256), (300, 2064)])
def test_product_bad_offsets(m, ws, rows, k):
    """Offsets outside the rows or descending: reported, and nothing written. Offsets that begin late or end early
    leave the rows around them as they were."""
    n = 144
    a, w, _, _ = make_product(m, 11, [rows, 0, 0, 0], n, k, False)
    one = [m.gemm_e4m3(a, m.E4m3Weights(w.q[e:e + 1], w.scale[e:e + 1]), None, ws) for e in range(4)]
    for offsets in ([0, 2, 2, rows + 1, rows + 1], [-5, 3, 4, 4, rows], [0, 4, 2, 5, 6], [0, rows, 0, rows, 0],
                    [2 ** 31 - 1, -2 ** 31, 5, 5, 5], [-1] * 5, [0, 0, 0, 0, 2 ** 31 - 1]):
        whole, out = guarded(rows, n, 0x7FC0)
        m.gemm_e4m3(a, w, torch.tensor(offsets, dtype=torch.int32, device="cuda"), ws, out=out)
        assert m.read_device_status(ws) == 9, offsets
        assert (whole == 0x7FC0).all()
    for offsets in ([1, 3, 3, 5, 6], [rows] * 5, [0] * 5, [0, 0, 2, 2, 2], [0, 1, 2, 3, rows]):
        whole, out = guarded(rows, n, 0x7FC0)
        m.gemm_e4m3(a, w, torch.tensor(offsets, dtype=torch.int32, device="cuda"), ws, out=out)
        assert m.read_device_status(ws) == 0, offsets
        assert untouched(whole, rows, n, 0x7FC0)
        for e in range(4):
            lo, hi = offsets[e:e + 2]
            assert torch.equal(out[lo:hi], one[e][lo:hi]), offsets
        assert (out[:offsets[0]] == 0x7FC0).all() and (out[offsets[-1]:] == 0x7FC0).all()


@pytest.mark.parametrize("rows", [1, 64])
def test_product_sums_in_32_bits(m, ws, rows):
    """Large products that cancel leave the small ones, within a block and across blocks, up to fp32's precision: within
    a block 2^17.6 beside 2^-4, 22 bits; across blocks 2^18 beside 2^-4."""
    def run(a, w):
        k = len(a)
        code = lambda x: torch.tensor(x).to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
        r = m.E4m3Rows(code([a] * rows).cuda(), torch.ones(rows, C.blocks(k), device="cuda"))
        v = m.E4m3Weights(code([w] * 16)[None].cuda(), torch.ones(1, 1, C.blocks(k), device="cuda"))
        return m.gemm_e4m3(r, v, None, ws).view(torch.bfloat16)
    for k, far in ((128, 31), (128, 127), (1152, 128), (1152, 1151)):
        a, w = [0.0] * k, [0.0] * k
        a[0] = w[0] = w[far] = 448.0
        a[far] = -448.0
        a[5], w[5] = 0.25, 0.25
        assert (run(a, w) == 0.0625).all(), (k, far)


def test_product_directions_agree(m, ws):
    """The transposed product on W is the plain one on a copy of W^T."""
    counts, n, k = [40, 0, 200, 3], 384, 256
    a, w, offsets, _ = make_product(m, 21, counts, n, k, True)
    t = m.E4m3Weights(w.q.transpose(1, 2).contiguous(), w.scale.transpose(1, 2).contiguous())
    assert torch.equal(m.gemm_e4m3(a, w, offsets, ws, transposed=True), m.gemm_e4m3(a, t, offsets, ws))


def test_product_same_bits(m):
    """Calls repeat bit for bit, on any stream, two at once with a workspace each, and from a graph."""
    for counts, n, k in (([700, 0, 333, 1], 784, 1040), ([1, 2, 0, 1], 528, 2064)):
        a, w, offsets, _ = make_product(m, 3, counts, n, k, False)
        spaces = [m.expert_workspace(4) for _ in range(2)]
        want = m.gemm_e4m3(a, w, offsets, spaces[0])
        for _ in range(10):
            assert torch.equal(m.gemm_e4m3(a, w, offsets, spaces[0]), want)
        torch.cuda.synchronize()
        streams, outs = [torch.cuda.Stream() for _ in range(2)], [[], []]
        for _ in range(5):
            for s, sp, o in zip(streams, spaces, outs):
                with torch.cuda.stream(s):
                    o.append(m.gemm_e4m3(a, w, offsets, sp))
        torch.cuda.synchronize()
        assert all(torch.equal(x, want) for o in outs for x in o)
        assert all(m.read_device_status(sp) == 0 for sp in spaces)


# ------------------------------------------------------------------------------------ long strides
def test_rows_far_apart(m, ws):
    """Rows whose distance from the first passes 2^31 values and bytes."""
    rows, d, n, stride = 140, 256, 144, 1 << 24
    buf16, buf8 = (torch.empty(rows * stride, dtype=t, device="cuda") for t in (torch.int16, torch.uint8))
    bufs = torch.empty(rows * stride, dtype=torch.float32, device="cuda")

    def far16(cols):
        return buf16.as_strided((rows, cols), (stride, 1))

    def far8(cols):
        return m.E4m3Rows(buf8.as_strided((rows, cols), (stride, 1)), bufs.as_strided((rows, C.blocks(cols)), (stride, 1)))

    x = dev(rand(1, rows, d))
    inv = torch.arange(rows, dtype=torch.int32, device="cuda").flip(0).view(rows, 1).contiguous()
    near = m.dispatch(x, inv, ws, e4m3=True)
    far = m.dispatch(x, inv, ws, out=far8(d))
    assert torch.equal(far.q, near.q) and torch.equal(far.scale, near.scale)
    w = m.E4m3Weights.quantise(dev(rand(2, 1, n, d, gain=0.1)))
    y = m.gemm_e4m3(near, w, None, ws)
    assert torch.equal(m.gemm_e4m3(far, w, None, ws, out=far16(n)), y)
    one = torch.ones(rows, 1, device="cuda")
    back = m.combine(y, inv, one, ws)
    assert torch.equal(m.combine(far16(n), inv, one, ws), back) and torch.equal(back, y.flip(0))
    dys, dw = m.combine_grad(back, y, inv, one, ws)
    far_dys, far_dw = m.combine_grad(back, far16(n), inv, one, ws, out=far8(n))
    assert torch.equal(dw, far_dw) and torch.equal(far_dys.q, m.dispatch(dys, None, ws, e4m3=True).q)
    far16(d).copy_(x)
    assert torch.equal(m.swiglu(far16(d), ws), m.swiglu(x, ws))
    dh = dev(rand(3, rows, d // 2))
    assert torch.equal(m.swiglu_grad(far16(d), dh, ws), m.swiglu_grad(x, dh, ws))
    assert torch.equal(m.dispatch(far16(d), inv, ws), m.dispatch(x, inv, ws))


# ------------------------------------------------------------------------------------ together
class Layer:
    """A layer of e4m3 experts and its gradients, as a program would run them; every intermediate is kept."""

    def __init__(self, m, E, d, inter, seed):
        self.m, self.E, self.ws = m, E, m.expert_workspace(E)
        self.gate_up = m.E4m3Weights.quantise(dev(rand(seed, E, 2 * inter, d, gain=d ** -0.5)))
        self.down = m.E4m3Weights.quantise(dev(rand(seed + 1, E, d, inter, gain=inter ** -0.5)))

    def forward(self, x, ids, w):
        m, ws, s = self.m, self.ws, {}
        s["offsets"], s["perm"], s["inv"] = m.sort_tokens(ids, self.E, ws)
        s["xs"] = m.dispatch(x, s["inv"], ws, e4m3=True)
        s["gu"] = m.gemm_e4m3(s["xs"], self.gate_up, s["offsets"], ws)
        s["h"] = m.swiglu(s["gu"], ws, total=s["offsets"][-1:], e4m3=True)
        s["ys"] = m.gemm_e4m3(s["h"], self.down, s["offsets"], ws)
        s["y"] = m.combine(s["ys"], s["inv"], w, ws, add=x)
        return s

    def backward(self, s, dy, w):
        m, ws = self.m, self.ws
        s["dys"], s["dw"] = m.combine_grad(dy, s["ys"], s["inv"], w, ws, e4m3=True)
        s["dh"] = m.gemm_e4m3(s["dys"], self.down, s["offsets"], ws, transposed=True)
        s["dgu"] = m.swiglu_grad(s["gu"], s["dh"], ws, total=s["offsets"][-1:], e4m3=True)
        s["dxs"] = m.gemm_e4m3(s["dgu"], self.gate_up, s["offsets"], ws, transposed=True)
        s["dx"] = m.dispatch_grad(s["dxs"], s["inv"], ws, add=dy)
        return s


def check_layer(layer, s, x, ids, w, dy):
    """Every step against 64 bits on what the step before made."""
    E, T, k = layer.E, *ids.shape
    offsets, perm, inv = C.sort(ids, E)
    for name, want in (("offsets", offsets), ("perm", perm), ("inv", inv)):
        assert torch.equal(s[name].cpu(), want), name
    n = int(offsets[-1])
    counts = (offsets[1:] - offsets[:-1]).tolist()
    q, scale = C.quantise(x[(perm[:n] // k).long()].float())
    assert C.same_codes(s["xs"].q[:n], q) and torch.equal(s["xs"].scale[:n].cpu(), scale)
    gate_up, down = (C.weight_values(v.q, v.scale) for v in (layer.gate_up, layer.down))

    def rows(r):
        return C.code_values(r.q[:n], r.scale[:n])

    def product(got, a, v, weights, transposed, nb):
        ref, size = C.product(rows(a), weights, counts, transposed)
        C.check_product(got[:n], ref, size, nb, v)

    d, inter = x.shape[1], down.shape[2]
    product(s["gu"], s["xs"], "gu", gate_up, False, C.blocks(d))
    gu = C.values(s["gu"])[:n]
    E4 = type(s["h"])
    C.check_rows(E4(s["h"].q[:n], s["h"].scale[:n]), *C.swiglu(gu), "h")
    product(s["ys"], s["h"], "ys", down, False, C.blocks(inter))
    ys = torch.zeros(T * k, d).double()
    ys[:n] = C.values(s["ys"])[:n]
    C.check_combine(s["y"], *C.combine(ys, inv, w.double(), x.double()), k, "y")
    there = inv >= 0
    of, place = there.nonzero()[:, 0], inv[there].long()
    q, scale = C.quantise(dy.float()[of] * w[there][:, None])
    assert C.same_codes(s["dys"].q[place], q) and torch.equal(s["dys"].scale[place].cpu(), scale)
    dw, size = torch.zeros(T, k).double(), torch.zeros(T, k).double()
    dw[there] = (dy.double()[of] * ys[place]).sum(-1)
    size[there] = (dy.double()[of] * ys[place]).abs().sum(-1)
    C.close(s["dw"], dw, ((d + 511) // 512 * 16 + 8) * 2.0 ** -24 * size, "dw")
    product(s["dh"], s["dys"], "dh", down, True, C.blocks(d))
    C.check_rows(E4(s["dgu"].q[:n], s["dgu"].scale[:n]), *C.swiglu_grad(gu, C.values(s["dh"])[:n]), "dgu")
    product(s["dxs"], s["dgu"], "dxs", gate_up, True, C.blocks(2 * inter))
    dxs = torch.zeros(T * k, d).double()
    dxs[:n] = C.values(s["dxs"])[:n]
    C.check_combine(s["dx"], *C.combine(dxs, inv, None, dy.double()), k, "dx")


def batch(seed, T, k, E, d):
    x, dy = rand(seed, T, d), rand(seed + 1, T, d, gain=0.01)
    ids = some_ids(seed + 2, T, k, E)
    ids[T - T // 8:] = -1  # padding at the end of the batch
    return x, dy, ids, torch.softmax(torch.randn(T, k, generator=gen(seed + 3)), -1)


@pytest.mark.parametrize("T,k,E,d,inter", [(1, 2, 8, 256, 128), (7, 4, 16, 272, 144), (150, 3, 6, 512, 256), (40, 8, 64, 128, 80)])
def test_layer(m, T, k, E, d, inter):
    layer = Layer(m, E, d, inter, seed=T)
    x, dy, ids, w = batch(T, T, k, E, d)
    s = layer.backward(layer.forward(dev(x), ids.cuda(), w.cuda()), dev(dy), w.cuda())
    assert m.read_device_status(layer.ws) == 0
    check_layer(layer, s, x, ids, w, dy)


def test_layer_from_a_graph(m):
    """Forward and backward captured once, replayed on other inputs: other routing, other absent tokens."""
    T, k, E, d, inter = 60, 3, 12, 256, 144
    layer = Layer(m, E, d, inter, seed=1)
    x, dy, ids, w = (t.cuda() for t in batch(1, T, k, E, d))
    x, dy = x.view(torch.int16), dy.view(torch.int16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.backward(layer.forward(x, ids, w), dy, w)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s = layer.backward(layer.forward(x, ids, w), dy, w)
    for seed in (5, 9):
        new = batch(seed, T, k, E, d)
        for to, t in zip((x, dy, ids, w), new):
            to.copy_(dev(t))
        graph.replay()
        torch.cuda.synchronize()
        assert m.read_device_status(layer.ws) == 0
        check_layer(layer, s, new[0], new[2], new[3], new[1])
        eager = layer.backward(layer.forward(x, ids, w), dy, w)
        for name in ("y", "dx", "dw", "inv"):
            assert torch.equal(eager[name], s[name]), name


def test_no_rows(m, ws):
    """Nothing to do is nothing done."""
    x, inv = torch.empty(0, 64, dtype=torch.int16, device="cuda"), torch.empty(0, 3, dtype=torch.int32, device="cuda")
    w = torch.empty(0, 3, device="cuda")
    assert m.dispatch(x, inv, ws).shape == (0, 64) and m.dispatch(x, inv, ws, e4m3=True).shape == (0, 64)
    assert m.combine(x, inv, w, ws).shape == (0, 64)
    assert m.combine_grad(x, x, inv, w, ws)[1].shape == (0, 3)
    v = m.E4m3Weights.quantise(dev(rand(0, 2, 32, 64)))
    offsets = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert m.gemm_e4m3(m.E4m3Rows.empty(0, 64), v, offsets, ws).shape == (0, 32)
    out = torch.full((5, 32), 0x7FC0, dtype=torch.int16, device="cuda")
    m.gemm_e4m3(m.dispatch(dev(rand(1, 5, 64)), None, ws, e4m3=True), v, offsets, ws, out=out)  # no expert has rows
    assert (out == 0x7FC0).all()


# ------------------------------------------------------------------------------------ the widest rows
@pytest.mark.parametrize("n,k,rows", [(16, 65536, 3), (16, 65536, 40), (65536, 16, 5), (65536, 48, 200), (32, 65520, 129)])
def test_product_widest(m, ws, n, k, rows):
    for transposed in (False, True):
        a, w, offsets, (ref, size) = make_product(m, 1, [rows], n, k, transposed)
        got = m.gemm_e4m3(a, w, None, ws, transposed=transposed)
        C.check_product(got, ref, size, C.blocks(n if transposed else k))


def test_rows_widest(m, ws):
    d = 65536
    x, inv = rand(1, 2, d), torch.tensor([[1, 2], [0, -1]], dtype=torch.int32)
    rows = m.dispatch(dev(x), inv.cuda(), ws, e4m3=True)
    q, scale = C.quantise(x.float()[[1, 0, 0]])
    assert C.same_codes(rows.q[:3], q) and torch.equal(rows.scale[:3].cpu(), scale)
    ys = rand(2, 4, d)
    w = torch.tensor([[0.5, 2.0], [1.5, 9.0]])
    y = m.combine(dev(ys), inv.cuda(), w.cuda(), ws)
    C.check_combine(y, *C.combine(ys.double(), inv, w.double(), None), 2)
    dys, dw = m.combine_grad(dev(x), dev(ys), inv.cuda(), w.cuda(), ws)
    assert torch.equal(dys[:3].cpu(), C.bits(x.float()[[1, 0, 0]] * torch.tensor([[1.5], [0.5], [2.0]])))
    ref = torch.stack([x[0].double() @ ys[1].double(), x[0].double() @ ys[2].double(), x[1].double() @ ys[0].double()])
    size = torch.stack([x[0].double().abs() @ ys[1].double().abs(), x[0].double().abs() @ ys[2].double().abs(),
                        x[1].double().abs() @ ys[0].double().abs()])
    C.close(dw.reshape(-1)[:3], ref, (d // 512 * 16 + 8) * 2.0 ** -24 * size)
    gu, dh = rand(3, 2, d, gain=2.0), rand(4, 2, d // 2)
    C.check_rows(m.swiglu(dev(gu), ws, e4m3=True), *C.swiglu(gu.double()))
    C.check_rows(m.swiglu_grad(dev(gu), dev(dh), ws, e4m3=True), *C.swiglu_grad(gu.double(), dh.double()))
