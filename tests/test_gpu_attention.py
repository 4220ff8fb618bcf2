"""The attention calls on a GB300 against plain 64-bit arithmetic (tests/attn_check.py): packed
prompts, the paged cache's append, one new token per sequence over the cache."""
import math

import pytest

torch = pytest.importorskip("torch")

from tests import attn_check as C  # noqa: E402

pytestmark = pytest.mark.gpu

HEADS = [(16, 2), (8, 8), (7, 1), (12, 4), (10, 2), (64, 1)]


@pytest.fixture(scope="module")
def m():
    from quantized_grouped_gemm_router_gb300 import build as B
    B.build()
    import quantized_grouped_gemm_router_gb300 as mod
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return mod


def rand(seed, *shape, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * gain).to(torch.bfloat16)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cu(lens):
    return ints([0] + torch.tensor(lens).cumsum(0).tolist())


def status(m, ws):
    return m.read_device_status(ws)


# ------------------------------------------------------------------------------------ prompts
def run_prefill(m, dims, q, k, v, lens, causal, scale=None, ws=None):
    """q, k, v: CUDA int16 views; returns o, lse with every element pre-filled with NaN."""
    ws = m.attn_workspace(dims) if ws is None else ws
    o = torch.full((q.shape[0], dims.n_q_heads, dims.head_dim), 0x7FC0, dtype=torch.int16, device="cuda")
    lse = torch.full((q.shape[0], dims.n_q_heads), math.nan, device="cuda")
    r = m.attn_prefill(dims, q, k, v, cu([x for x, _ in lens]), cu([x for _, x in lens]), ws, causal=causal,
                       scale=scale, o=o, lse=lse)
    assert r is o
    assert status(m, ws) == 0
    return o, lse


def prompt_case(m, heads, d, lens, causal, seed=0, scale=None, gain=2.0):
    hq, hkv = heads
    tq, tk = sum(x for x, _ in lens), sum(x for _, x in lens)
    q, k, v = rand(seed, tq, hq, d, gain=gain), rand(seed + 1, tk, hkv, d), rand(seed + 2, tk, hkv, d)
    o, lse = run_prefill(m, m.AttnDims(hq, hkv, d), *(x.view(torch.int16).cuda() for x in (q, k, v)), lens, causal,
                         scale)
    ref = C.prefill(q.double(), k.double(), v.double(), lens, 1 / math.sqrt(d) if scale is None else scale, causal)
    C.check(o, lse, ref, 8, f"{heads} {d} {lens} causal={causal}")


LENS = {
    "one": [(1, 1)],
    "odd": [(131, 131)],
    "ragged": [(0, 0), (1, 1), (70, 70), (0, 3), (129, 129), (2, 2)],
    "continued": [(5, 133), (1, 260), (64, 64), (33, 161)],
    "fewer_keys": [(40, 7), (3, 0), (130, 129), (1, 1)],   # rows that see nothing
}


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "both"])
@pytest.mark.parametrize("lens", LENS.values(), ids=LENS.keys())
@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompt_lengths(m, d, lens, causal):
    prompt_case(m, (16, 2), d, lens, causal)


@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompt_heads(m, heads, d):
    prompt_case(m, heads, d, [(37, 37), (19, 150)], True, seed=5)


@pytest.mark.parametrize("d,n", [(64, 700), (128, 641), (256, 515)])
def test_prompt_many_tiles(m, d, n):
    prompt_case(m, (4, 2), d, [(n, n)], True, seed=9, gain=4.0)
    prompt_case(m, (2, 2), d, [(n, n + 100)], False, seed=10, gain=4.0)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompt_whole_tiles(m, d):
    """Every row sees every tile whole, and the last tiles count: nothing delays the end of an item."""
    for n, gain in ((640, 4.0), (576, 4.0), (128, 4.0), (1280, 8.0)):
        prompt_case(m, (2, 2), d, [(515, n)], False, seed=21, gain=gain)
        prompt_case(m, (16, 2), d, [(70, n), (3, n)], False, seed=22, gain=gain)


@pytest.mark.parametrize("heads,d,n", [((2, 2), 64, 200), ((16, 2), 128, 2600), ((4, 2), 256, 150)])
def test_prompt_output_alignment(m, heads, d, n):
    """Output rows on 16-byte boundaries that are no 32-byte ones."""
    hq, hkv = heads
    q, k, v = (x.view(torch.int16).cuda() for x in (rand(30, n, hq, d), rand(31, n, hkv, d), rand(32, n, hkv, d)))
    dims = m.AttnDims(hq, hkv, d)
    ws = m.attn_workspace(dims)
    want = m.attn_prefill(dims, q, k, v, cu([n]), cu([n]), ws)
    buf = torch.full((n * hq * d + 16,), 0x7FC0, dtype=torch.int16, device="cuda")
    o = buf[8:-8].view(n, hq, d)
    assert o.data_ptr() % 32 == 16
    m.attn_prefill(dims, q, k, v, cu([n]), cu([n]), ws, o=o)
    assert torch.equal(o, want)
    assert (buf[:8] == 0x7FC0).all() and (buf[-8:] == 0x7FC0).all()


@pytest.mark.parametrize("heads,d,lens,causal", [
    ((16, 2), 128, [2600], True), ((8, 8), 64, [250] * 24, False), ((16, 2), 128, [300] * 30, True),
    ((16, 2), 256, [300] * 30, True)])
def test_prompt_same_bits(m, heads, d, lens, causal):
    """Which SM computes what varies from call to call; the result does not."""
    (hq, hkv), n = heads, sum(lens)
    q, k, v = (x.view(torch.int16).cuda() for x in (rand(40, n, hq, d, gain=4.0), rand(41, n, hkv, d), rand(42, n, hkv, d)))
    dims = m.AttnDims(hq, hkv, d)
    ws, c = m.attn_workspace(dims), cu(lens)
    first = None
    for _ in range(20):
        lse = torch.empty(n, hq, device="cuda")
        got = m.attn_prefill(dims, q, k, v, c, c, ws, causal=causal, lse=lse), lse
        first = first or got
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])


@pytest.mark.parametrize("heads", [(7, 1), (16, 2), (4, 4)], ids=str)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompt_neighbours(m, heads, d):
    """A sequence's bits do not depend on the queries of the next one, nor on what ran before."""
    (hq, hkv), lens = heads, [300, 77]
    q, k, v = rand(50, 377, hq, d), rand(51, 377, hkv, d), rand(52, 377, hkv, d)
    k *= torch.linspace(0.2, 3.0, 377).to(torch.bfloat16)[:, None, None]  # maxima that grow
    dims, c = m.AttnDims(hq, hkv, d), cu(lens)
    ws = m.attn_workspace(dims)
    outs = []
    for gain in (1.0, 1000.0, -1000.0):
        q2 = q.clone()
        q2[300:] *= gain
        x, y, z = (t.view(torch.int16).cuda() for t in (q2, k, v))
        outs.append(m.attn_prefill(dims, x, y, z, c, c, ws)[:300].clone())
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_prompt_many_sequences(m):
    prompt_case(m, (4, 2), 64, [(i % 4, (i * 7) % 9) for i in range(300)], True, seed=11)


def test_prompt_growing_scores(m):
    """Scores that grow along the keys: the running maximum moves in every tile."""
    d, n = 128, 600
    q, v = torch.full((n, 1, d), 0.5).to(torch.bfloat16), rand(1, n, 1, d)
    k = (torch.arange(n).double()[:, None, None] / 40 * torch.ones(1, 1, d)).to(torch.bfloat16)
    o, lse = run_prefill(m, m.AttnDims(1, 1, d), *(x.view(torch.int16).cuda() for x in (q, k, v)), [(n, n)], True,
                         scale=1.0)
    C.check(o, None, C.prefill(q.double(), k.double(), v.double(), [(n, n)], 1.0, True), 8)
    # scores up to 960: an fp32 sum of 128 equal products below 2^11, in steps of 2^-13 at most
    ref = C.prefill(q.double(), k.double(), v.double(), [(n, n)], 1.0, True)[1]
    assert (lse.cpu().double() - ref).abs().max() < 2.0 ** -9


def test_prompt_scale_and_negative_scores(m):
    prompt_case(m, (4, 2), 64, [(90, 90)], True, seed=12, scale=0.01)
    d, n = 64, 300                                   # every score strongly negative
    q, v = torch.ones(n, 2, d).to(torch.bfloat16), rand(2, n, 1, d)
    k = -torch.ones(n, 1, d).to(torch.bfloat16) * 4 + rand(3, n, 1, d, gain=0.1)
    o, lse = run_prefill(m, m.AttnDims(2, 1, d), *(x.view(torch.int16).cuda() for x in (q, k, v)), [(n, n)], True,
                         scale=1.0)
    C.check(o, None, C.prefill(q.double(), k.double(), v.double(), [(n, n)], 1.0, True), 8)


@pytest.mark.parametrize("layout", ["fused", "heads_first", "padded"])
def test_prompt_strides(m, layout):
    hq, hkv, d, n = 6, 2, 64, 150
    q, k, v = rand(1, n, hq, d), rand(2, n, hkv, d), rand(3, n, hkv, d)
    if layout == "fused":
        rows = torch.cat([q, k, v], 1).contiguous().view(torch.int16).cuda()
        dev = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
    elif layout == "heads_first":
        dev = [x.permute(1, 0, 2).contiguous().view(torch.int16).cuda().permute(1, 0, 2) for x in (q, k, v)]
    else:
        dev = [torch.cat([x, torch.full((n, x.shape[1], 8), math.nan, dtype=torch.bfloat16)], 2).view(torch.int16)
               .cuda()[:, :, :d] for x in (q, k, v)]
    o, lse = run_prefill(m, m.AttnDims(hq, hkv, d), *dev, [(n, n)], True)
    C.check(o, lse, C.prefill(q.double(), k.double(), v.double(), [(n, n)], 1 / 8, True), 8, layout)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf], ids=str)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompt_nonfinite_unseen(m, d, bad):
    """Keys and values that a row does not see (later tokens of its own sequence, other sequences)
    never reach it; the rows that see them are not compared."""
    lens, hq, hkv = [(50, 50), (140, 140), (20, 20)], 4, 2
    n = sum(x for x, _ in lens)
    q, k, v = rand(1, n, hq, d), rand(2, n, hkv, d), rand(3, n, hkv, d)
    ref = C.prefill(q.double(), k.double(), v.double(), lens, 1 / math.sqrt(d), True)
    kb, vb = k.clone(), v.clone()
    kb[50 + 100:50 + 140], vb[50 + 90:50 + 140] = bad, bad      # seen from row 90 of the middle sequence on
    kb[190, 0], vb[190, 1, 3] = bad, bad                        # first key of the last sequence
    o, lse = run_prefill(m, m.AttnDims(hq, hkv, d), *(x.view(torch.int16).cuda() for x in (q, kb, vb)), lens, True)
    C.check(o[:140], lse[:140], [x[:140] for x in ref], 8)
    got = C.values(o)
    assert not torch.isfinite(got[140:190]).all(dim=-1).any()   # and rows that do see them show it
    # in the last sequence only the heads and columns that read the bad cells
    assert torch.isfinite(got[190:, 2:, :3]).all() and torch.isfinite(got[190:, 2:, 4:]).all()
    assert not torch.isfinite(got[190:, 2:, 3]).any()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompt_nonfinite_many_heads(m, d):
    """The same with more row tiles than SMs: single bad values, first rows before them compared."""
    lens, h = [(620, 620), (404, 404)], 64
    n = 1024
    q, k, v = rand(4, n, h, d), rand(5, n, h, d), rand(6, n, h, d)
    at = [17, 128, 255, 256, 383, 500, 619]
    sel = torch.arange(0, h, 9)                                 # heads compared; the reference takes a while
    ref = C.prefill(q[:, sel].double(), k[:, sel].double(), v[:, sel].double(), lens, 1 / math.sqrt(d), True)
    vb = v.clone()
    for i, x in enumerate(at):
        vb[x, :, i] = (math.nan, math.inf, -math.inf)[i % 3]    # one column each
    vb[620 + 400:] = math.nan
    o, lse = run_prefill(m, m.AttnDims(h, h, d), *(x.view(torch.int16).cuda() for x in (q, k, vb)), lens, True)
    o, lse = o[:, sel.cuda()], lse[:, sel.cuda()]
    got = C.values(o)
    for i, x in enumerate(at):
        assert not torch.isfinite(got[x:620, :, i]).any() and torch.isfinite(got[:x, :, i]).all()
    clean = torch.ones(n, 1, d, dtype=torch.bool)
    for i, x in enumerate(at):
        clean[x:620, :, i] = False
    clean[620 + 400:] = False
    fixed = torch.where(clean, got, ref[0]).to(torch.bfloat16).view(torch.int16)
    C.check(fixed, lse, ref, 8)


def test_prompt_nonfinite_both_ways(m):
    """Without causality the tail of a tile still belongs to another sequence."""
    lens, d = [(70, 70), (30, 30)], 128
    q, k, v = rand(1, 100, 2, d), rand(2, 100, 1, d), rand(3, 100, 1, d)
    ref = C.prefill(q.double(), k.double(), v.double(), lens, 1 / math.sqrt(d), False)
    k[70:], v[70:] = math.inf, math.nan
    o, lse = run_prefill(m, m.AttnDims(2, 1, d), *(x.view(torch.int16).cuda() for x in (q, k, v)), lens, False)
    C.check(o[:70], lse[:70], [x[:70] for x in ref], 8)


def test_prompt_bad_offsets(m):
    """Offsets outside the rows raise the status and touch nothing outside the buffers."""
    dims = m.AttnDims(4, 2, 64)
    x = rand(1, 40, 4, 64).view(torch.int16).cuda()
    for cq, ck in (([0, 30, 20, 40], [0, 30, 30, 40]), ([0, 10, 20, 400], [0, 10, 20, 40]),
                   ([0, 10, 20, 40], [0, 10, 20, 1000000]), ([-5, 10, 20, 40], [0, 10, 20, 40]),
                   ([0, 10, 20, 40], [0, -1000000, 20, 40])):
        ws = m.attn_workspace(dims)
        m.attn_prefill(dims, x, x[:, :2], x[:, 2:], ints(cq), ints(ck), ws)
        assert status(m, ws) == 9, (cq, ck)
        assert status(m, ws) == 0


def test_prompt_streams_graphs_and_repeats(m):
    dims, lens = m.AttnDims(8, 2, 128), [(200, 200), (77, 77)]
    q, k, v = (rand(i, 277, h, 128).view(torch.int16).cuda() for i, h in ((1, 8), (2, 2), (3, 2)))
    c, ws = cu([200, 77]), m.attn_workspace(dims)
    a, _ = run_prefill(m, dims, q, k, v, lens, True, ws=ws)
    b, _ = run_prefill(m, dims, q, k, v, lens, True, ws=ws)
    assert torch.equal(a, b)
    o = torch.zeros_like(a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.attn_prefill(dims, q, k, v, c, c, ws, o=o)
    side.synchronize()
    assert torch.equal(a, o)
    o.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.attn_prefill(dims, q, k, v, c, c, ws, o=o)
    for _ in range(2):
        o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, o)


def test_prompt_far_offsets(m):
    """Rows more than 2^32 bytes apart (2^31 elements and more from the base)."""
    d, n, step = 64, 1100, 1 << 22
    big = torch.empty((n * step,), dtype=torch.int16, device="cuda")
    rows = big.as_strided((n, 4, d), (step, d, 1))
    x = rand(1, n, 4, d)
    rows.copy_(x.view(torch.int16).cuda())
    lens = [(1000, 1000), (100, 100)]
    o, lse = run_prefill(m, m.AttnDims(2, 1, d), rows[:, :2], rows[:, 2:3], rows[:, 3:], lens, True)
    ref = C.prefill(x[1000:, :2].double(), x[1000:, 2:3].double(), x[1000:, 3:].double(), lens[1:], 1 / 8, True)
    C.check(o[1000:], lse[1000:], ref, 8)


def test_prompt_empty(m):
    dims = m.AttnDims(4, 2, 64)
    ws = m.attn_workspace(dims)
    none = torch.empty((0, 4, 64), dtype=torch.int16, device="cuda")
    assert m.attn_prefill(dims, none, none[:, :2], none[:, :2], ints([0, 0]), ints([0, 0]), ws).shape == (0, 4, 64)
    q = rand(1, 5, 4, 64).view(torch.int16).cuda()
    o, lse = run_prefill(m, dims, q, none[:, :2], none[:, :2], [(5, 0)], False)
    assert (o == 0).all() and (lse == -math.inf).all()


# ------------------------------------------------------------------------------------ the cache
def table_for(lens, page, seed=0, spare=2):
    """A random page table; entries past a sequence's pages name no page at all."""
    g = torch.Generator().manual_seed(seed)
    need = [(n + page - 1) // page for n in lens]
    total = sum(need) + spare
    order = torch.randperm(total, generator=g).tolist()
    t = torch.full((len(lens), max(1, max(need))), -7, dtype=torch.int32)
    for b, n in enumerate(need):
        for i in range(n):
            t[b, i] = order.pop()
    return t, total


def e4m3(x, scale):
    return (x.float() / scale).clamp(-448, 448).to(torch.float8_e4m3fn)


def make_cache(m, dims, lens, page, fp8, seed=0, table=None):
    """Random keys and values of every position, in the cache's own cells (all others hold NaN), and
    the values they stand for, [hkv, len, d] in 64 bits per sequence."""
    hkv, d = dims.n_kv_heads, dims.head_dim
    t, total = table_for(lens, page, seed) if table is None else table
    scales = [torch.rand(hkv, generator=torch.Generator().manual_seed(seed + i)) * 0.02 + 0.01 for i in range(2)]
    cells = [torch.full((total, hkv, page, d), 0x7F if fp8 else 0x7FC0, dtype=torch.uint8 if fp8 else torch.int16)
             for _ in range(2)]
    vals = []
    for b, n in enumerate(lens):
        both = []
        pos = torch.arange(n)
        at = t[b, pos // page].long()
        for i in range(2):
            x = rand(seed + 10 * b + i, n, hkv, d)
            if fp8:
                code = e4m3(x, scales[i][None, :, None])
                cells[i][at, :, pos % page] = code.view(torch.uint8)
                both.append((code.float().double() * scales[i].double()[None, :, None]).transpose(0, 1))
            else:
                cells[i][at, :, pos % page] = x.view(torch.int16)
                both.append(x.double().transpose(0, 1))
        vals.append(both)
    cache = m.KvCache(dims, cells[0].cuda(), cells[1].cuda(), *((s.cuda() for s in scales) if fp8 else ()))
    return cache, t.cuda(), vals


def run_decode(m, cache, q, lens, table, ws=None, scale=None):
    dims = cache.dims
    ws = m.attn_workspace(dims) if ws is None else ws
    o = torch.full((q.shape[0], dims.n_q_heads, dims.head_dim), 0x7FC0, dtype=torch.int16, device="cuda")
    lse = torch.full((q.shape[0], dims.n_q_heads), math.nan, device="cuda")
    m.attn_decode(cache, q, ints(lens), table, ws, o=o, lse=lse, scale=scale)
    assert status(m, ws) == 0
    return o, lse


def decode_ref(q, vals, scale):
    b, hq, d = q.shape
    g = hq // vals[0][0].shape[0]
    out = [torch.zeros(b, hq, d).double(), torch.zeros(b, hq).double(), torch.zeros(b, hq, d).double()]
    for i in range(b):
        for h in range(hq):
            k, v = vals[i][0][h // g], vals[i][1][h // g]
            r = C.attend(q[i, h:h + 1].double(), k, v, scale, torch.ones(1, len(k), dtype=torch.bool))
            for to, x in zip(out, r):
                to[i, h] = x[0]
    return out


def decode_case(m, heads, d, lens, page, fp8, seed=0, gain=2.0):
    dims = m.AttnDims(*heads, d)
    cache, table, vals = make_cache(m, dims, lens, page, fp8, seed)
    q = rand(seed + 7, len(lens), heads[0], d, gain=gain)
    o, lse = run_decode(m, cache, q.view(torch.int16).cuda(), lens, table)
    C.check(o, lse, decode_ref(q, vals, 1 / math.sqrt(d)), 11 if fp8 else 8, f"{heads} {d} {lens} {page} {fp8}")


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("lens,page", [([1], 16), ([0, 5, 0], 16), ([15, 16, 17, 33], 16), ([700], 64), ([129, 1, 64], 128),
                                       ([7, 300], 1), ([100, 55, 3], 48), ([513], 7)], ids=str)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_token_lengths_and_pages(m, d, lens, page, fp8):
    decode_case(m, (16, 2), d, lens, page, fp8)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("heads", HEADS + [(17, 1), (32, 2)], ids=str)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_token_heads(m, heads, d, fp8):
    decode_case(m, heads, d, [90, 33, 1], 16, fp8, seed=3)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_token_long_and_batched(m, fp8):
    decode_case(m, (4, 2), 128, [9001], 64, fp8, seed=4, gain=4.0)
    decode_case(m, (4, 4), 64, [(37 * i) % 211 for i in range(190)], 32, fp8, seed=5)
    decode_case(m, (8, 1), 256, [3000, 1, 0, 2999], 16, fp8, seed=6)


def test_token_batch_with_long_one(m):
    """More sequences than SMs and one that is far longer than the rest."""
    decode_case(m, (2, 1), 64, [3] * 100 + [20000] + [40] * 99, 16, False, seed=8)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_token_large_and_small_queries(m, fp8):
    """Queries far from 1 (fp16 holds neither end of bf16's range)."""
    dims, lens = m.AttnDims(4, 1, 64), [50, 20]
    cache, table, vals = make_cache(m, dims, lens, 16, fp8)
    for size in (1e-30, 1e6, 1e35):
        q = rand(3, 2, 4, 64) * size
        scale = float(1.0 / (8.0 * size))
        o, lse = run_decode(m, cache, q.view(torch.int16).cuda(), lens, table, scale=scale)
        C.check(o, lse, decode_ref(q, vals, scale), 11 if fp8 else 8, f"{size}")


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_token_small_weights(m, fp8):
    """Values behind weights of 2^-20 of the largest, whose own value is zero."""
    d, n, page = 64, 40, 16
    level = torch.full((n,), 0.4375)
    level[11] = 1.0
    k = level[None, :, None].expand(1, n, d).double()
    v = (torch.arange(n * d) % 29 - 14).reshape(1, n, d).double() / 8
    v[0, 11] = 0.0
    to = torch.float8_e4m3fn if fp8 else torch.bfloat16
    cells = [torch.zeros(3, 1, page, d, dtype=to) for _ in range(2)]
    for c, x in zip(cells, (k, v)):
        for i in range(n):
            c[i // page, 0, i % page] = x[0, i].to(to)
        assert torch.equal(torch.cat([c[i // page, 0, i % page][None] for i in range(n)]).double(), x[0])  # exact codes
    one = (torch.ones(1, device="cuda"),) * 2
    cache = m.KvCache(m.AttnDims(8, 1, d), *(c.view(torch.uint8 if fp8 else torch.int16).cuda() for c in cells),
                      *(one if fp8 else ()))
    q = torch.full((1, 8, d), 3.125).to(torch.bfloat16)   # scores 25 and 10.94
    o, lse = run_decode(m, cache, q.view(torch.int16).cuda(), [n], ints([[0, 1, 2]]))
    C.check(o, lse, decode_ref(q, [[k, v]], 1 / math.sqrt(d)), 11 if fp8 else 8)


def test_token_workspace_reused(m):
    """One workspace over calls of different batches; same call, same bits; another stream; a graph."""
    dims = m.AttnDims(16, 2, 128)
    ws = m.attn_workspace(dims)
    first = None
    for lens in ([5000, 3], [17] * 30, [1], [0], [2222, 1111, 4444], [5000, 3]):
        cache, table, vals = make_cache(m, dims, lens, 32, False, seed=len(lens))
        q = rand(1, len(lens), 16, 128)
        o, lse = run_decode(m, cache, q.view(torch.int16).cuda(), lens, table, ws)
        if lens == [5000, 3]:
            if first is None:
                first = o
                C.check(o, lse, decode_ref(q, vals, 1 / math.sqrt(128)), 8)
            else:
                assert torch.equal(first, o)
    qd, n, out = q.view(torch.int16).cuda(), ints(lens), torch.zeros_like(first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.attn_decode(cache, qd, n, table, ws, o=out)
    side.synchronize()
    assert torch.equal(first, out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.attn_decode(cache, qd, n, table, ws, o=out)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, out)


def test_token_bad_pages_and_lengths(m):
    dims = m.AttnDims(4, 2, 64)
    cache, table, _ = make_cache(m, dims, [100, 100], 16, False)
    q = rand(1, 2, 4, 64).view(torch.int16).cuda()
    for bad in (-1, 1 << 30, cache.k.shape[0]):
        t, ws = table.clone(), m.attn_workspace(dims)
        t[1, 3] = bad
        m.attn_decode(cache, q, ints([100, 100]), t, ws)
        assert status(m, ws) == 9 and status(m, ws) == 0
    for lens in ([100, -1], [100, 7 * 16 + 1], [1 << 30, 100]):
        ws = m.attn_workspace(dims)
        m.attn_decode(cache, q, ints(lens), table, ws)
        assert status(m, ws) == 9, lens


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_cache_far_offsets(m, fp8):
    """Pages more than 2^32 bytes into the cache, appended to and read back."""
    dims, page, lens = m.AttnDims(4, 2, 128), 64, [200]
    size = 1 if fp8 else 2
    n_pages = (5 << 30) // (2 * page * 128 * size)
    s = torch.tensor([0.02, 0.03], device="cuda") if fp8 else None
    cache = m.KvCache.empty(dims, n_pages, page, s, s)
    table = ints([[n_pages - 1, n_pages - 3, 0, n_pages - 2]])
    k, v, ws = rand(1, 200, 2, 128), rand(2, 200, 2, 128), m.attn_workspace(dims)
    m.kv_append(cache, k.view(torch.int16).cuda(), v.view(torch.int16).cuda(), cu([200]), ints([0]), table, ws)
    q = rand(3, 1, 4, 128)
    o, lse = run_decode(m, cache, q.view(torch.int16).cuda(), lens, table, ws)
    if fp8:
        sc = s.cpu()[None, :, None]
        k, v = (e4m3(x, sc).float().double() * sc.double() for x in (k, v))
    ref = decode_ref(q, [[k.double().transpose(0, 1), v.double().transpose(0, 1)]], 1 / math.sqrt(128))
    C.check(o, lse, ref, 11 if fp8 else 8)


# ------------------------------------------------------------------------------------ the append
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("new,start,page", [([1], [0], 16), ([3, 0, 40, 1], [5, 9, 14, 0], 16), ([1] * 70, list(range(70)), 32),
                                            ([200, 7], [1000, 3], 7)], ids=["one", "ragged", "tokens", "long"])
@pytest.mark.parametrize("hkv,d", [(2, 128), (1, 64), (3, 256), (5, 64), (8, 128), (40, 128)])
def test_append(m, hkv, d, new, start, page, fp8):
    dims = m.AttnDims(hkv, hkv, d)
    lens = [a + b for a, b in zip(new, start)]
    t, total = table_for(lens, page)
    n = sum(new)
    scales = torch.rand(2, hkv, generator=torch.Generator().manual_seed(1)) * 0.02 + 0.01
    cells = torch.randint(0, 100, (2, total, hkv, page, d), dtype=torch.uint8 if fp8 else torch.int16)
    x = rand(4, n, 2 * hkv, d)
    x[0, 0, :6] = torch.tensor([math.nan, math.inf, -math.inf, 1e30, -0.0, 1e-30])
    cache = m.KvCache(dims, cells[0].cuda(), cells[1].cuda(), *((scales[0].cuda(), scales[1].cuda()) if fp8 else ()))
    rows, ws = x.view(torch.int16).cuda(), m.attn_workspace(dims)
    m.kv_append(cache, rows[:, :hkv], rows[:, hkv:], cu(new), ints(start), t.cuda(), ws)
    assert status(m, ws) == 0
    want, r = cells.clone(), 0
    for b, c in enumerate(new):
        for i in range(c):
            pos = start[b] + i
            for s in range(2):
                y = x[r, s * hkv:(s + 1) * hkv]
                want[s, t[b, pos // page], :, pos % page] = (e4m3(y, scales[s][:, None]).view(torch.uint8) if fp8
                                                             else y.view(torch.int16))
            r += 1
    got = torch.stack([cache.k.cpu(), cache.v.cpu()])
    if fp8:  # a NaN may carry either sign
        got, want = (torch.where((y & 0x7F) == 0x7F, torch.full_like(y, 0x7F), y) for y in (got, want))
    assert torch.equal(got, want)


def test_append_bad_places(m):
    """Rows without a place are skipped, the others written."""
    dims = m.AttnDims(2, 2, 64)
    k = rand(1, 4, 2, 64).view(torch.int16).cuda()
    for start, table, cuq in (([60, 0], [[0, 1], [2, 3]], [0, 2, 4]), ([-3, 0], [[0, 1], [2, 3]], [0, 2, 4]),
                              ([0, 0], [[9, 1], [2, 3]], [0, 2, 4]), ([0, 0], [[-1, 1], [2, 3]], [0, 2, 4]),
                              ([0, 0], [[0, 1], [2, 3]], [0, 5, 3]), ([0, 0], [[0, 1], [2, 3]], [1, 2, 4])):
        cache, ws = m.KvCache.empty(dims, 4, 16), m.attn_workspace(dims)
        cache.k.fill_(7), cache.v.fill_(7)
        m.kv_append(cache, k, k, ints(cuq), ints(start), ints(table), ws)
        assert status(m, ws) == 9, (start, table, cuq)
        if cuq == [0, 2, 4]:
            assert torch.equal(cache.k[2, :, 0], k[2]) and torch.equal(cache.v[2, :, 1], k[3])
            assert (cache.k[:2] == 7).all()


# ------------------------------------------------------------------------------------ together
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_prompt_then_tokens(m, fp8):
    """A prompt's keys and values appended to the cache, then new tokens one by one: each token's
    output is the last row of attention over the whole text so far."""
    dims, page, d = m.AttnDims(4, 2, 128), 16, 128
    lens, steps = [45, 3], 3
    scale = torch.tensor([0.02, 0.015])
    q, k, v = (rand(i, len(lens), 60, h, d) for i, h in ((1, 4), (2, 2), (3, 2)))
    ws = m.attn_workspace(dims)
    s = scale.cuda() if fp8 else None
    cache = m.KvCache.empty(dims, 10, page, s, s)
    table = ints([[3, 9, 1, 0], [5, 2, 8, 7]])
    pack = lambda x: torch.cat([x[b, :n] for b, n in enumerate(lens)]).view(torch.int16).cuda()  # noqa: E731
    c = cu(lens)
    m.attn_prefill(dims, pack(q), pack(k), pack(v), c, c, ws)
    m.kv_append(cache, pack(k), pack(v), c, ints([0, 0]), table, ws)
    if fp8:
        k, v = ((e4m3(x, scale[:, None]).float() * scale[:, None]).double() for x in (k, v))
    at = list(lens)
    one = ints([0, 1, 2])
    for _ in range(steps):
        row = lambda x: torch.stack([x[b, n] for b, n in enumerate(at)])  # noqa: E731
        if fp8:  # the new rows before rounding
            kn, vn = (torch.stack([rand(i, len(lens), 60, 2, d)[b, n] for b, n in enumerate(at)]) for i in (2, 3))
        else:
            kn, vn = row(k), row(v)
        m.kv_append(cache, kn.view(torch.int16).cuda(), vn.view(torch.int16).cuda(), one, ints(at), table, ws)
        at = [n + 1 for n in at]
        qn = torch.stack([q[b, n - 1] for b, n in enumerate(at)])
        o, lse = run_decode(m, cache, qn.view(torch.int16).cuda(), at, table, ws)
        vals = [[x[b, :n].double().transpose(0, 1) for x in (k, v)] for b, n in enumerate(at)]
        C.check(o, lse, decode_ref(qn, vals, 1 / math.sqrt(d)), 11 if fp8 else 8)


def test_binding_refusals(m):
    dims = m.AttnDims(4, 2, 64)
    q, kv = (torch.zeros(5, h, 64, dtype=torch.int16, device="cuda") for h in (4, 2))
    c, ws = cu([5]), m.attn_workspace(dims)
    cache = m.KvCache.empty(dims, 4, 16)
    table, lens = torch.zeros(5, 1, dtype=torch.int32, device="cuda"), ints([1] * 5)

    def prefill(q=q, k=kv, v=kv, cu_q=c, cu_k=c, ws=ws, **kw):
        m.attn_prefill(dims, q, k, v, cu_q, cu_k, ws, **kw)

    def decode(q=q, lens=lens, table=table, ws=ws, **kw):
        m.attn_decode(cache, q, lens, table, ws, **kw)

    def append(k=kv, v=kv, cu_=c, start=ints([0]), table=table[:1], ws=ws):
        m.kv_append(cache, k, v, cu_, start, table, ws)

    prefill(), decode(), append()
    for call in (prefill, decode, append):
        for bad in (ws.cpu(), ws.view(torch.int16), ws[::2]):
            with pytest.raises(ValueError):
                call(ws=bad)
        with pytest.raises(m.MoeError):
            call(ws=ws[:128])
    for kw in (dict(q=q[:, :3]), dict(q=q.float()), dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)), dict(v=kv[:4]),
               dict(cu_k=cu([5, 0])), dict(cu_q=c.long()), dict(o=torch.empty_like(q[:4])), dict(o=q.cpu()),
               dict(lse=torch.empty(4, 5, device="cuda").t()), dict(lse=torch.empty(5, 3, device="cuda"))):
        with pytest.raises(ValueError):
            prefill(**kw)
    for kw in (dict(lens=lens[:4]), dict(table=table[:4]), dict(table=table[:, 0]), dict(q=q.cpu()),
               dict(lens=lens.float()), dict(o=torch.empty(5, 64, 4, dtype=torch.int16, device="cuda"))):
        with pytest.raises(ValueError):
            decode(**kw)
    for kw in (dict(k=kv[:4]), dict(start=ints([0, 0])), dict(table=table), dict(cu_=c.cpu())):
        with pytest.raises(ValueError):
            append(**kw)
    assert status(m, ws) == 0


@pytest.mark.parametrize("lens", [[700], [20000], [0, 40, 9001, 3]], ids=str)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_token_infinite_values_seen(m, d, lens):
    """An infinite value in a sequence that is cut over warps and SMs gives an infinite output, wherever it
    lies (the last key too, which the last part holds), and changes no other column."""
    dims, at = m.AttnDims(4, 2, d), max(range(len(lens)), key=lambda b: lens[b])
    n = lens[at]
    cache, table, vals = make_cache(m, dims, lens, 16, False, seed=31)
    where = {0: n - 1, 5: 0, 6: n // 2, d - 1: n - 2}                 # column -> key
    for i, (c, key) in enumerate(where.items()):
        bad = math.inf if i % 2 == 0 else -math.inf
        cache.v[table[at, key // 16].long(), :, key % 16, c] = -128 if bad < 0 else 0x7F80  # 0xFF80, 0x7F80
        vals[at][1][:, key, c] = 0.0
    q = rand(33, len(lens), 4, d, gain=0.5)
    o, lse = run_decode(m, cache, q.view(torch.int16).cuda(), lens, table)
    ref, got = decode_ref(q, vals, 1 / math.sqrt(d)), C.values(o)
    for i, c in enumerate(where):
        assert (got[at, :, c] == (math.inf if i % 2 == 0 else -math.inf)).all(), (c, got[at, :, c])
        got[at, :, c] = ref[0][at, :, c]
    C.check(got.to(torch.bfloat16).view(torch.int16), lse, ref, 8, f"{d} {lens}")


@pytest.mark.parametrize("less", [0, 1], ids=["whole_tiles", "ragged"])
def test_prompt_item_longer_than_a_wait(m, less):
    """A row over 100 million keys of 256 values: its one item takes longer than any single wait may (2e9 cycles;
    64 keys take 1600). Three keys, the first and the last among them, have all the weight."""
    d, n, lk = 256, 100_000_000, 100_000_000 - less
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 51 GB of keys")
    rows = torch.zeros((n, 1, d), dtype=torch.int16, device="cuda")     # keys and values alike
    q = torch.zeros(1, 1, d, dtype=torch.bfloat16)
    q[..., :16] = 10.0
    x = rand(1, 3, 1, d)
    x[..., :16] = 8.0                                                   # a score of 80, and 0 for every other key
    for at, row in zip((0, 31_234_567, lk - 1), x):
        rows[at] = row.view(torch.int16).cuda()
    k = rows[:lk]
    o, lse = run_prefill(m, m.AttnDims(1, 1, d), q.view(torch.int16).cuda(), k, k, [(1, lk)], False)
    del rows, k
    torch.cuda.empty_cache()
    C.check(o, lse, [x.double().mean(0)[None], torch.tensor([[80 + math.log(3)]]).double(),
                     x.double().abs().mean(0)[None]], 8)


def long_context_case(m, heads, d, lens, causal, seed, shape=None, sel=None):
    """Values of one sign (what the sums lose would show) behind long contexts, made and checked on the GPU: `sel` rows
    of the first and last head. shape(position / length), 0..1, adds up to 40 to the scores: as one exact product, the last
    of a score, so that its rounding (2^-22 of at most 640, scaled by 1/16) stays within the scores' tolerance."""
    (hq, hkv), g = heads, torch.Generator(device="cuda").manual_seed(seed)
    tq, tk = sum(x for x, _ in lens), sum(x for _, x in lens)
    q = (torch.randn(tq, hq, d, generator=g, device="cuda") * 0.5).to(torch.bfloat16)
    if shape is not None:
        q[:, :, d - 1] = 4.0
    k = torch.empty((tk, hkv, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    for i in range(0, tk, 1 << 18):
        n = min(1 << 18, tk - i)
        k[i:i + n] = torch.randn(n, hkv, d, generator=g, device="cuda")
        if shape is not None:
            k[i:i + n, :, d - 1] = torch.round(10 * math.sqrt(d) * shape(torch.arange(i, i + n, device="cuda") / tk))[:, None]
        v[i:i + n] = torch.rand(n, hkv, d, generator=g, device="cuda") + 0.5
    o, lse = run_prefill(m, m.AttnDims(hq, hkv, d), *(x.view(torch.int16) for x in (q, k, v)), lens, causal)
    a = b = 0
    for lq, lk in lens:
        rows = torch.tensor(range(lq) if sel is None else [r % lq for r in sel], device="cuda")
        for h in {0, hq - 1}:
            qd, top = q[a + rows, h].double(), torch.full((len(rows),), -math.inf, dtype=torch.float64, device="cuda")
            acc, den = torch.zeros(len(rows), d, dtype=torch.float64, device="cuda"), torch.zeros_like(top)
            for i in range(0, lk, 1 << 18):  # the definition, a running maximum over long pieces
                n, kv = min(1 << 18, lk - i), h // (hq // hkv)
                s = qd @ k[b + i:b + i + n, kv].double().t() / math.sqrt(d)
                if causal:
                    s.masked_fill_(torch.arange(i, i + n, device="cuda")[None] > (rows + lk - lq)[:, None], -math.inf)
                t2 = torch.maximum(top, s.amax(1))
                p, f = torch.exp(s - t2[:, None]), torch.exp(top - t2)
                acc, den, top = acc * f[:, None] + p @ v[b + i:b + i + n, kv].double(), den * f + p.sum(1), t2
            ref = [(acc / den[:, None]).cpu(), (top + den.log()).cpu(), (acc / den[:, None]).cpu()]
            C.check(o[a + rows, h], lse[a + rows, h], ref, 8, f"{heads} {d} {lq} on {lk}, head {h}")
        a, b = a + lq, b + lk


@pytest.mark.parametrize("heads,d,lens,causal", [
    ((2, 1), 64, [(3, 4_000_000)], True), ((2, 1), 128, [(3, 4_000_001)], False), ((2, 1), 256, [(3, 4_000_000)], True),
    ((64, 8), 64, [(1300, 3_000_000)], True), ((64, 8), 128, [(1300, 3_000_001)], False)], ids=str)
def test_prompt_millions_of_keys(m, heads, d, lens, causal):
    """The tensor cores' sums lose a little with every product; over millions of keys it may not add up."""
    long_context_case(m, heads, d, lens, causal, seed=3, sel=(0, 130, 1299))
    torch.cuda.empty_cache()


@pytest.mark.parametrize("shape", [None, lambda x: x, lambda x: 1 - x, lambda x: 1.0 * (x > 0.5)],
                         ids=["flat", "rising", "falling", "step"])
@pytest.mark.parametrize("heads,causal", [((16, 2), True), ((7, 1), False), ((2, 2), True)], ids=str)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompt_long_contexts(m, d, heads, causal, shape):
    """Around the lengths at which sums are put aside (32768 keys of a stream of key tiles), with maxima that move."""
    long_context_case(m, heads, d, [(3, 32768), (20, 65536), (1, 65700), (33, 131073), (5, 40)], causal, 5, shape)
    many = (48 * heads[0] // heads[1], 48)                       # two row tiles to an item
    long_context_case(m, many, d, [(300, 32900), (301, 70001)], causal, 6, shape, sel=(0, 150, 299))


# ------------------------------------------------------------------------------------ forms chosen by size
RAGGED = [(0, 0), (1, 1), (37, 37), (5, 133), (40, 7), (33, 161), (3, 0), (64, 64), (130, 129), (0, 3), (17, 90)]


def two_row_tiles(m, heads, lens):
    """Enough rows for two row tiles to a CTA: at least two such items per SM."""
    hq, hkv = heads
    rows = 2 * (128 // (hq // hkv))
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return sum(x for x, _ in lens) // rows * hkv >= 2 * sms


def some_heads_case(m, heads, d, lens, causal, seed, gain=2.0):
    """The first and last head of the first and last group against 64 bits; all rows, all columns."""
    hq, hkv = heads
    g, tq, tk = hq // hkv, sum(x for x, _ in lens), sum(x for _, x in lens)
    q, k, v = rand(seed, tq, hq, d, gain=gain), rand(seed + 1, tk, hkv, d), rand(seed + 2, tk, hkv, d)
    o, lse = run_prefill(m, m.AttnDims(hq, hkv, d), *(x.view(torch.int16).cuda() for x in (q, k, v)), lens, causal)
    assert torch.isfinite(o.view(torch.bfloat16)).all()
    for h in (0, hkv - 1):
        sel = sorted({h * g, h * g + g - 1})
        ref = C.prefill(q[:, sel].double(), k[:, h:h + 1].double(), v[:, h:h + 1].double(), lens, 1 / math.sqrt(d), causal)
        C.check(o[:, sel], lse[:, sel], ref, 8, f"{heads} {d} causal={causal} heads {sel}")


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "both"])
@pytest.mark.parametrize("heads,times", [((64, 8), 4), ((56, 8), 5), ((48, 16), 5)], ids=["8", "7", "3"])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_two_row_tiles_ragged(m, d, heads, times, causal):
    """Many short sequences with two row tiles to an item: rows that see nothing, tiles without a position,
    groups that do not divide 128."""
    lens = RAGGED * times
    assert two_row_tiles(m, heads, lens)
    some_heads_case(m, heads, d, lens, causal, seed=60)


@pytest.mark.parametrize("heads,lens,causal", [
    ((64, 8), [(1300, 1300)], True), ((64, 8), [(1251, 1400)], False), ((56, 8), [(1411, 1500)], True),
    ((48, 16), [(1601, 1500)], True), ((48, 16), [(1650, 70)], False), ((64, 8), [(1300, 128), (33, 256)], False)],
    ids=str)
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_two_row_tiles_long(m, d, heads, lens, causal):
    assert two_row_tiles(m, heads, lens)
    some_heads_case(m, heads, d, lens, causal, seed=70, gain=4.0)


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "both"])
@pytest.mark.parametrize("d", [64, 256])
def test_prompt_thousands_of_sequences(m, d, causal):
    prompt_case(m, (2, 1), d, [((i * 5) % 4, (i * 7) % 9) for i in range(4096)], causal, seed=80)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_token_thousands_of_sequences(m, fp8):
    """All 128 groups of 32 sequences, some of them empty, long sequences among the short ones."""
    lens = [0 if 640 <= i < 704 or i % 7 == 3 else 3000 if i % 1500 == 9 else i % 23 for i in range(4096)]
    decode_case(m, (2, 1), 64, lens, 16, fp8, seed=90)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("heads", [(64, 1), (12, 1), (40, 2)], ids=str)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_token_many_heads_long(m, d, heads, fp8):
    """More than 8 and more than 16 query heads to a cache head, cut over warps and SMs."""
    decode_case(m, heads, d, [1501, 3, 260], 16, fp8, seed=95)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompt_odd_strides(m, d):
    """A token stride that is no multiple of the head stride."""
    hq, hkv, n = 4, 2, 130
    q, k, v = rand(1, n, hq, d), rand(2, n, hkv, d), rand(3, n, hkv, d)
    dev = []
    for x in (q, k, v):
        h = x.shape[1]
        buf = torch.full((n * (h * (d + 8) + 40),), 0x7FC0, dtype=torch.int16, device="cuda")
        dev.append(buf.as_strided((n, h, d), (h * (d + 8) + 40, d + 8, 1)))
        dev[-1].copy_(x.view(torch.int16).cuda())
    o, lse = run_prefill(m, m.AttnDims(hq, hkv, d), *dev, [(n, n)], True)
    C.check(o, lse, C.prefill(q.double(), k.double(), v.double(), [(n, n)], 1 / math.sqrt(d), True), 8)


# ------------------------------------------------------------------------------------ bad device data
def guarded(shape, dtype, fill):
    """A tensor of `fill` inside a buffer of the same value, 4096 elements on either side; and a check of these."""
    n = math.prod(shape)
    buf = torch.full((n + 8192,), fill, dtype=dtype, device="cuda")

    def untouched():
        return bool((buf[:4096] == fill).all() and (buf[-4096:] == fill).all())
    return buf[4096:-4096].view(shape), untouched


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("cq,ck,good", [
    ([0, 30, 20, 40], [0, 30, 30, 40], []), ([0, 10, 20, 400], [0, 10, 20, 40], [0, 1]),
    ([0, 10, 20, 40], [0, 10, 20, 1000000], [0, 1]), ([0, 10, 20, 40], [0, 10, 1 << 30, 40], [0]),
    ([0, 10, 20, 1 << 30], [0, 10, 20, 40], [0, 1]), ([0, 10, 20, 40], [0, -1000000, 20, 40], [2])])
def test_prompt_bad_offsets_margins(m, d, cq, ck, good):
    """Bad offsets write nothing outside o and lse, and leave the sequences beside them right."""
    dims = m.AttnDims(4, 2, d)
    x = rand(1, 40, 8, d)
    dev, ws = x.view(torch.int16).cuda(), m.attn_workspace(dims)
    o, o_ok = guarded((40, 4, d), torch.int16, 0x1234)
    lse, lse_ok = guarded((40, 4), torch.float32, 7.25)
    m.attn_prefill(dims, dev[:, :4], dev[:, 4:6], dev[:, 6:], ints(cq), ints(ck), ws, o=o, lse=lse)
    assert status(m, ws) == 9
    assert o_ok() and lse_ok()
    for b in good:
        (a, z), (s, e) = cq[b:b + 2], ck[b:b + 2]
        z = min(z, 40)
        ref = C.prefill(x[a:z, :4].double(), x[s:e, 4:6].double(), x[s:e, 6:].double(), [(z - a, e - s)], 1 / math.sqrt(d), True)
        C.check(o[a:z], lse[a:z], ref, 8, f"sequence {b}")


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_token_bad_pages_and_lengths_margins(m, fp8):
    """Bad pages and lengths write nothing outside o and lse, and leave the other sequences right."""
    dims, lens = m.AttnDims(4, 2, 64), [100, 90, 1000]
    cache, table, vals = make_cache(m, dims, lens, 16, fp8)
    q = rand(1, 3, 4, 64)
    ref = decode_ref(q, vals, 1 / 8)
    for page, n in ((-1, 90), (1 << 30, 90), (cache.k.shape[0], 90), (None, -1), (None, 1 << 30), (None, 63 * 16 + 1)):
        t, ws = table.clone(), m.attn_workspace(dims)
        if page is not None:
            t[1, 3] = page
        o, o_ok = guarded((3, 4, 64), torch.int16, 0x1234)
        lse, lse_ok = guarded((3, 4), torch.float32, 7.25)
        m.attn_decode(cache, q.view(torch.int16).cuda(), ints([100, n, 1000]), t, ws, o=o, lse=lse)
        assert status(m, ws) == 9, (page, n)
        assert o_ok() and lse_ok()
        C.check(o[::2], lse[::2], [x[::2] for x in ref], 11 if fp8 else 8, f"{page} {n}")


# ------------------------------------------------------------------------------------ seen infinities, ends of ranges
@pytest.mark.parametrize("heads,n", [((4, 2), 700), ((64, 8), 1300)], ids=str)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompt_infinite_values_seen(m, d, heads, n):
    """Rows that see an infinite value have it in their output, in that column only."""
    hq, hkv = heads
    q, k, v = rand(1, n, hq, d, gain=0.5), rand(2, n, hkv, d), rand(3, n, hkv, d)
    where = {0: n - 3, 5: 0, 6: n // 2, d - 1: n - 140}                # column -> key
    vb = v.clone()
    for i, (c, key) in enumerate(where.items()):
        vb[key, :, c], v[key, :, c] = math.inf if i % 2 == 0 else -math.inf, 0.0
    o, lse = run_prefill(m, m.AttnDims(hq, hkv, d), *(x.view(torch.int16).cuda() for x in (q, k, vb)), [(n, n)], True)
    sel, g = [0, hq - 1], hq // hkv
    for h in sel:
        ref = C.prefill(q[:, h:h + 1].double(), k[:, h // g:h // g + 1].double(), v[:, h // g:h // g + 1].double(), [(n, n)],
                        1 / math.sqrt(d), True)
        got = C.values(o[:, h:h + 1])
        for i, (c, key) in enumerate(where.items()):
            assert (got[key:, :, c] == (math.inf if i % 2 == 0 else -math.inf)).all(), (h, c)
            got[key:, :, c] = ref[0][key:, :, c]
        C.check(got.to(torch.bfloat16).view(torch.int16), lse[:, h:h + 1], ref, 8, f"{heads} {d} head {h}")


@pytest.mark.parametrize("d", [64, 128, 256])
def test_infinite_keys_seen(m, d):
    """A key whose score is minus infinity has no weight, in a prompt and in the cache."""
    n, at = 300, [0, 17, 255, 299]
    q, k, v = rand(1, n, 2, d, gain=0.5), rand(2, n, 1, d), rand(3, n, 1, d)
    q[:, :, 3] = -1.0
    rest = torch.tensor([i for i in range(n) if i not in at])
    k[at, 0, 3] = math.inf
    o, lse = run_prefill(m, m.AttnDims(2, 1, d), *(x.view(torch.int16).cuda() for x in (q, k, v)), [(n, n)], False)
    ref = C.prefill(q.double(), k[rest].double(), v[rest].double(), [(n, len(rest))], 1 / math.sqrt(d), False)
    C.check(o, lse, ref, 8)
    cache, ws = m.KvCache.empty(m.AttnDims(2, 1, d), 20, 16), m.attn_workspace(m.AttnDims(2, 1, d))
    table = torch.arange(19, dtype=torch.int32, device="cuda")[None].contiguous()
    m.kv_append(cache, k.view(torch.int16).cuda(), v.view(torch.int16).cuda(), cu([n]), ints([0]), table, ws)
    o, lse = run_decode(m, cache, q[:1].view(torch.int16).cuda(), [n], table, ws)
    C.check(o, lse, [x[:1] for x in ref], 8)


@pytest.mark.parametrize("heads", [(1024, 16), (1024, 1024), (1023, 1023)], ids=str)
@pytest.mark.parametrize("d", [64, 256])
def test_most_heads(m, d, heads):
    """As many heads as are accepted: a prompt, its append, and one token; the first, a middle and the last group."""
    (hq, hkv), n, page = heads, 35, 16
    g, dims = hq // hkv, m.AttnDims(hq, hkv, d)
    q, k, v = rand(1, n, hq, d), rand(2, n, hkv, d), rand(3, n, hkv, d)
    dev = [x.view(torch.int16).cuda() for x in (q, k, v)]
    o, lse = run_prefill(m, dims, *dev, [(n, n)], True)
    cache, ws, table = m.KvCache.empty(dims, 4, page), m.attn_workspace(dims), ints([[2, 0, 3]])
    m.kv_append(cache, dev[1], dev[2], cu([n]), ints([0]), table, ws)
    o1, lse1 = run_decode(m, cache, dev[0][-1:].contiguous(), [n], table, ws)
    for h in (0, hkv // 2, hkv - 1):
        sel = sorted({h * g, h * g + g - 1})
        ref = C.prefill(q[:, sel].double(), k[:, h:h + 1].double(), v[:, h:h + 1].double(), [(n, n)], 1 / math.sqrt(d), True)
        C.check(o[:, sel], lse[:, sel], ref, 8, f"prompt {h}")
        C.check(o1[:, sel], lse1[:, sel], [x[-1:] for x in ref], 8, f"token {h}")


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_largest_pages(m, fp8):
    """Pages of 65536 rows, a length that fills the table."""
    dims, page, n = m.AttnDims(2, 1, 64), 65536, 131072
    s = torch.tensor([0.02], device="cuda") if fp8 else None
    cache, ws = m.KvCache.empty(dims, 3, page, s, s), m.attn_workspace(dims)
    k, v, q = rand(1, n, 1, 64), rand(2, n, 1, 64), rand(3, 1, 2, 64)
    table = ints([[2, 0]])
    m.kv_append(cache, k.view(torch.int16).cuda(), v.view(torch.int16).cuda(), cu([n]), ints([0]), table, ws)
    o, lse = run_decode(m, cache, q.view(torch.int16).cuda(), [n], table, ws)
    if fp8:
        k, v = (e4m3(x, 0.02).float().double() * float(s[0]) for x in (k, v))
    C.check(o, lse, decode_ref(q, [[k.double().transpose(0, 1), v.double().transpose(0, 1)]], 1 / 8), 11 if fp8 else 8)


@pytest.mark.parametrize("heads,tokens,d", [((16, 2), 20, 64), ((16, 2), 20, 128), ((16, 2), 20, 256), ((64, 8), 1300, 128)],
                         ids=str)
def test_prompt_long_same_bits(m, heads, tokens, d):
    """Sums put aside along a long context: the same bits from call to call."""
    (hq, hkv), n = heads, 140_000
    g = torch.Generator(device="cuda").manual_seed(7)
    q, k, v = ((torch.randn(r, h, d, generator=g, device="cuda")).to(torch.bfloat16).view(torch.int16)
               for r, h in ((tokens + 3, hq), (n + 90, hkv), (n + 90, hkv)))
    dims, cq, ck = m.AttnDims(hq, hkv, d), cu([tokens, 3]), cu([n, 90])
    ws, first = m.attn_workspace(dims), None
    for _ in range(5):
        lse = torch.empty(tokens + 3, hq, device="cuda")
        got = m.attn_prefill(dims, q, k, v, cq, ck, ws, lse=lse), lse
        first = first or got
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])
