"""The measured cases of the 8-bit expert operators: tokens sorted by expert and brought back with
their weights, both with their gradients; matrix products of e4m3 rows with e4m3 weights that carry
a scale for each block of 128; and the SwiGLU activation between two such products, with its gradient.

Every case runs in two forms. The plain form (own = False) is elementary torch arithmetic in 32
bits; the other calls the package's entry points as a program does that runs, or trains through,
experts held in 8 bits. bf16 tensors travel as int16 bit patterns, as everywhere in this package.

Eight bits: e4m3 codes of a row carry one fp32 scale per 128 columns (the last block may be
shorter), a weight matrix one per block of 128 x 128; a code c stands for scale * c. Quantising a
block of a row takes a = the largest finite magnitude, at least 2^-100; the scale is a / 448, a code
x * (448 / a) rounded to e4m3, NaN for a value that is not finite.

Shapes: hidden size 2048, 256 experts of 512, 8 to a token, is the layer of this package's pages and
benchmark, and 512, 2048 and 4096 tokens its prefill lengths; the other sizes are generic.
"""
import math
import random

import torch

own = False

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn
FLOPS = 2 * 8191 * 8192 * 8192     # of the largest listed product
ROW_BYTES = 16383 * 8 * 2048       # 8-bit values of the largest listed sorted batch


# ------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # a small decode batch: latency of sorting eight tokens and laying out their rows
        dict(name="sort_8", op="sort", tokens=8, k=8, experts=256, d=2048, e4m3=False, absent=0.0),
        # a long prompt, padded at the end of its batch: the padding's rows belong to no expert
        dict(name="sort_16383", op="sort", tokens=16383, k=8, experts=256, d=2048, e4m3=True, absent=0.03),
        # the same decode batch on its way back, added to the shared expert's rows
        dict(name="back_8", op="back", tokens=8, k=8, experts=256, d=2048, add=True, weighted=True, absent=0.0),
        # the benchmark's prefill on its way back
        dict(name="back_4096", op="back", tokens=4096, k=8, experts=256, d=2048, add=False, weighted=True, absent=0.0),
        # gradients of the rows and of the routing weights, for a batch of odd length
        dict(name="grad_513", op="grad", tokens=513, k=8, experts=256, d=2048, e4m3=False, absent=0.0),
        # the same for a training batch, the rows' gradients in 8 bits for the product that follows
        dict(name="grad_16383", op="grad", tokens=16383, k=8, experts=256, d=2048, e4m3=True, absent=0.03),
        # one token through its 8 experts' gate and up projections: a weight-bound product, latency counts
        dict(name="product_token", op="product", rows=8, experts=256, n=1024, k=2048, transposed=False, skew=0.0),
        # the benchmark's prefill through the same projections
        dict(name="product_4096", op="product", rows=32768, experts=256, n=1024, k=2048, transposed=False, skew=0.5),
        # the gradient of the down projections' inputs, 2048 tokens whose experts are uneven
        dict(name="product_back", op="product", rows=16384, experts=256, n=2048, k=512, transposed=True, skew=1.2),
        # a dense layer over a long batch of odd length: the arithmetic's rate
        dict(name="product_dense", op="product", rows=8191, experts=1, n=8192, k=8192, transposed=False, skew=0.0),
        # the activation between the two products of the benchmark's prefill, in 8 bits for the second
        dict(name="swiglu_32768", op="swiglu", rows=32768, inter=512, grad=False, e4m3=True, tail=0),
        # its gradient, for fewer rows than the buffers hold
        dict(name="swiglu_grad", op="swiglu", rows=16384, inter=512, grad=True, e4m3=True, tail=491),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["sort", "back", "grad", "product", "product", "product", "swiglu"])
    experts = rng.choice([8, 16, 60, 128, 256, 256, 512])
    if op in ("sort", "back", "grad"):
        k = rng.choice([1, 2, 4, 6, 8, 8, 10])
        case = dict(op=op, tokens=_log(rng, 1, 32768), k=min(k, experts), experts=experts,
                    d=16 * _log(rng, 8, 512), absent=rng.choice([0.0, 0.0, 0.1, 0.6]))
        if op == "back":
            case.update(add=rng.random() < 0.5, weighted=rng.random() < 0.7)
        else:
            case.update(e4m3=rng.random() < 0.5)
        while case["tokens"] * case["k"] * case["d"] > ROW_BYTES:
            case["tokens"] = max(1, case["tokens"] // 2)
    elif op == "product":
        case = dict(op=op, rows=_log(rng, 1, 32768), experts=rng.choice([1, 1, experts]), n=16 * _log(rng, 8, 512),
                    k=16 * _log(rng, 8, 512), transposed=rng.random() < 0.35, skew=rng.choice([0.0, 0.5, 1.2]))
        while case["experts"] * case["n"] * case["k"] > 256 * 1024 * 2048:
            case.update(n=max(128, case["n"] // 32 * 16), k=max(128, case["k"] // 32 * 16))
        while 2 * case["rows"] * case["n"] * case["k"] > FLOPS:
            case["rows"] = max(1, case["rows"] // 2)
    else:
        case = dict(op=op, rows=_log(rng, 1, 65536), inter=16 * _log(rng, 8, 512), grad=rng.random() < 0.5,
                    e4m3=rng.random() < 0.6)
        while case["rows"] * case["inter"] > 32768 * 512:
            case["rows"] = max(1, case["rows"] // 2)
        case["tail"] = rng.choice([0, case["rows"] // 7])
    return case


def _counts(case):
    """Rows of every expert: drawn by a popularity that is even (skew 0) or uneven; few rows go to
    experts of their own, as one token's do."""
    rows, E = case["rows"], case["experts"]
    if E == 1:
        return [rows]
    rng = random.Random(rows * 1000003 + E * 1009 + case["n"])
    counts = [0] * E
    if rows * 16 <= E:
        for e in rng.sample(range(E), rows):
            counts[e] = 1
        return counts
    w = [math.exp(rng.gauss(0.0, case["skew"])) for _ in range(E)]
    for e in rng.choices(range(E), w, k=rows):
        counts[e] += 1
    return counts


def _blocks(n):
    return (n + 127) // 128


def _absent(case):
    """Tokens at the end of the batch that no expert sees."""
    return min(case["tokens"] - 1, int(case["absent"] * case["tokens"]))


def work(case):
    op = case["op"]
    if op == "product":
        E, n, k, rows = case["experts"], case["n"], case["k"], case["rows"]
        hit = sum(1 for c in _counts(case) if c)
        a, o = (n, k) if case["transposed"] else (k, n)
        return {"bytes": rows * (a + 4 * _blocks(a) + 2 * o) + hit * (n * k + 4 * _blocks(n) * _blocks(k)) +
                (4 * (E + 1) if E > 1 else 0), "flops": 2 * rows * n * k}
    if op == "swiglu":
        I, rows = case["inter"], case["rows"] - case["tail"]
        cols = 2 * I if case["grad"] else I
        return {"bytes": rows * (4 * I + (2 * I if case["grad"] else 0) +
                                 (cols + 4 * _blocks(cols) if case["e4m3"] else 2 * cols)),
                "flops": rows * I * (14 if case["grad"] else 6)}
    T, k, d = case["tokens"], case["k"], case["d"]
    there = (T - _absent(case)) * k
    if op == "back":
        return {"bytes": there * 2 * d + T * 2 * d * (2 if case["add"] else 1) +
                4 * T * k * (2 if case["weighted"] else 1), "flops": 2 * there * d}
    out = d + 4 * _blocks(d) if case["e4m3"] else 2 * d
    if op == "sort":
        return {"bytes": (T - _absent(case)) * 2 * d + there * out + 12 * T * k + 4 * (case["experts"] + 1), "flops": 0}
    return {"bytes": (T - _absent(case)) * 2 * d + there * (2 * d + out) + 12 * T * k, "flops": 3 * there * d}


# ------------------------------------------------------------------------------------ the inputs
def _ids(case, gen):
    """Experts of every token, distinct, uneven in popularity; -1 for the tokens at the end that have none."""
    T, k, E = case["tokens"], case["k"], case["experts"]
    scores = torch.randn((T, E), generator=gen, device="cuda") + 0.7 * torch.randn(E, generator=gen, device="cuda")
    ids = torch.topk(scores, k, dim=1).indices.to(torch.int32)
    ids[T - _absent(case):] = -1
    return ids


def _sorted_places(ids, E):
    """offsets, perm, inv of assignments sorted by expert; those without an expert come last and have
    no place (-1)."""
    flat = ids.reshape(-1).long()
    key = torch.where(flat < 0, E, flat)
    order = torch.argsort(key, stable=True)
    counts = torch.zeros(E + 1, dtype=torch.int64, device="cuda").index_add_(0, key, torch.ones_like(key))
    offsets = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = counts[:E].cumsum(0)
    place = torch.empty_like(order)
    place[order] = torch.arange(len(order), device="cuda")
    inv = torch.where(flat < 0, -1, place).to(torch.int32).view(ids.shape)
    perm = torch.where(torch.arange(len(order), device="cuda") < offsets[E], order, -1).to(torch.int32)
    return offsets.to(torch.int32), perm, inv


def _bits(x):
    return x.to(BF16).view(torch.int16)


def _codes(shape, gen, size):
    """e4m3 codes of normal values, made in pieces."""
    n = math.prod(shape)
    q = torch.empty(n, dtype=torch.uint8, device="cuda")
    step = 1 << 26
    for i in range(0, n, step):
        x = torch.randn(min(step, n - i), generator=gen, device="cuda").mul_(size).clamp_(-448.0, 448.0)
        q[i:i + step] = x.to(E4M3).view(torch.uint8)
    return q.view(shape)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, s = case["op"], dict(case)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def uniform(lo, hi, *shape):
        return lo + (hi - lo) * torch.rand(shape, generator=gen, device="cuda")

    if op == "product":
        E, n, k, rows = case["experts"], case["n"], case["k"], case["rows"]
        cols = n if case["transposed"] else k
        s["counts"] = _counts(case)
        c = [0]
        for x in s["counts"]:
            c.append(c[-1] + x)
        s["offsets"] = torch.tensor(c, dtype=torch.int32, device="cuda")
        s["aq"], s["as"] = _codes((rows, cols), gen, 110.0), uniform(0.004, 0.02, rows, _blocks(cols))
        s["wq"] = _codes((E, n, k), gen, 100.0)
        s["ws"] = uniform(0.005, 0.015, E, _blocks(n), _blocks(k)) / math.sqrt(k)
    elif op == "swiglu":
        rows, I = case["rows"], case["inter"]
        s["gu"] = _bits(normal(rows, 2 * I) * uniform(0.3, 3.0, rows, 1))
        if case["grad"]:
            s["dh"] = _bits(normal(rows, I) * uniform(0.001, 0.01, rows, 1))
        s["total"] = torch.tensor([rows - case["tail"]], dtype=torch.int32, device="cuda")
        cols = 2 * I if case["grad"] else I
        s["out"], s["out_scale"] = _rows_out(rows, cols, case["e4m3"])
    else:
        T, k, E, d = case["tokens"], case["k"], case["experts"], case["d"]
        s["ids"] = _ids(case, gen)
        rows = T * k
        if op == "sort":
            s["x"] = _bits(normal(T, d) * uniform(0.2, 2.0, T, 1))
            s["out"], s["out_scale"] = _rows_out(rows, d, case["e4m3"])
        else:
            s["inv"] = _sorted_places(s["ids"], E)[2]
            s["w"] = torch.softmax(normal(T, k), -1)
            s["ys"] = _bits(normal(rows, d))
            if op == "grad":
                s["dy"] = _bits(normal(T, d) * uniform(0.001, 0.01, T, 1))
                s["out"], s["out_scale"] = _rows_out(rows, d, case["e4m3"])
            elif case["add"]:
                s["add"] = _bits(normal(T, d))
    if own:
        import quantized_grouped_gemm_router_gb300 as moe
        s["space"] = moe.expert_workspace(case.get("experts", 1))
        if op == "product":
            s["a"], s["weights"] = moe.E4m3Rows(s["aq"], s["as"]), moe.E4m3Weights(s["wq"], s["ws"])
        elif "out" in s:
            s["rows_out"] = moe.E4m3Rows(s["out"], s["out_scale"]) if case["e4m3"] else s["out"]
    return s


def _rows_out(rows, cols, e4m3):
    """Zeroed buffers for rows in 16 or 8 bits: rows that belong to no expert stay as they were."""
    if e4m3:
        return (torch.zeros((rows, cols), dtype=torch.uint8, device="cuda"),
                torch.zeros((rows, _blocks(cols)), dtype=torch.float32, device="cuda"))
    return torch.zeros((rows, cols), dtype=torch.int16, device="cuda"), None


# ------------------------------------------------------------------------------------ one pass
def run(s):
    return _own(s) if own else {"sort": _plain_sort, "back": _plain_back, "grad": _plain_grad,
                                "product": _plain_product, "swiglu": _plain_swiglu}[s["op"]](s)


def _own(s):
    import quantized_grouped_gemm_router_gb300 as moe
    op, ws = s["op"], s["space"]
    if op == "sort":
        offsets, perm, inv = moe.sort_tokens(s["ids"], s["experts"], ws)
        moe.dispatch(s["x"], inv, ws, out=s["rows_out"])
        return {"offsets": offsets, "perm": perm, "inv": inv, **_rows(s)}
    if op == "back":
        y = moe.combine(s["ys"], s["inv"], s["w"] if s["weighted"] else None, ws,
                        add=None if s["add"] is False else s["add"])
        return {"y": y.view(BF16)}
    if op == "grad":
        _, dw = moe.combine_grad(s["dy"], s["ys"], s["inv"], s["w"], ws, out=s["rows_out"])
        return {"dw": dw, **_rows(s)}
    if op == "product":
        y = moe.gemm_e4m3(s["a"], s["weights"], s["offsets"] if s["experts"] > 1 else None, ws,
                          transposed=s["transposed"])
        return {"y": y.view(BF16)}
    if s["grad"]:
        moe.swiglu_grad(s["gu"], s["dh"], ws, total=s["total"], out=s["rows_out"])
    else:
        moe.swiglu(s["gu"], ws, total=s["total"], out=s["rows_out"])
    return _rows(s)


def _rows(s):
    if s["e4m3"]:
        return {"q": s["out"].view(E4M3), "scale": s["out_scale"]}
    return {"rows": s["out"].view(BF16)}


def _quantise(x):
    """Codes and scales of fp32 rows."""
    rows, cols = x.shape
    nb = _blocks(cols)
    x = torch.nn.functional.pad(x, (0, nb * 128 - cols)).view(rows, nb, 128)
    fine = torch.isfinite(x)
    a = torch.where(fine, x.abs(), 0.0).amax(-1).clamp_min(2.0 ** -100)
    q = (x * (448.0 / a)[..., None]).clamp(-448.0, 448.0)
    q = torch.where(fine, q, math.nan).view(rows, nb * 128)[:, :cols]
    return q.to(E4M3).view(torch.uint8), a / 448.0


def _store(s, at, x):
    """fp32 rows x to the rows `at` of the state's buffers."""
    if s["e4m3"]:
        q, scale = _quantise(x)
        s["out"][at] = q
        s["out_scale"][at] = scale
    else:
        s["out"][at] = x.to(BF16).view(torch.int16)
    return _rows(s)


def _there(s):
    """Places of the assignments that have an expert, and their numbers."""
    a = (s["inv"].reshape(-1) >= 0).nonzero()[:, 0]
    return s["inv"].reshape(-1)[a].long(), a


def _plain_sort(s):
    offsets, perm, inv = _sorted_places(s["ids"], s["experts"])
    at = perm[perm >= 0].long() // s["k"]
    return {"offsets": offsets, "perm": perm, "inv": inv,
            **_store(s, torch.arange(len(at), device="cuda"), s["x"].view(BF16)[at].float())}


def _plain_back(s):
    inv = s["inv"].long()
    y = s["add"].view(BF16).float() if s["add"] is not False else torch.zeros((s["tokens"], s["d"]), device="cuda")
    for j in range(s["k"]):
        row = s["ys"].view(BF16)[inv[:, j].clamp_min(0)].float()
        if s["weighted"]:
            row *= s["w"][:, j, None]
        y = y + torch.where(inv[:, j, None] >= 0, row, 0.0)
    return {"y": y.to(BF16)}


def _plain_grad(s):
    place, a = _there(s)
    dy = s["dy"].view(BF16).float()[a // s["k"]]
    dw = torch.zeros(s["tokens"] * s["k"], device="cuda")
    dw[a] = (dy * s["ys"].view(BF16)[place].float()).sum(-1)
    return {"dw": dw.view(s["tokens"], s["k"]), **_store(s, place, dy * s["w"].reshape(-1)[a][:, None])}


def _spread(scale, n, k):
    """Scales of blocks of 128 x 128 for every element of [n, k]."""
    return scale.repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]


def _plain_product(s):
    n, k = s["n"], s["k"]
    y = torch.empty((s["rows"], k if s["transposed"] else n), dtype=BF16, device="cuda")
    at = 0
    for e, rows in enumerate(s["counts"]):
        if rows:
            a = s["aq"][at:at + rows].view(E4M3).float()
            a *= s["as"][at:at + rows].repeat_interleave(128, 1)[:, :a.shape[1]]
            w = s["wq"][e].view(E4M3).float() * _spread(s["ws"][e], n, k)
            y[at:at + rows] = (a @ (w if s["transposed"] else w.t())).to(BF16)
            at += rows
    return {"y": y}


def _plain_swiglu(s):
    n, I = s["rows"] - s["tail"], s["inter"]
    gu = s["gu"].view(BF16)[:n].float()
    g, u = gu[:, :I], gu[:, I:]
    sig = 1.0 / (1.0 + torch.exp(-g))
    if not s["grad"]:
        return _store(s, torch.arange(n, device="cuda"), g * sig * u)
    dh = s["dh"].view(BF16)[:n].float()
    d = torch.cat([dh * u * sig * (1.0 + g * (1.0 - sig)), dh * g * sig], 1)
    return _store(s, torch.arange(n, device="cuda"), d)


# ------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """One expert, or one place of a token's list, at a time, from the definitions."""
    s = prepare(case, seed)
    f64, op = torch.float64, case["op"]

    def rows64(rows):
        """What the buffers hold where rows[p] = the 64-bit row of place p."""
        out = torch.zeros(s["out"].shape, dtype=f64, device="cuda")
        if not case["e4m3"]:
            for at, x in rows:
                out[at] = x
            return {"rows": out}
        scale = torch.zeros(s["out_scale"].shape, dtype=f64, device="cuda")
        for at, x in rows:
            q = torch.empty_like(x)
            for b in range(scale.shape[1]):
                block = x[:, 128 * b:128 * b + 128]
                a = block.abs().max(1).values.clamp(min=2.0 ** -100) / 448
                scale[at, b] = a
                q[:, 128 * b:128 * b + 128] = block / a[:, None]
            out[at] = q
        return {"q": out, "scale": scale}

    if op == "product":
        n, k, cols = case["n"], case["k"], s["aq"].shape[1]
        y = torch.zeros((case["rows"], k if case["transposed"] else n), dtype=f64, device="cuda")
        for e, c in enumerate(s["counts"]):
            first = sum(s["counts"][:e])
            if c == 0:
                continue
            w = s["wq"][e].view(E4M3).to(f64)
            for i in range(0, n, 128):
                for j in range(0, k, 128):
                    w[i:i + 128, j:j + 128] *= s["ws"][e, i // 128, j // 128].to(f64)
            a = s["aq"][first:first + c].view(E4M3).to(f64)
            for j in range(0, cols, 128):
                a[:, j:j + 128] *= s["as"][first:first + c, j // 128, None].to(f64)
            y[first:first + c] = torch.einsum("pn,nk->pk" if case["transposed"] else "pk,nk->pn", a, w)
        return {"y": y}
    if op == "swiglu":
        n, I = case["rows"] - case["tail"], case["inter"]
        parts = []
        for i in range(0, n, 8192):
            at = slice(i, min(n, i + 8192))
            g, u = s["gu"][at].view(BF16).to(f64).split(I, 1)
            if case["grad"]:
                dh, up = s["dh"][at].view(BF16).to(f64), torch.sigmoid(g)
                parts.append((at, torch.cat([dh * u * (up + g * up * torch.sigmoid(-g)), dh * g * up], 1)))
            else:
                parts.append((at, u * g / (1 + torch.exp(-g))))
        return rows64(parts)
    T, k = case["tokens"], case["k"]
    if op == "back":
        y = s["add"].view(BF16).to(f64) if case["add"] else torch.zeros((T, case["d"]), dtype=f64, device="cuda")
        for j in range(k):
            t = (s["inv"][:, j] >= 0).nonzero()[:, 0]
            x = s["ys"].view(BF16)[s["inv"][t, j].long()].to(f64)
            y[t] += x * s["w"][t, j, None].to(f64) if case["weighted"] else x
        return {"y": y}
    if op == "grad":
        dw, parts = torch.zeros((T, k), dtype=f64, device="cuda"), []
        for j in range(k):
            t = (s["inv"][:, j] >= 0).nonzero()[:, 0]
            p, dy = s["inv"][t, j].long(), s["dy"].view(BF16)[t].to(f64)
            dw[t, j] = torch.einsum("td,td->t", dy, s["ys"].view(BF16)[p].to(f64))
            parts.append((p, dy * s["w"][t, j, None].to(f64)))
        return {"dw": dw, **rows64(parts)}
    # sorting: by counting, one expert after the other
    flat = s["ids"].reshape(-1)
    offsets = torch.zeros(case["experts"] + 1, dtype=torch.int32, device="cuda")
    perm, inv = (torch.full((T * k,), -1, dtype=torch.int32, device="cuda") for _ in range(2))
    at = 0
    for e in range(case["experts"]):
        a = (flat == e).nonzero()[:, 0]
        offsets[e] = at
        perm[at:at + len(a)] = a.int()
        inv[a] = torch.arange(at, at + len(a), dtype=torch.int32, device="cuda")
        at += len(a)
    offsets[case["experts"]] = at
    rows = [(slice(i, min(at, i + 16384)), s["x"].view(BF16)[perm[i:min(at, i + 16384)].long() // k].to(f64))
            for i in range(0, at, 16384)]
    return {"offsets": offsets, "perm": perm, "inv": inv.view(T, k), **rows64(rows)}
