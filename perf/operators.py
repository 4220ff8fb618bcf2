"""The attention operators' measured cases: packed prompt attention, the paged key-value cache's
append, and one-token attention over that cache.

Every case runs in two forms. The plain form (own = False) is elementary torch arithmetic in 32
bits; the other calls the package's entry points as a serving program does. bf16 tensors travel as
int16 bit patterns, as everywhere in this package.

Shapes: 16 query heads over 2 key-value heads is the grouping of the attention layers that this
package's pages describe next to the mixture-of-experts layer; the other groupings, head sizes and
page sizes are generic. Prompt lengths of 512 and 4096 tokens are the benchmark's prefill configurations; contexts
up to 131072 tokens are the range the pages report.
"""
import math
import random

import torch

own = False

GROUPS = [(16, 2), (8, 8), (12, 4), (32, 4), (7, 1)]  # (query heads, key-value heads) drawn
SPAN = 16384 * 16384 * 16 * 128                       # padded score work of the longest listed prompt


# ------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # one short question: latency of a call
        dict(name="prompt_4", op="prefill", heads=16, kv=2, d=128, seqs=1, tokens=4, ctx=0, causal=True, fused=False),
        # one prompt of the benchmark's short prefill length, read from a fused q|k|v projection
        dict(name="prompt_512", op="prefill", heads=16, kv=2, d=128, seqs=1, tokens=512, ctx=0, causal=True,
             fused=True),
        # requests of different lengths packed into the benchmark's 4096-token prefill
        dict(name="packed_4096", op="prefill", heads=16, kv=2, d=128, seqs=9, tokens=4096, ctx=0, causal=True,
             fused=True),
        # the next chunk of long prompts: 1021 new tokens see 8192 earlier ones, wide heads
        dict(name="chunk_on_8192", op="prefill", heads=16, kv=2, d=256, seqs=1, tokens=1021, ctx=8192, causal=True,
             fused=False),
        # short texts scored in both directions, one key-value head per query head, narrow heads
        dict(name="both_ways", op="prefill", heads=8, kv=8, d=64, seqs=24, tokens=6001, ctx=0, causal=False,
             fused=True),
        # one long document
        dict(name="prompt_16384", op="prefill", heads=16, kv=2, d=128, seqs=1, tokens=16384, ctx=0, causal=True,
             fused=False),
        # one user early in a conversation: latency of a call
        dict(name="token_511", op="decode", heads=16, kv=2, d=128, seqs=1, longest=511, page=16, fp8=False),
        # one user at the far end of a long context: the cache's length has to be split
        dict(name="token_131071", op="decode", heads=16, kv=2, d=128, seqs=1, longest=131071, page=64, fp8=False),
        # a serving batch of different lengths
        dict(name="batch_64", op="decode", heads=16, kv=2, d=128, seqs=64, longest=16384, page=32, fp8=False),
        # a larger batch with the cache in 8 bits and wide heads
        dict(name="batch_fp8", op="decode", heads=16, kv=2, d=256, seqs=129, longest=8191, page=64, fp8=True),
        # the new token of every sequence of a batch written to the 8-bit cache
        dict(name="append_64", op="append", heads=16, kv=2, d=128, seqs=64, tokens=64, before=4096, page=32, fp8=True),
        # the keys and values of packed prompts written to the cache
        dict(name="append_8192", op="append", heads=16, kv=8, d=128, seqs=9, tokens=8192, before=700, page=64,
             fp8=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "decode", "decode", "append"])
    heads, kv = rng.choice(GROUPS)
    d = rng.choice([64, 128, 128, 256])
    case = dict(op=op, heads=heads, kv=kv, d=d)
    if op == "prefill":
        seqs = _log(rng, 1, 32)
        tokens = max(seqs, _log(rng, 1, 16384))
        ctx = rng.choice([0, 0, _log(rng, 1, 8192)])
        case.update(seqs=seqs, tokens=tokens, ctx=ctx, causal=rng.random() < 0.75, fused=rng.random() < 0.5)
        while _padded(case) > SPAN or _pairs(case) * heads * d > 16384 * 8192 * 16 * 128:
            case.update(tokens=max(1, case["tokens"] // 2), seqs=max(1, min(case["seqs"], case["tokens"] // 4)),
                        ctx=case["ctx"] // 2)
    elif op == "decode":
        case.update(seqs=_log(rng, 1, 256), longest=_log(rng, 1, 131072), page=rng.choice([16, 32, 48, 64, 128]),
                    fp8=rng.random() < 0.5)
        while case["seqs"] * case["longest"] * kv * d > 64 * 16384 * 2 * 128 * 2:
            case.update(longest=max(1, case["longest"] // 2), seqs=max(1, (case["seqs"] * 3 + 1) // 4))
    else:
        seqs = _log(rng, 1, 128)
        case.update(seqs=seqs, tokens=max(seqs, _log(rng, 1, 8192)), before=_log(rng, 1, 4096),
                    page=rng.choice([16, 32, 48, 64, 128]), fp8=rng.random() < 0.5)
    return case


def _parts(case):
    """Lengths of the packed sequences: uneven, an empty and a one-token one among them from eight
    sequences on."""
    n, total = case["seqs"], case["tokens"]
    if n == 1:
        return [total]
    rng = random.Random(n * 1000003 + total)
    w = [math.exp(rng.gauss(0.0, 0.8)) for _ in range(n)]
    lens = [int(total * x / sum(w)) for x in w]
    if n >= 8:
        lens[1], lens[n // 2] = 0, min(1, total)
    lens[0] += total - sum(lens)
    return lens


def _lens(case):
    """Cache lengths of a batch: the first is the longest, the others spread over their logarithm."""
    rng = random.Random(case["seqs"] * 1000003 + case["longest"])
    return [case["longest"]] + [_log(rng, max(1, case["longest"] // 16), case["longest"])
                                for _ in range(case["seqs"] - 1)]


def _padded(case):
    lens = _parts(case)
    return len(lens) * max(lens) * (max(lens) + case["ctx"]) * case["heads"] * case["d"]


def _pairs(case):
    """Query-key pairs that the mask leaves, for one head."""
    c = case["ctx"]
    return sum(n * (n + c) if not case["causal"] else n * c + n * (n + 1) // 2 for n in _parts(case))


def work(case):
    H, K, d = case["heads"], case["kv"], case["d"]
    if case["op"] == "prefill":
        tq = case["tokens"]
        tk = tq + case["ctx"] * case["seqs"]
        return {"bytes": 2 * d * (2 * tq * H + 2 * tk * K) + 4 * tq * H, "flops": 4 * d * H * _pairs(case)}
    size = 1 if case["fp8"] else 2
    if case["op"] == "decode":
        n = sum(_lens(case))
        return {"bytes": 2 * n * K * d * size + case["seqs"] * H * (4 * d + 4), "flops": 4 * d * H * n}
    return {"bytes": 2 * case["tokens"] * K * d * (2 + size), "flops": 0}


# ------------------------------------------------------------------------------------ the inputs
def _cu(lens):
    c = [0]
    for n in lens:
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int32, device="cuda")


def _pages(lens, page, gen, spare):
    """A page table of randomly placed pages; what lies past a sequence's pages is never used."""
    need = [(n + page - 1) // page for n in lens]
    width, total = max(1, max(need)), sum(need) + spare
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros((len(lens), width), dtype=torch.int32, device="cuda")
    at = torch.arange(width, device="cuda")[None] < torch.tensor(need, device="cuda")[:, None]
    table[at] = order[: sum(need)]
    return table, total


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    H, K, d = case["heads"], case["kv"], case["d"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    gain = 0.5 + 2.0 * torch.rand((H, 1), generator=gen, device="cuda")  # flat heads and peaked ones
    s = dict(case)
    if case["op"] == "prefill":
        lens = _parts(case)
        tq, tk = case["tokens"], case["tokens"] + case["ctx"] * case["seqs"]
        s["max_q"], s["max_k"] = max(lens), max(lens) + case["ctx"]
        s["cu_q"], s["cu_k"] = _cu(lens), _cu([n + case["ctx"] for n in lens])
        if case["fused"] and tq == tk:
            rows = normal(tq, H + 2 * K, d)
            rows[:, :H] *= gain
            rows = rows.to(torch.bfloat16).view(torch.int16)
            s["q"], s["k"], s["v"] = rows[:, :H], rows[:, H:H + K], rows[:, H + K:]
        else:
            for name, t, heads in (("q", tq, H), ("k", tk, K), ("v", tk, K)):
                x = normal(t, heads, d)
                s[name] = (x * gain if name == "q" else x).to(torch.bfloat16).view(torch.int16)
        s["lse"] = torch.empty((tq, H), dtype=torch.float32, device="cuda")
    else:
        page, fp8 = case["page"], case["fp8"]
        if case["op"] == "decode":
            lens = _lens(case)
            s["q"] = (normal(len(lens), H, d) * gain).to(torch.bfloat16).view(torch.int16)
            s["lse"] = torch.empty((len(lens), H), dtype=torch.float32, device="cuda")
            s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        else:
            new = _parts(case)
            rng = random.Random(case["before"])
            before = [rng.randint(0, case["before"]) for _ in new]
            lens = [a + b for a, b in zip(before, new)]
            s["k_new"], s["v_new"] = (normal(case["tokens"], K, d).to(torch.bfloat16).view(torch.int16)
                                      for _ in range(2))
            s["cu"] = _cu(new)
            s["start"] = torch.tensor(before, dtype=torch.int32, device="cuda")
            s["max_new"] = max(new)
        s["table"], n = _pages(lens, page, gen, 3)
        s["k_scale"], s["v_scale"] = ((0.01 + 0.02 * torch.rand(K, generator=gen, device="cuda")) if fp8 else None
                                      for _ in range(2))
        for name in ("k", "v"):
            x = normal(n, K, page, d) if case["op"] == "decode" else torch.zeros((n, K, page, d), device="cuda")
            s[name] = ((x * 40.0).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8) if fp8
                       else x.to(torch.bfloat16).view(torch.int16))
            del x
    if own:
        import quantized_grouped_gemm_router_gb300 as moe
        s["dims"] = moe.AttnDims(H, K, d)
        s["ws"] = moe.attn_workspace(s["dims"])
        if case["op"] != "prefill":
            s["cache"] = moe.KvCache(s["dims"], s["k"], s["v"], s["k_scale"], s["v_scale"])
    return s


# ------------------------------------------------------------------------------------ one pass
def run(s):
    return _own(s) if own else {"prefill": _plain_prefill, "decode": _plain_decode, "append": _plain_append}[s["op"]](s)


def _own(s):
    import quantized_grouped_gemm_router_gb300 as moe
    if s["op"] == "prefill":
        o = moe.attn_prefill(s["dims"], s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["ws"], causal=s["causal"],
                             lse=s["lse"])
        return {"o": o.view(torch.bfloat16), "lse": s["lse"]}
    if s["op"] == "decode":
        o = moe.attn_decode(s["cache"], s["q"], s["lens"], s["table"], s["ws"], lse=s["lse"])
        return {"o": o.view(torch.bfloat16), "lse": s["lse"]}
    moe.kv_append(s["cache"], s["k_new"], s["v_new"], s["cu"], s["start"], s["table"], s["ws"])
    return _values(s)


def _values(s):
    t = torch.float8_e4m3fn if s["fp8"] else torch.bfloat16
    return {"k": s["k"].view(t), "v": s["v"].view(t)}


def _softmax_av(scores, seen, v):
    """Softmax over the keys that `seen` leaves and its product with v; a row that sees none gives
    0 and -inf."""
    scores.masked_fill_(~seen, -math.inf)
    m = scores.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = scores.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(total == 0, torch.ones_like(total), total)
    return o, (total.log() + m).squeeze(-1)


def _plain_prefill(s):
    H, K, d = s["heads"], s["kv"], s["d"]
    G, B, Lq, Lk = H // K, s["seqs"], s["max_q"], s["max_k"]
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    nq, nk = (cu_q[1:] - cu_q[:-1])[:, None], (cu_k[1:] - cu_k[:-1])[:, None]
    iq, ik = torch.arange(Lq, device="cuda")[None], torch.arange(Lk, device="cuda")[None]
    at_q = (cu_q[:-1, None] + iq).clamp_(max=s["q"].shape[0] - 1)
    at_k = (cu_k[:-1, None] + ik).clamp_(max=s["k"].shape[0] - 1)
    q = s["q"].view(torch.bfloat16).float()[at_q].reshape(B, Lq, K, G, d).permute(0, 2, 3, 1, 4)
    k = s["k"].view(torch.bfloat16).float()[at_k].permute(0, 2, 3, 1)
    v = s["v"].view(torch.bfloat16).float()[at_k].permute(0, 2, 1, 3)
    scores = (q.reshape(B, K, G * Lq, d) @ k).mul_(1.0 / math.sqrt(d)).view(B, K, G, Lq, Lk)
    seen = (ik < nk)[:, None, :].expand(B, Lq, Lk)
    if s["causal"]:
        seen = seen & (ik[:, None, :] <= (iq + nk - nq)[:, :, None])
    o, lse = _softmax_av(scores, seen[:, None, None], v[:, :, None])
    there = iq < nq
    o = o.permute(0, 3, 1, 2, 4).reshape(B, Lq, H, d)[there]
    return {"o": o.to(torch.bfloat16), "lse": lse.permute(0, 3, 1, 2).reshape(B, Lq, H)[there]}


def _plain_decode(s):
    H, K, d, page = s["heads"], s["kv"], s["d"], s["page"]
    table, B = s["table"].long(), s["seqs"]

    def rows(name):
        x = s[name][table]                                      # [B, pages, K, page, d]
        x = x.view(torch.float8_e4m3fn if s["fp8"] else torch.bfloat16).float()
        if s["fp8"]:
            x.mul_(s[name + "_scale"][None, None, :, None, None])
        return x.permute(0, 2, 1, 3, 4).reshape(B, K, -1, d)

    q = s["q"].view(torch.bfloat16).float().view(B, K, H // K, d)
    scores = (q @ rows("k").transpose(-1, -2)).mul_(1.0 / math.sqrt(d))
    seen = torch.arange(scores.shape[-1], device="cuda")[None] < s["lens"][:, None]
    o, lse = _softmax_av(scores, seen[:, None, None], rows("v"))
    return {"o": o.reshape(B, H, d).to(torch.bfloat16), "lse": lse.reshape(B, H)}


def _plain_append(s):
    page, n = s["page"], s["k_new"].shape[0]
    cu = s["cu"].long()
    t = torch.arange(n, device="cuda")
    b = (t[:, None] >= cu[None, 1:]).sum(1)
    pos = s["start"].long()[b] + t - cu[b]
    at = s["table"].long()[b, pos // page]
    for name in ("k", "v"):
        x = s[name + "_new"].view(torch.bfloat16)
        if s["fp8"]:
            x = (x.float() / s[name + "_scale"][None, :, None]).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
            s[name][at, :, pos % page] = x.view(torch.uint8)
        else:
            s[name][at, :, pos % page] = x.view(torch.int16)
    return _values(s)


# ------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """One sequence and one head at a time, from the definition: o = sum_j p_j v_j / sum_j p_j with
    p_j = exp(scale q.k_j), and lse = log sum_j p_j."""
    s = prepare(case, seed)
    H, K, d = case["heads"], case["kv"], case["d"]
    f64 = torch.float64

    def attend(q, k, v, first):
        """q [n, d] against k, v [m, d]; row i sees the keys below first + i."""
        o, lse = torch.zeros((len(q), d), dtype=f64, device="cuda"), torch.full((len(q),), -math.inf, dtype=f64,
                                                                               device="cuda")
        for i in range(0, len(q), 4096):
            n = min(4096, len(q) - i)
            m = len(k) if first is None else max(0, min(len(k), first + i + n - 1))
            if m == 0:
                continue
            x = (q[i:i + n] @ k[:m].t()) / math.sqrt(d)
            if first is not None:
                limit = first + torch.arange(i, i + n, device="cuda")
                x[torch.arange(m, device="cuda")[None] >= limit[:, None]] = -math.inf
            z = torch.logsumexp(x, -1)
            some = z > -math.inf
            o[i:i + n][some] = torch.exp(x[some] - z[some, None]) @ v[:m]
            lse[i:i + n] = z
        return o, lse

    if case["op"] == "append":
        out = {}
        lens = _parts(case)
        begin, table = s["start"].tolist(), s["table"].tolist()
        for name in ("k", "v"):
            cells = s[name].view(torch.float8_e4m3fn if case["fp8"] else torch.bfloat16).float().to(f64)
            x = s[name + "_new"].view(torch.bfloat16).to(f64)
            if case["fp8"]:
                x = (x / s[name + "_scale"].to(f64)[None, :, None]).clamp(-448.0, 448.0)
            at, slots = 0, []
            for b, n in enumerate(lens):
                slots += [(table[b][p // case["page"]], p % case["page"]) for p in range(begin[b], begin[b] + n)]
            where = torch.tensor(slots, device="cuda")
            cells[where[:, 0], :, where[:, 1]] = x
            out[name] = cells
        return out
    if case["op"] == "decode":
        o = torch.zeros((case["seqs"], H, d), dtype=f64, device="cuda")
        lse = torch.zeros((case["seqs"], H), dtype=f64, device="cuda")
        q = s["q"].view(torch.bfloat16).to(f64)
        for b, n in enumerate(_lens(case)):
            ids = s["table"][b, : (n + case["page"] - 1) // case["page"]].long()
            for h in range(K):
                k, v = (s[name][ids, h].reshape(-1, d)[:n].view(torch.float8_e4m3fn if case["fp8"] else torch.bfloat16)
                        .float().to(f64) * (float(s[name + "_scale"][h]) if case["fp8"] else 1.0) for name in ("k", "v"))
                mine = slice(h * (H // K), (h + 1) * (H // K))
                o[b, mine], lse[b, mine] = attend(q[b, mine], k, v, None)
        return {"o": o, "lse": lse}
    q, k, v = (s[name].view(torch.bfloat16) for name in ("q", "k", "v"))
    o = torch.zeros((case["tokens"], H, d), dtype=f64, device="cuda")
    lse = torch.zeros((case["tokens"], H), dtype=f64, device="cuda")
    a = b = 0
    for n in _parts(case):
        m = n + case["ctx"]
        for h in range(H if n else 0):
            kh, vh = k[b:b + m, h // (H // K)].to(f64), v[b:b + m, h // (H // K)].to(f64)
            o[a:a + n, h], lse[a:a + n, h] = attend(q[a:a + n, h].to(f64), kh, vh,
                                                    m - n + 1 if case["causal"] else None)
        a, b = a + n, b + m
    return {"o": o, "lse": lse}
