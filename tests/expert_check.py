"""Plain 64-bit forms of the 8-bit expert calls and the comparison rules of their tests.

Tolerances, from the arithmetic that the calls promise (fp32 sums, one rounding at the end):
  * rounding x to bf16 costs at most 2^-8 |x|, to e4m3 at most 2^-4 |x| for normal codes and half of
    the smallest code's step, 2^-10, times the scale below them;
  * quantising itself is a fixed fp32 formula of IEEE operations: codes and scales of given fp32 rows
    are compared bit by bit (`quantise`);
  * a sum of n fp32 products, each rounded, is off by at most (n + 1) 2^-24 times the sum of magnitudes S;
  * combine adds at most top_k + 1 terms; dw adds d / 32 products in a lane and 5 lanes' sums, rounded up
    to whole pieces of 512 columns;
  * a product of codes (8 significant bits at most) is exact in fp32; a block of 128 is summed with fewer
    than 128 roundings, of at most 2^-23 where the tensor cores cut rather than round, and B blocks with B
    scalings (2 roundings) and additions: (2^-16 + 3 B 2^-24) S covers both;
  * the sigmoid: the exponent's argument g log2(e) is off by |g| 2^-23, which shifts the exponential by
    that share; the exponential's approximation 2^-22, the sum 2^-24, the reciprocal 2^-23, two
    products 2^-24 each: e(g) = (|g| + 8) 2^-23 relative covers them. Where e^-g passes 2^128, or its
    reciprocal is subnormal, s is off by at most 2^-126.
"""
from __future__ import annotations

import torch

F64 = torch.float64


def bits(x: torch.Tensor) -> torch.Tensor:
    """bf16 bit patterns as int16."""
    return x.to(torch.bfloat16).view(torch.int16)


def values(x: torch.Tensor) -> torch.Tensor:
    """bf16 bit patterns in 64 bits, on the host."""
    return x.cpu().view(torch.bfloat16).to(F64)


def blocks(n: int) -> int:
    return (n + 127) // 128


def sort(ids: torch.Tensor, E: int):
    """offsets, perm, inv by hand."""
    flat = ids.reshape(-1).tolist()
    lists = [[a for a, e in enumerate(flat) if e == x] for x in range(E)]
    offsets, perm, inv = [0], [-1] * len(flat), [-1] * len(flat)
    at = 0
    for rows in lists:
        for a in rows:
            perm[at], inv[a] = a, at
            at += 1
        offsets.append(at)
    i32 = torch.int32
    return (torch.tensor(offsets, dtype=i32), torch.tensor(perm, dtype=i32),
            torch.tensor(inv, dtype=i32).view(ids.shape))


def quantise(x: torch.Tensor):
    """Codes (uint8) and scales of fp32 rows [rows, cols], the calls' formula in IEEE fp32."""
    assert x.dtype == torch.float32
    rows, cols = x.shape
    nb = blocks(cols)
    p = torch.nn.functional.pad(x, (0, nb * 128 - cols)).view(rows, nb, 128)
    fine = torch.isfinite(p)
    a = torch.where(fine, p.abs(), torch.zeros(())).amax(-1).clamp_min(2.0 ** -100)
    y = torch.where(fine, p, torch.zeros(())) * (torch.tensor(448.0) / a)[..., None]
    q = y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    q = torch.where(fine, q, torch.tensor(0x7F, dtype=torch.uint8))
    return q.view(rows, nb * 128)[:, :cols], a / torch.tensor(448.0)


def same_codes(q: torch.Tensor, want: torch.Tensor) -> bool:
    """Equal codes; any NaN equals any other, and +0 equals -0."""
    q, want = q.cpu().view(torch.float8_e4m3fn).float(), want.view(torch.float8_e4m3fn).float()
    return torch.equal(torch.isnan(q), torch.isnan(want)) and torch.equal(torch.nan_to_num(q), torch.nan_to_num(want))


def code_values(q: torch.Tensor, scale: torch.Tensor) -> torch.Tensor:
    """What e4m3 rows stand for, in 64 bits, on the host."""
    s = scale.cpu().to(F64).repeat_interleave(128, -1)[..., :q.shape[-1]]
    return q.cpu().view(torch.float8_e4m3fn).float().to(F64) * s


def weight_values(q: torch.Tensor, scale: torch.Tensor) -> torch.Tensor:
    s = scale.cpu().to(F64).repeat_interleave(128, 1)[:, :q.shape[1]].repeat_interleave(128, 2)[:, :, :q.shape[2]]
    return q.cpu().view(torch.float8_e4m3fn).float().to(F64) * s


def close(got: torch.Tensor, ref: torch.Tensor, tol: torch.Tensor, what=""):
    """|got - ref| <= tol, elementwise in 64 bits."""
    assert got.shape == ref.shape, what
    got = got.cpu().to(F64)
    assert torch.isfinite(got).all(), f"{what}: non-finite"
    if ref.numel():
        worst = ((got - ref).abs() / (tol + 1e-300)).max().item()
        assert worst <= 1.0, f"{what}: off by {worst:.3f} x tolerance"


def combine(ys, inv, w, add):
    """ys [rows, d], w [T, k] or None, add [T, d] or None, in 64 bits -> y and its sum of magnitudes."""
    T, k = inv.shape
    y = torch.zeros(T, ys.shape[1], dtype=F64) if add is None else add.clone()
    size = y.abs()
    for t in range(T):
        for j in range(k):
            if inv[t, j] >= 0:
                x = ys[inv[t, j]] * (1.0 if w is None else w[t, j])
                y[t] += x
                size[t] += x.abs()
    return y, size


def check_combine(y, ref, size, k, what=""):
    err = (k + 2) * 2.0 ** -24 * size
    close(values(y), ref, 2.0 ** -8 * (ref.abs() + err) + err + 2.0 ** -133, what)


def product(a, w, counts, transposed):
    """a [rows, in], w [E, n, k] in 64 bits -> out and the sums of magnitudes."""
    cols = w.shape[2] if transposed else w.shape[1]
    out, size = torch.zeros(a.shape[0], cols, dtype=F64), torch.zeros(a.shape[0], cols, dtype=F64)
    at = 0
    for e, c in enumerate(counts):
        m = w[e] if transposed else w[e].t()
        out[at:at + c] = a[at:at + c] @ m
        size[at:at + c] = a[at:at + c].abs() @ m.abs()
        at += c
    return out, size


def check_product(y, ref, size, n_blocks, what=""):
    err = (2.0 ** -16 + 3 * n_blocks * 2.0 ** -24) * size
    close(values(y), ref, 2.0 ** -8 * (ref.abs() + err) + err + 2.0 ** -133, what)


def swiglu(gu):
    """gu [rows, 2 I] in 64 bits -> h and the bound of its fp32 error."""
    g, u = gu.chunk(2, 1)
    h = g * torch.sigmoid(g) * u
    return h, h.abs() * (g.abs() + 8) * 2.0 ** -23 + (g * u).abs() * 2.0 ** -126


def swiglu_grad(gu, dh):
    """dgu and the bound of its fp32 error: 1 - s carries e s + 2^-24, times |g|; the rest are products."""
    (g, u), s = gu.chunk(2, 1), torch.sigmoid(gu.chunk(2, 1)[0])
    e = (g.abs() + 8) * 2.0 ** -23
    rest = 1 + g * torch.sigmoid(-g)
    dg, du = dh * u * s * rest, dh * g * s
    tiny = 2.0 ** -126 * (1 + g.abs()) ** 2
    err_g = (dh * u).abs() * (s * (rest.abs() * (e + 2.0 ** -22) + (g.abs() + 1) * (e * s + 2.0 ** -23)) + tiny)
    err_u = du.abs() * e + (dh * g).abs() * 2.0 ** -126
    return torch.cat([dg, du], 1), torch.cat([err_g, err_u], 1)


def check_rows(got, ref, err, what=""):
    """bf16 rows (int16) or E4m3Rows against 64-bit values with a bound of their fp32 error."""
    if isinstance(got, torch.Tensor):
        close(values(got), ref, 2.0 ** -8 * (ref.abs() + err) + err + 2.0 ** -133, what)
        return
    q, scale = got.q, got.scale.cpu().to(F64)
    nb = scale.shape[1]

    def by_block(x):
        return torch.nn.functional.pad(x, (0, nb * 128 - x.shape[1])).view(len(x), nb, 128)

    want = by_block(ref.abs()).amax(-1).clamp_min(2.0 ** -100) / 448
    close(scale, want, want * 2.0 ** -22 + by_block(err).amax(-1) / 448, f"{what}: scales")
    s = scale.repeat_interleave(128, 1)[:, :ref.shape[1]]
    close(code_values(q, got.scale), ref, (2.0 ** -4 + 2.0 ** -20) * (ref.abs() + err) + 2.0 ** -10 * s + err, what)
