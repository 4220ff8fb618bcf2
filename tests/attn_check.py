"""Plain 64-bit attention and the comparison rules of the attention tests.

Tolerances, from the arithmetic that the calls promise (fp32 scores, statistics and accumulation;
softmax weights rounded once to 16 bits, the output once to bf16). Let A_i = sum_j p_ij |v_j| / l_i:
  * rounding o to bf16 (8 significant bits) costs at most 2^-8 |o|;
  * rounding the weights costs at most u A, u = 2^-8 for bf16 weights and 2^-11 for fp16 ones;
  * a score's fp32 error (up to 256 products of size a few, scaled) is below 2^-15, and shifts a
    weight by that share: 2^-14 A covers it together with exp and the fp32 sums;
  * lse carries the scores' error, 2^-15, and the fp32 rounding of its own value, 2^-22 |lse|.
"""
from __future__ import annotations

import math

import torch


def bits(x: torch.Tensor) -> torch.Tensor:
    """bf16 bit patterns as int16."""
    return x.to(torch.bfloat16).view(torch.int16)


def values(x: torch.Tensor) -> torch.Tensor:
    return x.cpu().view(torch.bfloat16).double()


def attend(q, k, v, scale, seen):
    """q [n, d], k and v [m, d] in 64 bits, seen [n, m] -> o, lse, A. Keys that a row does not see
    are left out of its sums, whatever they hold."""
    n, d = q.shape
    o, lse, size = torch.zeros(n, d).double(), torch.full((n,), -math.inf).double(), torch.zeros(n, d).double()
    for i in range(n):
        at = seen[i].nonzero()[:, 0]
        if len(at):
            s = (k[at] @ q[i]) * scale
            m = s.max()
            p = torch.exp(s - m)
            o[i] = (p @ v[at]) / p.sum()
            size[i] = (p @ v[at].abs()) / p.sum()
            lse[i] = m + torch.log(p.sum())
    return o, lse, size


def prefill(q, k, v, lens, scale, causal):
    """q [tq, hq, d], k and v [tk, hkv, d] in 64 bits; lens: (lq, lk) of each sequence."""
    hq, g = q.shape[1], q.shape[1] // k.shape[1]
    out = [torch.zeros_like(q), torch.zeros(q.shape[:2]).double(), torch.zeros_like(q)]
    a = b = 0
    for lq, lk in lens:
        i, j = torch.arange(lq)[:, None], torch.arange(lk)[None]
        seen = (j <= i + lk - lq) if causal else torch.ones(lq, lk, dtype=torch.bool)
        for h in range(hq):
            r = attend(q[a:a + lq, h], k[b:b + lk, h // g], v[b:b + lk, h // g], scale, seen)
            for to, x in zip(out, r):
                to[a:a + lq, h] = x
        a, b = a + lq, b + lk
    return out


def check(o, lse, ref, weight_bits, what=""):
    """o: bf16 bits, lse: fp32, ref: (o, lse, A); weight_bits: 8 (bf16) or 11 (fp16)."""
    ro, rl, size = ref
    got = values(o)
    assert got.shape == ro.shape
    assert torch.isfinite(got).all(), f"{what}: non-finite output"
    tol = 2.0 ** -8 * ro.abs() + (2.0 ** -weight_bits + 2.0 ** -14) * size + 1e-30
    worst = ((got - ro).abs() / tol).max().item() if ro.numel() else 0.0
    assert worst <= 1.0, f"{what}: o off by {worst:.2f} x tolerance"
    if lse is not None:
        x = lse.cpu().double()
        empty = rl == -math.inf
        assert torch.equal(x == -math.inf, empty), f"{what}: empty rows"
        d = (x - rl)[~empty].abs() / (2.0 ** -15 + 2.0 ** -22 * rl[~empty].abs())
        assert not len(d) or d.max().item() <= 1.0, f"{what}: lse off by {d.max().item():.2f} x tolerance"
