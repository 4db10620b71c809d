"""64-bit statements of the model-side calls, for the tests: attention of one
sequence's rows with a visibility matrix, RoPE, and how far a kernel that holds
logits and sums in fp32 and rounds the probabilities and the output to bf16 may
be from them."""

from __future__ import annotations

import math

import torch

BF16 = 2.0 ** -8   # half a step, relative: torch.finfo(torch.bfloat16).eps / 2
D = 128


def attention(q, K, V, see):
    """q [n][H][d], K, V [kv][L][d] (bf16), see [n][L] -> (out, lse, out_tol, lse_tol), all
    float64, [n][H][d] and [n][H].

    Tolerances. A logit is a 128-term fp32 sum, off by at most 127 * 2^-23 * sum |q_i k_i|
    whatever the order and rounding direction, scaled by 1/sqrt(d); the scaling, the exponent
    and ex2.approx (2 ulp) add at most (|l| log2 e + 4) * 2^-22. With that bound, e, over the
    row's visible keys, every exponential and the row's sum are within a factor exp(e), and
    summing n of them in fp32 adds n * 2^-24. A probability is rounded to bf16 (2^-8), the
    product sum adds n * 2^-23, the output's rounding 2^-8 of its value."""
    n, H, _ = q.shape
    kv, L = K.shape[:2]
    G = H // kv
    out = torch.zeros((n, H, D), dtype=torch.float64, device=q.device)
    lse = torch.full((n, H), -math.inf, dtype=torch.float64, device=q.device)
    out_tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    if n == 0 or L == 0:
        return out, lse, out_tol, lse_tol
    for h in range(H):
        x, k, v = q[:, h].double(), K[h // G].double(), V[h // G].double()
        l = (x @ k.T / math.sqrt(D)).masked_fill(~see, -math.inf)
        any_key = see.any(dim=1)
        size = (x.abs() @ k.abs().T / math.sqrt(D)).masked_fill(~see, 0.0).amax(dim=1)
        e = 127 * 2.0 ** -23 * size + (l.masked_fill(~see, 0.0).abs().amax(dim=1) * 1.4427 + 4) * 2.0 ** -22
        lse[:, h] = torch.logsumexp(l, dim=1)
        p = torch.exp(l - lse[:, h:h + 1]).masked_fill(~see, 0.0)
        out[:, h] = torch.where(any_key[:, None], p @ v, torch.zeros((), dtype=torch.float64, device=q.device))
        lse_tol[:, h] = e + L * 2.0 ** -24 + lse[:, h].masked_fill(~any_key, 0.0).abs() * 2.0 ** -22
        spread = (p @ v.abs()) * (BF16 + 2 * e + L * 2.0 ** -23 + L * 2.0 ** -24)[:, None]
        out_tol[:, h] = torch.where(any_key[:, None], spread + BF16 * (out[:, h].abs() + spread), spread * 0)
    return out, lse, out_tol, lse_tol


def close(got, want, tol):
    """Largest excess over the tolerance (<= 0: within); equal infinities count as equal."""
    g = got.double()
    same = (g == want) & torch.isinf(want)
    off = torch.where(same, torch.zeros_like(g), (g - want).abs() - tol)
    return float(torch.nan_to_num(off, nan=math.inf).max()) if off.numel() else 0.0


def rope(x, pos, theta):
    """x [tokens][heads][d] rotated to pos [tokens], float64."""
    inv = torch.tensor([theta ** (-2.0 * i / D) for i in range(D // 2)], dtype=torch.float64, device=x.device)
    a = pos.double()[:, None, None] * inv
    c, s = torch.cos(a), torch.sin(a)
    lo, hi = x.double()[..., :D // 2], x.double()[..., D // 2:]
    return torch.cat([lo * c - hi * s, hi * c + lo * s], dim=-1)
