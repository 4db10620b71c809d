"""Attention over caches of 2^17 slots, in every form of the kernel: the far tiles, the borders
of the key shares and the last slots all count. A few keys of each cache are aligned with the
queries, so that every row is the mean of their values and one of them left out shows."""

from __future__ import annotations

import math

import pytest
import torch

from tests import attend_ref as ref

pytestmark = pytest.mark.gpu
D = 128
SLOTS = 1 << 17


@pytest.fixture(scope="module")
def bkv():
    from kv_cache_eviction_head_gb300.build import build
    build()
    from kv_cache_eviction_head_gb300 import bkv as mod
    return mod


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# split over clusters of 16 and 4, one tile per CTA unsplit, two tiles split and unsplit
@pytest.mark.parametrize("kind,heads,kv,n", [("tree", 8, 2, 3), ("prompt", 8, 2, 3), ("tree", 32, 32, 1), ("tree", 160, 160, 1),
                                             ("tree", 160, 80, 64),
                                             ("tree", 28, 4, 64), ("tree", 280, 40, 64), ("prompt", 32, 8, 700)])
def test_far_slots(bkv, kind, heads, kv, n):
    g = torch.Generator(device="cuda").manual_seed(heads + n)
    normal = lambda *shape: torch.randn(shape, device="cuda", generator=g)
    past = SLOTS - n
    u = normal(D)
    u *= math.sqrt(D) / u.norm()
    K = torch.empty((1, kv, SLOTS, D), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    V = torch.empty_like(K).normal_(generator=g)
    q = (u + 0.1 * normal(1, n, heads, D)).to(torch.bfloat16)
    # logits of about 25 against a sum of exponentials of the others of about e^12
    share = past // 16
    at = [0, 127, 128, *(share * i // 128 * 128 + j for i in (1, 5, 8, 11, 15) for j in (-1, 0)), past - 129, past - 1, SLOTS - 1]
    at += [past, past + n // 2]
    K[0][:, at] = (25 * math.sqrt(D) / D * u + 0.02 * normal(kv, len(at), D)).to(torch.bfloat16)
    cfg = bkv.make_config(heads=heads, kv_heads=kv, d=D, budget=1, period=16, prefix=0, recent=0, layers=1, batch=1,
                          max_cache=SLOTS, rope_theta=1e6)
    out, lse = torch.empty_like(q), torch.empty((1, n, heads), device="cuda")
    status, cs = i32([77]), torch.cuda.current_stream()
    if kind == "tree":
        bkv.bkv_attend_tree(cfg, q, K, V, i32([past]), out, lse=lse, status=status, stream=cs)
    else:
        bkv.bkv_attend_prompt(cfg, q[0], K, V, i32([0, n]), i32([past]), out[0], lse=lse[0], status=status, stream=cs)
    assert int(status) == 0
    see = torch.arange(SLOTS, device="cuda")[None] <= past + torch.arange(n, device="cuda")[:, None]
    G = heads // kv
    for h in sorted({0, heads // 2 - 1, heads - 1}):
        k = slice(h // G, h // G + 1)
        want, wlse, tol, ltol = ref.attention(q[0, :, h:h + 1], K[0, k], V[0, k], see)
        assert ref.close(out[0, :, h:h + 1], want, tol) <= 0 and ref.close(lse[0, :, h:h + 1], wlse, ltol) <= 0
        # the bounds are narrow enough for one slot of `at` left out
        less = see.clone()
        less[:, at[7]] = False
        other, olse, _, _ = ref.attention(q[0, -1:, h:h + 1], K[0, k], V[0, k], less[-1:])
        assert ref.close(other, want[-1:], tol[-1:]) > 0 and ref.close(olse, wlse[-1:], ltol[-1:]) > 0
