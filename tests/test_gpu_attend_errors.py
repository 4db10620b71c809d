"""Device-side errors of the model-side calls that a status word must name, and what a call
leaves untouched then."""

from __future__ import annotations

import math

import pytest
import torch

from tests import attend_ref as ref

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module")
def bkv():
    from kv_cache_eviction_head_gb300.build import build
    build()
    from kv_cache_eviction_head_gb300 import bkv as mod
    return mod


def config(bkv, heads, kv, batch, max_cache, layers=1):
    return bkv.make_config(heads=heads, kv_heads=kv, d=D, budget=1, period=16, prefix=0, recent=0, layers=layers,
                           batch=batch, max_cache=max_cache, rope_theta=1e6)


def randn(shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, device="cuda", generator=g) * scale).to(torch.bfloat16)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def new_status():
    return torch.full((1,), 77, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("cu,total", [([0, 4, 9], 8), ([-5, 0, 4], 8), ([0, 6, 4], 8), ([-2, 2, 4], 8), ([0, 9, 9], 8),
                                      ([0, 0, -1], 8), ([0, 700, 1301], 1300)])
def test_store_latches_offsets_out_of_range_or_order(bkv, cu, total):
    """No token is written but to its sequence's slots, one place behind the other."""
    batch, slots = 2, max(16, total)
    cfg = config(bkv, 4, 1, batch, slots)
    x = randn((total, 6, D), 1)
    K, V = torch.full((batch, 1, slots, D), 7.0, dtype=torch.bfloat16, device="cuda"), randn((batch, 1, slots, D), 2)
    V.fill_(7.0)
    q_rot, status = torch.empty((total, 4, D), dtype=torch.bfloat16, device="cuda"), new_status()
    bkv.bkv_store_kv(cfg, x[:, :4], x[:, 4:5], x[:, 5:], i32(cu), i32([0, 3]), i32([0, 0]), q_rot, K, V, status=status,
                     stream=torch.cuda.current_stream())
    assert int(status) == bkv.BKV_ERR_INVALID_ARG
    for b, first in enumerate([0, 3]):
        begin, end = max(cu[b], 0), min(cu[b + 1], total)
        for slot in range(min(slots, 40)):
            t = begin + slot - first
            row = V[b, 0, slot]
            if first <= slot and begin <= t < end:
                assert torch.equal(row, x[t, 5]) or bool((row == 7).all())  # its own token's or skipped
            else:
                assert bool((row == 7).all())


def test_store_looks_at_every_sequence_s_offsets(bkv):
    """300 sequences without tokens around one with some; one offset is wrong, or none."""
    batch = 300
    cfg = config(bkv, 4, 1, batch, 16)
    x = randn((5, 6, D), 1)
    K, V, q_rot = randn((batch, 1, 16, D), 2), randn((batch, 1, 16, D), 3), torch.empty((5, 4, D), dtype=torch.bfloat16, device="cuda")
    for at, value in ((None, 0), (0, -1), (299, 4), (300, 6), (40, 2)):
        cu = [0] * 100 + [5] * 201
        if at is not None:
            cu[at] = value
        status = new_status()
        bkv.bkv_store_kv(cfg, x[:, :4], x[:, 4:5], x[:, 5:], i32(cu), i32([0] * batch), i32([0] * batch), q_rot, K, V,
                         status=status, stream=torch.cuda.current_stream())
        assert int(status) == (0 if at is None else bkv.BKV_ERR_INVALID_ARG)


def attend(bkv, kind, q, K, V, past, mask=None, slots=None):
    """q [batch][n][heads][d] behind `past` slots of each sequence; (out, lse, status)."""
    batch, n, heads, _ = q.shape
    cfg = config(bkv, heads, K.shape[1], batch, K.shape[2])
    out, lse, status = torch.full_like(q, 7.0), torch.full((batch, n, heads), 7.0, device="cuda"), new_status()
    cs = torch.cuda.current_stream()
    if kind == "tree":
        bkv.bkv_attend_tree(cfg, q, K, V, i32(past), out, mask=mask, lse=lse, status=status, stream=cs)
    else:
        bkv.bkv_attend_prompt(cfg, q.reshape(-1, heads, D), K, V, i32([n * b for b in range(batch + 1)]), i32(past),
                              out.view(-1, heads, D), lse=lse.view(-1, heads), status=status, stream=cs)
    return out, lse, int(status)


def check_weightless(q, K, V, see, weightless, out, lse):
    """Rows against 64 bits with the slots of `weightless` [L] hidden; rows that see only such are NaN.
    Returns whether there is one."""
    want, wlse, tol, ltol = ref.attention(q, torch.where(weightless[None, :, None], torch.zeros_like(K), K), V, see & ~weightless)
    lost = see.any(dim=1) & ~(see & ~weightless).any(dim=1)
    assert bool(torch.isnan(out[lost]).all()) and bool(torch.isnan(lse[lost]).all())
    assert ref.close(out[~lost], want[~lost], tol[~lost]) <= 0 and ref.close(lse[~lost], wlse[~lost], ltol[~lost]) <= 0
    return bool(lost.any())


# (sequences, tokens, slots in front): split over a cluster, one tile, two tiles
@pytest.mark.parametrize("heads,kv,batch,n,past", [(8, 2, 2, 3, 900), (8, 2, 2, 3, 0), (28, 4, 2, 64, 2000), (32, 8, 1, 300, 0),
                                                   (32, 8, 12, 100, 40)])
@pytest.mark.parametrize("kind", ["prompt", "tree"])
def test_rows_that_see_only_logits_of_minus_infinity(bkv, kind, heads, kv, batch, n, past):
    """All of a sequence's keys up to its second token, then one more in the middle, are such
    that every logit is -inf: those rows are NaN and latched, the others as if the slots were
    not there; other sequences do not notice."""
    if kind == "tree":
        n = min(n, 64)
    L = past + n
    q = randn((batch, n, heads, D), 1).abs() + 0.5
    K, V = randn((batch, kv, L + 3, D), 2), randn((batch, kv, L + 3, D), 3)
    weightless = torch.zeros((batch, L), dtype=torch.bool, device="cuda")
    weightless[0, :past + 2] = True
    weightless[0, past + 2 + (n - 2) // 2:past + 3 + (n - 2) // 2] = True
    K[:, :, :L, 5] = torch.where(weightless[:, None], torch.full_like(K[:, :, :L, 5], -math.inf), K[:, :, :L, 5])
    masks = [None] if kind == "prompt" else [None, torch.tensor([[1 << i for i in range(63)] + [-1 << 63]] * batch, device="cuda")[:, :n].contiguous()]
    for mask in masks:
        out, lse, status = attend(bkv, kind, q, K, V, [past] * batch, mask)
        own = torch.arange(L, device="cuda")[None] - past - torch.arange(n, device="cuda")[:, None]
        see = own <= 0 if mask is None else (own == 0) | (torch.arange(L, device="cuda")[None] < past)
        lost = [check_weightless(q[b], K[b, :, :L], V[b, :, :L], see, weightless[b], out[b], lse[b]) for b in range(batch)]
        assert lost[0] and not any(lost[1:])
        assert status == bkv.BKV_ERR_NONFINITE


@pytest.mark.parametrize("poison", [math.inf, -math.inf])
@pytest.mark.parametrize("kind,batch,slots", [("tree", 1, 250), ("tree", 200, 250), ("prompt", 1, 250)])
def test_an_infinite_key_by_the_sign_of_the_query(bkv, kind, batch, slots, poison):
    """Heads whose logit is +inf are NaN and latched, for the others the slot has no weight."""
    heads = 4
    q, K, V = randn((batch, 1, heads, D), 1), randn((batch, 1, slots + 1, D), 2), randn((batch, 1, slots + 1, D), 3)
    K[0, 0, 17, 5] = poison
    see = torch.ones((1, slots + 1), dtype=torch.bool, device="cuda")
    weightless = torch.zeros((slots + 1,), dtype=torch.bool, device="cuda")
    weightless[17] = True
    for signs in ([1, 1, 1, 1], [-1, -1, -1, -1], [1, -1, -1, 1]):
        q[0, 0, :, 5] = torch.tensor(signs, device="cuda")
        out, lse, status = attend(bkv, kind, q, K, V, [slots] * batch)
        up = torch.tensor([s * poison > 0 for s in signs], device="cuda")
        assert bool(torch.isnan(out[0, 0, up]).all()) and not bool(torch.isfinite(lse[0, 0, up]).any())
        rest = q[0][:, ~up]
        if rest.shape[1]:
            assert not check_weightless(rest, K[0], V[0], see, weightless, out[0][:, ~up], lse[0][:, ~up])
        assert status == (bkv.BKV_ERR_NONFINITE if bool(up.any()) else 0)
        assert bool(torch.isfinite(out[1:]).all())


@pytest.mark.parametrize("length,count,bad", [(32, 0, False), (33, 0, True), (-1, 0, True), (2 ** 31 - 1, 2, True), (31, 1, False), (32, 1, True)])
def test_commit_latches_lengths_out_of_range(bkv, length, count, bad):
    cfg = config(bkv, 4, 1, 2, 32)
    K, V, status = randn((2, 1, 32, D), 1), randn((2, 1, 32, D), 2), new_status()
    K0, V0 = K.clone(), V.clone()
    bkv.bkv_commit_tree(cfg, [K], [V], i32([4, length]), i32([[0, 1], [0, 1]]), i32([2, count]), status=status,
                        stream=torch.cuda.current_stream())
    assert int(status) == (bkv.BKV_ERR_INVALID_ARG if bad else 0)
    assert torch.equal(K, K0) and torch.equal(V, V0)  # every path names its own place
