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
