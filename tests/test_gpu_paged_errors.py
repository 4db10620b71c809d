"""Errors that the calls over paged caches find on the device: latched in the status word,
clamped or skipped, and nothing outside the tensors touched."""

from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from tests import attend_ref as ref
from tests.paged_ref import D, Pool, i32, new_status, probabilities, randn, weight_sums

pytestmark = pytest.mark.gpu
INVALID, NONFINITE = 1, 5


@pytest.fixture(scope="module")
def bkv():
    from kv_cache_eviction_head_gb300.build import build
    build()
    from kv_cache_eviction_head_gb300 import bkv as mod
    return mod


def stream():
    return torch.cuda.current_stream()


def guarded(shape, dtype, fill):
    """A tensor with guard bands, and a check that they are untouched."""
    n = int(np.prod(shape))
    whole = torch.full((n + 256,), 77, dtype=dtype, device="cuda")
    inner = whole[128:128 + n].view(shape)
    inner.fill_(fill)
    return inner, lambda: bool((whole[:128] == 77).all()) and bool((whole[128 + n:] == 77).all())


def attend(bkv, cfg, pool, K, V, lens, weights, heads, seed=3, decay=1.0, table=None):
    q = randn((pool.batch, heads, D), seed)
    out, ok = guarded((pool.batch, heads, D), torch.bfloat16, 5.0)
    lse = torch.full((pool.batch, heads), 7.0, device="cuda")
    table = pool.table if table is None else table
    ws = torch.empty(bkv.bkv_attend_paged_bytes(cfg, K, table, weighed=weights is not None), dtype=torch.uint8, device="cuda")
    status = new_status()
    bkv.bkv_attend_paged(cfg, q, K, V, i32(lens), out, ws, table=table, lse=lse, weights=weights, decay=decay, status=status, stream=stream())
    assert ok()
    return q, out, lse, int(status)


@pytest.mark.parametrize("page", [None, 16])
@pytest.mark.parametrize("given", [-1, -2 ** 31, 10 ** 6, 2 ** 31 - 1])
def test_attend_lengths_out_of_range(bkv, page, given):
    """Clamped to what the table can hold; the neighbours get theirs."""
    slots = [64, 64, 64]
    pool = Pool(3, 2, slots, page, 1)
    cap = pool.size if page is None else 16 * pool.table.shape[1]
    if page:
        pool.table[1] = torch.arange(pool.table.shape[1], device="cuda") % pool.pages  # every entry names a page
    K, V = pool.fresh(slots, 5, fill=0.25), pool.fresh(slots, 6, fill=0.25)
    q, out, lse, status = attend(bkv, pool.config(bkv, 8), pool, K, V, [40, given, 64], None, 8)
    assert status == INVALID
    if given < 0:
        assert bool((out[1] == 0).all()) and bool((lse[1] == -math.inf).all())
    else:
        k, v = (x[1] if page is None else x[pool.table[1].long()].transpose(0, 1).reshape(2, cap, D) for x in (K, V))
        want, _, tol, _ = ref.attention(q[1:2], k, v, torch.ones((1, cap), dtype=torch.bool, device="cuda"))
        assert ref.close(out[1:2], want, tol) <= 0
    for b, n in ((0, 40), (2, 64)):
        want, _, tol, _ = ref.attention(q[b:b + 1], pool.get(K, b, n), pool.get(V, b, n), torch.ones((1, n), dtype=torch.bool, device="cuda"))
        assert ref.close(out[b:b + 1], want, tol) <= 0


@pytest.mark.parametrize("bad", [-1, -2 ** 31, 10 ** 6, 2 ** 31 - 1])
@pytest.mark.parametrize("heads,kv", [(8, 2), (24, 1)])
def test_attend_pages_out_of_range(bkv, bad, heads, kv):
    """The slots of a page that is none get no weight."""
    slots = [70, 33]
    pool = Pool(2, kv, slots, 16, 2)
    K, V = pool.fresh(slots, 5), pool.fresh(slots, 6)
    table = pool.table.clone()
    table[0, 1] = bad
    weights, ok = guarded(pool.shape(), torch.float32, 2.0)
    q, out, lse, status = attend(bkv, pool.config(bkv, heads), pool, K, V, slots, weights, heads, table=table)
    assert status == INVALID and ok()
    k, v = pool.get(K, 0, 70), pool.get(V, 0, 70)
    see = torch.ones((1, 70), dtype=torch.bool, device="cuda")
    see[:, 16:32] = False
    want, wlse, tol, ltol = ref.attention(q[:1], k, v, see)
    assert ref.close(out[:1], want, tol) <= 0 and ref.close(lse[:1], wlse, ltol) <= 0
    p, rel, _ = probabilities(q[:1], k, see)
    s, stol = weight_sums(p, rel, kv)
    got, old = pool.get(weights, 0, 70), torch.full((kv, 70), 2.0, dtype=torch.float64, device="cuda")
    old[:, 69] = 0
    old[:, 16:32] = 2.0
    assert ref.close(got, old + s, stol + 2.0 ** -22 * (old + s)) <= 0


def test_attend_shared_pages_without_weights(bkv):
    """Two sequences that begin with the same pages."""
    pool = Pool(2, 2, [64, 96], 16, 3)
    K, V = pool.fresh([64, 96], 5), pool.fresh([64, 96], 6)
    table = pool.table.clone()
    table[0, :3] = table[1, :3]
    q, out, lse, status = attend(bkv, pool.config(bkv, 8), pool, K, V, [64, 96], None, 8, table=table)
    assert status == 0
    k, v = (torch.cat([pool.get(x, 1, 48), pool.get(x, 0, 64)[:, 48:]], dim=1) for x in (K, V))
    want, _, tol, _ = ref.attention(q[:1], k, v, torch.ones((1, 64), dtype=torch.bool, device="cuda"))
    assert ref.close(out[:1], want, tol) <= 0


def test_attend_more_tiles_than_the_pool_has(bkv):
    """Weights with every sequence on the same pages: refused before anything is out of range."""
    pool = Pool(1, 2, [64], 16, 4, extra=0)
    K, V = pool.fresh([64], 5), pool.fresh([64], 6)
    pool.batch = 7
    weights, ok = guarded(pool.shape(), torch.float32, 2.0)
    table = pool.table[:, :4].repeat(7, 1).contiguous()
    cfg = bkv.make_config(heads=8, kv_heads=2, d=D, budget=1, period=16, prefix=0, recent=0, layers=1, batch=7, max_cache=64, rope_theta=1e6)
    _, _, _, status = attend(bkv, cfg, pool, K, V, [64] * 7, weights, 8, table=table)
    assert status == INVALID and ok() and bool((weights == 2).all())


@pytest.mark.parametrize("where", ["key", "value", "query"])
@pytest.mark.parametrize("lens", [[40, 50], [9000, 50]])
def test_attend_non_finite(bkv, where, lens):
    """Latched, and no other sequence's matter."""
    pool = Pool(2, 2, lens, 16, 5)
    K, V = pool.fresh(lens, 5), pool.fresh(lens, 6)
    page, place = pool.at(0, 21, 20)
    if where == "key":
        K[page, 1, place, 3] = math.nan
    if where == "value":
        V[page, 1, place, 3] = math.inf
    cfg = pool.config(bkv, 8)
    if where != "query":
        q, out, lse, status = attend(bkv, cfg, pool, K, V, lens, None, 8)
        assert status == NONFINITE
        assert not bool(torch.isfinite(out[0, 4:].float()).all()) and bool(torch.isfinite(out[0, :4].float()).all())
    else:
        q = randn((2, 8, D), 9)
        q[0, 2] = math.nan
        out = torch.zeros_like(q)
        ws = torch.empty(bkv.bkv_attend_paged_bytes(cfg, K, pool.table), dtype=torch.uint8, device="cuda")
        status = new_status()
        bkv.bkv_attend_paged(cfg, q, K, V, i32(lens), out, ws, table=pool.table, status=status, stream=stream())
        assert int(status) == NONFINITE
        assert bool(torch.isnan(out[0, 2].float()).all()) and bool(torch.isfinite(out[0, 3:].float()).all())
    assert bool(torch.isfinite(out[1].float()).all())


@pytest.mark.parametrize("lens", [[5, 50], [7000, 50]])
def test_attend_only_logits_of_minus_infinity(bkv, lens):
    """Infinite keys of the other sign: no slot has weight, the row is NaN and latched, not zeros."""
    pool = Pool(2, 1, lens, 16, 6)
    K, V = pool.fresh(lens, 5), pool.fresh(lens, 6)
    pool.put(K, 0, lens[0], torch.full((1, lens[0], D), -math.inf, device="cuda"))
    q = randn((2, 4, D), 9).abs() + 0.5
    out = torch.zeros_like(q)
    cfg = pool.config(bkv, 4)
    ws = torch.empty(bkv.bkv_attend_paged_bytes(cfg, K, pool.table), dtype=torch.uint8, device="cuda")
    status = new_status()
    bkv.bkv_attend_paged(cfg, q, K, V, i32(lens), out, ws, table=pool.table, status=status, stream=stream())
    assert int(status) == NONFINITE
    assert bool(torch.isnan(out[0].float()).all()) and bool(torch.isfinite(out[1].float()).all())


@pytest.mark.parametrize("cu,first", [([0, 20, 10, 40], [0, 0, 0]), ([-5, 10, 20, 30], [0, 0, 0]), ([0, 10, 20, 2 ** 31 - 1], [0, 0, 0]),
                                      ([0, 10, 20, 30], [0, -1, 0]), ([0, 10, 20, 30], [0, 10 ** 6, 0]), ([0, 10, 20, 30], [0, 60, 0])])
@pytest.mark.parametrize("page", [None, 16])
def test_weigh_offsets_out_of_range(bkv, cu, first, page):
    pool = Pool(3, 2, [64] * 3, page, 7)
    cap = pool.size if page is None else 16 * pool.table.shape[1]
    K = pool.fresh([64] * 3, 5, fill=0.5)
    q, lse = randn((40, 8, D), 8), torch.full((40, 8), 4.0, device="cuda")
    weights, ok = guarded(pool.shape(), torch.float32, 2.0)
    status = new_status()
    bkv.bkv_weigh_prompt(pool.config(bkv, 8), q, lse, K, i32(cu), i32(first), weights, table=pool.table, status=status, stream=stream())
    assert ok()
    if first != [0, 60, 0] or 60 + 10 > cap:
        assert int(status) == INVALID
    assert bool(torch.isfinite(weights).all())


def test_weigh_pages_out_of_range_and_odd_rows(bkv):
    """A page that is none, a row whose log-sum-exp is -inf (gives nothing) and one that is NaN."""
    pool = Pool(1, 1, [48], 16, 8)
    K = pool.fresh([48], 5)
    cfg = pool.config(bkv, 4)
    q, lse = randn((48, 4, D), 8), torch.full((48, 4), 4.0, device="cuda")
    args = (i32([0, 48]), i32([0]))
    one, two, part = (torch.zeros(pool.shape(), device="cuda") for _ in range(3))
    status = new_status()
    bkv.bkv_weigh_prompt(cfg, q, lse, K, *args, one, table=pool.table, status=status, stream=stream())
    assert int(status) == 0
    lse[7, 2] = -math.inf
    bkv.bkv_weigh_prompt(cfg, q, lse, K, *args, two, table=pool.table, status=status, stream=stream())
    assert int(status) == 0
    k = pool.get(K, 0, 48)[0].double()
    gone = torch.exp(q[7, 2].double() @ k.T / math.sqrt(D) - 4.0) * (torch.arange(48, device="cuda") <= 7)
    a, b = pool.get(one, 0, 48)[0].double(), pool.get(two, 0, 48)[0].double()
    assert float((a - gone - b).abs().max()) <= 2.0 ** -18 * float(a.max())
    table = pool.table.clone()
    table[0, 1] = -7
    bkv.bkv_weigh_prompt(cfg, q, lse, K, *args, part, table=table, status=status, stream=stream())
    assert int(status) == INVALID
    got = pool.get(part, 0, 48)[0].double()
    assert bool((got[16:32] == 0).all()) and torch.equal(got[:16], b[:16]) and torch.equal(got[32:], b[32:])
    lse[40, 1] = math.nan
    bkv.bkv_weigh_prompt(cfg, q, lse, K, *args, part, table=pool.table, status=status, stream=stream())
    assert int(status) == NONFINITE
    got = pool.get(part, 0, 48)[0]
    assert bool(torch.isnan(got[:41]).all()) and bool(torch.isfinite(got[41:]).all())


@pytest.mark.parametrize("odd", [math.nan, math.inf])
def test_weigh_onto_odd_weights(bkv, odd):
    """An old weight that is not finite stays so and is latched, unless decay is 0 or the slot is new."""
    pool = Pool(1, 1, [48], 16, 8)
    K = pool.fresh([48], 5)
    cfg = pool.config(bkv, 4)
    q, lse = randn((8, 4, D), 8), torch.full((8, 4), 4.0, device="cuda")
    for slot, decay, bad in [(39, 1.0, True), (39, 0.0, False), (40, 1.0, False)]:
        W, status = torch.zeros(pool.shape(), device="cuda"), new_status()
        page, place = pool.at(0, slot + 1, slot)
        W[page, :, place] = odd
        bkv.bkv_weigh_prompt(cfg, q, lse, K, i32([0, 8]), i32([40]), W, table=pool.table, decay=decay, status=status, stream=stream())
        assert int(status) == (NONFINITE if bad else 0)
        assert int((~torch.isfinite(pool.get(W, 0, 48))).sum()) == (1 if bad else 0)


@pytest.mark.parametrize("heads,group_fills", [(4, True), (5, False)])
def test_weigh_infinite_key(bkv, heads, group_fills):
    """A key of infinities: its logits are infinite, the other slots' as ever, whether the query
    heads fill the tiles of columns or not."""
    pool = Pool(1, 1, [300], 16, 9)
    K = pool.fresh([300], 5)
    page, place = pool.at(0, 11, 10)
    K[page, :, place] = -math.inf
    q, lse = (randn((300, heads, D), 8).abs() + 0.5), torch.full((300, heads), 9.0, device="cuda")
    weights, status = torch.zeros(pool.shape(), device="cuda"), new_status()
    bkv.bkv_weigh_prompt(pool.config(bkv, heads), q, lse, K, i32([0, 300]), i32([0]), weights, table=pool.table, status=status, stream=stream())
    assert int(status) == 0
    got = pool.get(weights, 0, 300)[0]
    assert float(got[10]) == 0.0 and bool(torch.isfinite(got).all()) and bool((got[11:] > 0).all())


@pytest.mark.parametrize("order_free", [False, True])
def test_evict_out_of_range(bkv, order_free):
    """Lengths are clamped, a bad page's slots rank last and do not move; the neighbours are evicted."""
    lens = [60, 60, 60]
    pool = Pool(3, 2, lens, 16, 10)
    flags = bkv.BKV_FLAG_ORDER_FREE if order_free else 0
    cfg = pool.config(bkv, 4, budget=40, prefix=2, recent=4, max_cache=64, flags=flags)
    (K, okK), (V, okV) = (guarded(pool.shape() + (D,), torch.bfloat16, 0.0) for _ in range(2))
    K.copy_(pool.fresh(lens, 5, fill=1.0)), V.copy_(pool.fresh(lens, 6, fill=1.0))
    W, okW = guarded(pool.shape(), torch.float32, 0.0)
    W.copy_(torch.rand(pool.shape(), device="cuda"))
    kept, okk = guarded((1, 3, 2, 40), torch.int32, -9)
    left, status = i32([0, 0, 0]), new_status()
    table = pool.table.clone()
    table[1, 1] = 10 ** 6
    before = K.clone()
    bkv.bkv_evict_weight(cfg, [K], [V], [W], i32([-3, 60, 60]), kept, table=table, new_lens=left, status=status, stream=stream())
    assert int(status) == INVALID and okK() and okV() and okW() and okk()
    assert left.tolist() == [0, 40, 40]
    assert bool((kept[0, 0] == -1).all()) and bool((kept[0, 1:] >= 0).all()) and bool((kept[0, 1:] < 60).all())
    assert torch.equal(pool.get(K, 0, 60), pool.get(before, 0, 60))
    i = kept[0, 2].long()
    if order_free:
        assert sorted(i[0].tolist()) == sorted(set(i[0].tolist()))
    now, old = pool.get(K, 2, 60)[:, :40], pool.get(before, 2, 60)
    assert torch.equal(now, torch.gather(old, 1, i[..., None].expand(-1, -1, D)))


def test_evict_order_free_too_short(bkv):
    """Fewer slots over the budget than the recent window: refused, and nothing moves."""
    lens = [44, 41, 60, 40]
    pool = Pool(4, 1, lens, 16, 11)
    cfg = pool.config(bkv, 4, budget=40, prefix=2, recent=5, max_cache=64, flags=bkv.BKV_FLAG_ORDER_FREE)
    K, V, W = pool.fresh(lens, 5), pool.fresh(lens, 6), torch.rand(pool.shape(), device="cuda")
    before, kept, left, status = K.clone(), torch.zeros((1, 4, 1, 40), dtype=torch.int32, device="cuda"), i32([0] * 4), new_status()
    bkv.bkv_evict_weight(cfg, [K], [V], [W], i32(lens), kept, table=pool.table, new_lens=left, status=status, stream=stream())
    assert int(status) == INVALID and left.tolist() == [44, 41, 40, 40]
    assert bool((kept[0, :2] == -1).all()) and kept[0, 3, 0].tolist() == list(range(40))
    for b in (0, 1, 3):
        assert torch.equal(pool.get(K, b, lens[b]), pool.get(before, b, lens[b]))


def test_store_out_of_range(bkv):
    """Slots outside the table and on no page: the query is turned, nothing is written."""
    pool = Pool(3, 2, [40, 40, 40], 16, 12)
    cfg, cap = pool.config(bkv, 4), 16 * pool.table.shape[1]
    (K, okK), (V, okV) = (guarded(pool.shape() + (D,), torch.bfloat16, 3.0) for _ in range(2))
    x = randn((6, 8, D), 5)
    q_rot, ok = guarded((6, 4, D), torch.bfloat16, 7.0)
    table = pool.table.clone()
    table[2, 0] = -1
    status = new_status()
    bkv.bkv_store_paged(cfg, bkv.make_rope(), x[:, :4], x[:, 4:6], x[:, 6:], i32([0, 2, 4, 6]), i32([cap - 1, -1, 0]), i32([0, 0, 0]), q_rot, K, V,
                        table=table, status=status, stream=stream())
    assert int(status) == INVALID and okK() and okV() and ok()
    assert not bool((q_rot == 7).all(dim=-1).any())
    written = (V != 3).any(dim=-1).sum()
    # sequence 0's last entry names no page; sequence 1's second token is slot 0
    assert int(written) == 2 and torch.equal(V[pool.table[1, 0].long(), :, 0], x[3, 6:])
