"""The calls over paged caches (bkv_store_paged, bkv_attend_paged, bkv_weigh_prompt,
bkv_evict_weight) against 64-bit statements of them."""

from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from tests import attend_ref as ref
from tests.paged_ref import D, Pool, i32, keep_set, new_status, order_free_layout, probabilities, randn, weight_sums

pytestmark = pytest.mark.gpu
SHAPES = [(4, 1), (32, 8), (40, 8), (28, 4), (8, 8), (16, 1), (32, 2), (24, 1)]
PAGES = [None, 16, 48, 64, 256]


@pytest.fixture(scope="module")
def bkv():
    from kv_cache_eviction_head_gb300.build import build
    build()
    from kv_cache_eviction_head_gb300 import bkv as mod
    return mod


def stream():
    return torch.cuda.current_stream()


# ---------------------------------------------------------------- one new token

def attend_case(bkv, heads, kv, lens, page, seed, *, decay=1.0, weighed=True, scale=1.0, status=None, strided=True):
    """Slots behind the lengths, unused pages and (where they must not be read) old weights hold NaN."""
    pool = Pool(len(lens), kv, lens, page, seed)
    cfg = pool.config(bkv, heads)
    K, V = pool.fresh(lens, seed + 100), pool.fresh(lens, seed + 300)
    wide = randn((len(lens), heads + 2, D), seed + 500, scale)
    q = wide[:, 1:1 + heads] if strided else wide[:, :heads].contiguous()
    out = torch.full((len(lens), heads, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((len(lens), heads), 7.0, dtype=torch.float32, device="cuda")
    weights = None
    if weighed:
        weights = torch.rand(pool.shape(), device="cuda") + 0.01
        for b, n in enumerate(lens):
            if n:
                page_, place = pool.at(b, n, 0 if decay == 0 else n - 1)
                weights[page_, :, place] = math.nan
        before = weights.clone()
    ws = torch.empty(bkv.bkv_attend_paged_bytes(cfg, K, pool.table, weighed=weighed), dtype=torch.uint8, device="cuda")
    status = new_status() if status is None else status
    bkv.bkv_attend_paged(cfg, q, K, V, i32(lens), out, ws, table=pool.table, lse=lse, weights=weights, decay=decay,
                         status=status, stream=stream())
    worst, touched = -math.inf, None
    if weighed:
        touched = torch.zeros(pool.shape(), dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        see = torch.ones((1, n), dtype=torch.bool, device="cuda")
        k, v = pool.get(K, b, n) if n else torch.zeros((kv, 0, D), device="cuda"), pool.get(V, b, n) if n else None
        if n == 0:
            assert bool((out[b] == 0).all()) and bool((lse[b] == -math.inf).all())
            continue
        want, wlse, tol, ltol = ref.attention(q[b:b + 1], k, v, see)
        worst = max(worst, ref.close(out[b:b + 1], want, tol), ref.close(lse[b:b + 1], wlse, ltol))
        if weighed:
            p, rel, _ = probabilities(q[b:b + 1], k, see)
            s, stol = weight_sums(p, rel, kv)
            old = pool.get(before, b, n).double()
            old = torch.zeros_like(old) if decay == 0 else torch.where(torch.arange(n, device="cuda") == n - 1, 0.0, old)
            worst = max(worst, ref.close(pool.get(weights, b, n), decay * old + s, stol + 2.0 ** -22 * (old + s)))
            page_, place = pool.at(b, n)
            touched[page_, :, place] = True
    assert int(status) == 0
    if weighed:
        assert torch.equal(weights[~touched].view(torch.int32), before[~touched].view(torch.int32))
    return worst


@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("heads,kv", SHAPES)
def test_attend_groups_and_pages(bkv, heads, kv, page):
    lens = [33, 0, 1, 15, 16, 17, 0, 250, 129]
    assert attend_case(bkv, heads, kv, lens, page, 10 + heads) <= 0


@pytest.mark.parametrize("lens", [[1], [0], [2000], [20011], [5, 0, 0, 3000], [40] * 100, [700, 1, 0, 333] * 30])
@pytest.mark.parametrize("page", [None, 16, 64])
def test_attend_few_and_many_slots(bkv, lens, page):
    assert attend_case(bkv, 28, 4, lens, page, 3) <= 0


@pytest.mark.parametrize("decay", [0.0, 0.5, 0.95, 1.0])
def test_attend_decay(bkv, decay):
    assert attend_case(bkv, 32, 8, [100, 1, 0, 64], 16, 4, decay=decay) <= 0


@pytest.mark.parametrize("heads,kv", [(128, 1), (96, 2), (40, 1)])
def test_attend_wide_groups(bkv, heads, kv):
    """More query heads than a unit takes: several chunks over the same keys, their weights one sum."""
    assert attend_case(bkv, heads, kv, [100, 0, 17, 1], 16, 5) <= 0
    assert attend_case(bkv, heads, kv, [5000], None, 6, decay=0.9) <= 0


def test_attend_without_weights(bkv):
    assert attend_case(bkv, 40, 8, [100, 0, 4000, 1], 48, 7, weighed=False) <= 0


def test_attend_large_logits(bkv):
    """Logits of some hundreds: the reference maximum moves, most probabilities vanish."""
    assert attend_case(bkv, 8, 2, [400, 90, 3000], 16, 8, scale=40.0) <= 0


def test_attend_contiguous_queries(bkv):
    assert attend_case(bkv, 8, 8, [12, 400], 16, 9, strided=False) <= 0


# ---------------------------------------------------------------- prompt weights

def weigh_case(bkv, heads, kv, lens, first, page, seed, *, decay=1.0, scale=1.0, extra=2):
    slots = [a + b for a, b in zip(lens, first)]
    pool = Pool(len(lens), kv, slots, page, seed)
    cfg = pool.config(bkv, heads)
    K = pool.fresh(slots, seed + 100)
    total = sum(lens) + extra
    wide = randn((total, heads + 3, D), seed + 500, scale)
    wide[sum(lens):] = math.nan  # tokens of no sequence
    q = wide[:, 2:2 + heads]
    lse = torch.full((total, heads), math.nan, dtype=torch.float32, device="cuda")
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    weights = torch.rand(pool.shape(), device="cuda") + 0.01
    want = []
    for b, (n, f) in enumerate(zip(lens, first)):
        want.append(None)
        if not n:
            continue
        see = torch.arange(f + n, device="cuda")[None] <= f + torch.arange(n, device="cuda")[:, None]
        p, rel, wlse = probabilities(q[cu[b]:cu[b + 1]], pool.get(K, b, f + n), see)
        lse[cu[b]:cu[b + 1]] = wlse.float()
        want[b] = weight_sums(p, rel + 2.0 ** -22 * wlse.abs(), kv)
        page_, place = pool.at(b, f + n, 0 if decay == 0 else f)
        weights[page_, :, place] = math.nan
    before = weights.clone()
    status = new_status()
    bkv.bkv_weigh_prompt(cfg, q, lse, K, i32(cu), i32(first), weights, table=pool.table, decay=decay, status=status,
                         stream=stream())
    assert int(status) == 0
    worst, touched = -math.inf, torch.zeros(pool.shape(), dtype=torch.bool, device="cuda")
    for b, (n, f) in enumerate(zip(lens, first)):
        if not n:
            continue
        s, tol = want[b]
        old = pool.get(before, b, f + n).double()
        old = torch.zeros_like(old) if decay == 0 else torch.where(torch.arange(f + n, device="cuda") >= f, 0.0, old)
        worst = max(worst, ref.close(pool.get(weights, b, f + n), decay * old + s, tol + 2.0 ** -22 * (old + s)))
        page_, place = pool.at(b, f + n)
        touched[page_, :, place] = True
    assert torch.equal(weights[~touched].view(torch.int32), before[~touched].view(torch.int32))
    return worst


@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("heads,kv", SHAPES + [(96, 1), (52, 1), (11, 1)])
def test_weigh_groups_and_pages(bkv, heads, kv, page):
    lens = [33, 0, 1, 127, 128, 0, 129, 97]
    first = [0, 5, 0, 1, 0, 0, 130, 127]
    assert weigh_case(bkv, heads, kv, lens, first, page, 10 + heads) <= 0


@pytest.mark.parametrize("decay", [0.0, 0.5, 1.0])
@pytest.mark.parametrize("lens,first", [([1], [0]), ([1], [300]), ([700], [0]), ([3, 1200], [900, 100]), ([24] * 40, [9] * 40)])
def test_weigh_few_and_many_sequences(bkv, lens, first, decay):
    assert weigh_case(bkv, 32, 8, lens, first, 16, 3, decay=decay) <= 0


@pytest.mark.parametrize("heads,kv", [(4, 1), (8, 8), (28, 4), (48, 1)])
@pytest.mark.parametrize("lens", [[1900], [900, 0, 1500, 40]])
def test_weigh_shared_by_clusters(bkv, heads, kv, lens):
    """Few tiles of slots: CTAs share a tile's queries, in numbers that do not divide them."""
    assert weigh_case(bkv, heads, kv, lens, [0] * len(lens), None, 31, decay=0.5) <= 0
    assert weigh_case(bkv, heads, kv, lens, [300] * len(lens), 64, 32, decay=0.5) <= 0


def test_weigh_large_logits(bkv):
    assert weigh_case(bkv, 8, 2, [400, 90], [0, 200], 64, 8, scale=40.0) <= 0


def test_weigh_more_tiles_than_blocks(bkv):
    """More tiles of slots than a launch has blocks: blocks take several."""
    lens = [130] * 320
    assert weigh_case(bkv, 4, 4, lens, [0] * 320, None, 9) <= 0


@pytest.mark.parametrize("heads,kv", [(8, 8), (16, 4)])
def test_weigh_chunks_of_one_tile(bkv, heads, kv):
    """Blocks take several tiles of slots, most of them seen by one tile of queries: half of the
    adding warps have none of it and come to the next item ahead of the others."""
    lens = [(1, 24, 97, 0, 23, 130, 5, 2)[b % 8] for b in range(310)]
    first = [(600, 130, 0, 50, 255, 300, 511, 17)[b % 7] for b in range(310)]
    assert weigh_case(bkv, heads, kv, lens, first, 16, 41, decay=0.5) <= 0


# ---------------------------------------------------------------- eviction by weight

def evict_case(bkv, heads, kv, lens, page, seed, *, budget, prefix=0, recent=0, layers=2, order_free=False, values=None, shift=0):
    flags = bkv.BKV_FLAG_ORDER_FREE if order_free else 0
    pool = Pool(len(lens), kv, lens, page, seed)
    cap = pool.size if pool.table is None else pool.size * pool.table.shape[1]
    if page is None and cap <= budget:
        pytest.skip("dense caches hold more than the budget")
    cfg = pool.config(bkv, heads, budget=budget, prefix=prefix, recent=recent, layers=layers, flags=flags,
                      max_cache=max(cap, budget + 1))
    g = torch.Generator(device="cuda").manual_seed(seed)
    K = [pool.fresh(lens, seed + 10 * l) for l in range(layers)]
    V = [pool.fresh(lens, seed + 500 + 10 * l) for l in range(layers)]
    W = [torch.exp(2 * torch.randn(pool.shape(), device="cuda", generator=g)) for _ in range(layers)]
    if values is not None:  # few different weights: ties, infinities, NaN
        pick = torch.tensor(values, device="cuda")
        W = [pick[torch.randint(0, len(values), pool.shape(), device="cuda", generator=g)] for _ in range(layers)]
    if shift:  # weights that begin `shift` elements behind a 16-byte boundary
        W = [torch.cat([x.new_zeros(shift), x.flatten()])[shift:].view(x.shape) for x in W]
        assert all(x.data_ptr() % 16 for x in W)
    K0, V0, W0 = ([x.clone() for x in y] for y in (K, V, W))
    kept = torch.full((layers, len(lens), kv, budget), 9999999, dtype=torch.int32, device="cuda")
    left, status = i32([5] * len(lens)), new_status()
    bkv.bkv_evict_weight(cfg, K, V, W, i32(lens), kept, table=pool.table, new_lens=left, status=status, stream=stream())
    assert int(status) == 0
    assert left.tolist() == [min(n, budget) for n in lens]
    got = kept.cpu().numpy()
    for l in range(layers):
        for old, new in ((K0[l], K[l]), (V0[l], V[l]), (W0[l], W[l])):
            want = old.clone()
            for b, n in enumerate(lens):
                if n > budget:
                    page_, place = pool.at(b, n)
                    i = torch.from_numpy(got[l, b].astype(np.int64)).cuda()
                    h = torch.arange(kv, device="cuda")[:, None]
                    want[page_[:budget], h, place[:budget]] = old[page_[i], h, place[i]]
            assert torch.equal(new.view(torch.int16), want.view(torch.int16))
        for b, n in enumerate(lens):
            w = pool.get(W0[l], b, n).cpu().numpy() if n else None
            for h in range(kv):
                if n <= budget:
                    assert got[l, b, h].tolist() == list(range(n)) + [-1] * (budget - n)
                    continue
                want = keep_set(w[h], budget, prefix, recent)
                if order_free:
                    want = order_free_layout(want, budget)
                assert np.array_equal(got[l, b, h], want)


@pytest.mark.parametrize("order_free", [False, True])
@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("budget,prefix,recent,over", [(1, 0, 0, 5), (8, 4, 4, 9), (64, 4, 16, 17), (255, 0, 16, 300), (256, 4, 0, 1),
                                                       (300, 4, 16, 16), (1000, 4, 16, 600), (31, 31, 0, 40), (33, 1, 1, 700)])
def test_evict_budgets(bkv, budget, prefix, recent, over, page, order_free):
    lens = [budget + over, 0, budget, 1, budget + recent + 1, budget + max(recent, 1)]
    evict_case(bkv, 4, 2, lens, page, 11, budget=budget, prefix=prefix, recent=recent, order_free=order_free)


@pytest.mark.parametrize("order_free", [False, True])
@pytest.mark.parametrize("values", [[1.0], [0.0, -0.0], [0.0, 1.0, 2.0], [math.nan, 1.0, math.inf], [math.nan], [-math.inf, -1.0, 0.0, math.nan],
                                    [1.0, 1.0000001, 1.0000002]])
def test_evict_ties_and_odd_weights(bkv, values, order_free):
    evict_case(bkv, 4, 1, [200, 90, 130], 16, 12, budget=70, prefix=4, recent=7, order_free=order_free, values=values)


@pytest.mark.parametrize("order_free", [False, True])
@pytest.mark.parametrize("shift", [1, 2, 3])
def test_evict_weights_off_the_boundary(bkv, shift, order_free):
    evict_case(bkv, 4, 2, [200, 131, 70, 94], 16, 18, budget=70, prefix=3, recent=7, order_free=order_free, shift=shift)


@pytest.mark.parametrize("over", [8, 9, 10, 11])
def test_evict_dense_caches_of_any_size(bkv, over):
    evict_case(bkv, 4, 2, [120 + over, 120, 119 + over], None, 19, budget=100, prefix=3, recent=7)


@pytest.mark.parametrize("order_free", [False, True])
@pytest.mark.parametrize("length,budget,prefix,recent", [(9001, 8400, 8300, 30), (8210, 8100, 4, 40), (9001, 8230, 4, 820), (8192, 8000, 0, 0),
                                                         (8193, 100, 50, 50)])
def test_evict_around_the_keys_on_chip(bkv, length, budget, prefix, recent, order_free):
    """Candidates, prefix and recent slots on either side of the 8,192nd."""
    if order_free and length - 1 - budget < recent:
        pytest.skip("an order-free eviction refuses sequences this short")
    evict_case(bkv, 2, 2, [length, length - 1], 16, 21, budget=budget, prefix=prefix, recent=recent, layers=1, order_free=order_free)


def test_evict_many_layers_and_sequences(bkv):
    evict_case(bkv, 4, 1, [60, 50, 40] * 20, 16, 13, budget=45, prefix=1, recent=2, layers=7)


@pytest.mark.parametrize("over", [7, 700])
def test_evict_many_units_order_free(bkv, over):
    """More than 304 units, with few dropped slots below the budget and with more than a list holds."""
    lens = [800 + over, 800 + over + 3, 800] * 20
    evict_case(bkv, 8, 2, lens, None, 15, budget=800, prefix=1, recent=4, layers=3, order_free=True)


def test_evict_long(bkv):
    evict_case(bkv, 4, 2, [9000], 64, 14, budget=4096, prefix=4, recent=16, layers=1)
    evict_case(bkv, 4, 2, [9000], None, 14, budget=5000, prefix=4, recent=16, layers=1, order_free=True)
    evict_case(bkv, 4, 1, [20000, 17000], 16, 14, budget=12345, prefix=4, recent=16, layers=1, values=[0.0, 1.0, 2.0, 3.0])
    evict_case(bkv, 4, 1, [20000], 16, 14, budget=12345, prefix=4, recent=16, layers=1, order_free=True, values=[0.0, 1.0])


# ---------------------------------------------------------------- rotary store

def frequencies(theta, r, scaling, factor, original):
    f, scale = [], 1.0
    for i in range(r // 2):
        w = theta ** (-2.0 * i / r)
        if scaling == "linear":
            w /= factor
        if scaling == "ntk":
            w = (theta * factor ** (r / (r - 2.0))) ** (-2.0 * i / r)
        if scaling == "yarn":
            g = min(1.0, max(0.0, (original * w / (2 * math.pi) - 1.0) / 31.0))
            w = (1 - g) * w / factor + g * w
            scale = 0.1 * math.log(factor) + 1.0
        f.append(w)
    return f, scale


def turned(x, pos, f, scale, interleaved):
    """x [tokens][heads][d] in float64, and how far fp32 arithmetic rounded to bf16 may be off: an
    angle is within pos 2^-53 + 2^-24 turns (2^-22 of the elements' size with the cosine's own
    error), products and sums 2^-22, the result's rounding 2^-8."""
    y = x.double().clone()
    r = 2 * len(f)
    if r == 0:
        return y, torch.zeros_like(y)
    a = pos.double()[:, None, None] * torch.tensor(f, dtype=torch.float64, device="cuda")
    c, s = torch.cos(a) * scale, torch.sin(a) * scale
    lo, hi = (y[..., 0:r:2], y[..., 1:r:2]) if interleaved else (y[..., :r // 2], y[..., r // 2:r])
    lo, hi = lo.clone(), hi.clone()
    size = (lo.abs() + hi.abs()) * scale
    new = torch.stack([lo * c - hi * s, hi * c + lo * s], dim=-1)
    err = torch.stack([size, size], dim=-1) * (2.0 ** -21 + float(pos.abs().max()) * 2.0 ** -50)
    new, err = (new.flatten(-2), err.flatten(-2)) if interleaved else (torch.cat(list(new.unbind(-1)), -1), torch.cat(list(err.unbind(-1)), -1))
    tol = torch.zeros_like(y)
    y[..., :r] = new
    tol[..., :r] = err + ref.BF16 * (new.abs() + err)
    return y, tol


def store_case(bkv, heads, kv, lens, first, page, seed, *, r=128, interleaved=False, scaling="none", factor=1.0, pos0=0, depths=False,
               extra=2, theta=1e6, in_place=False):
    slots = [a + b for a, b in zip(lens, first)]
    pool = Pool(len(lens), kv, slots, page, seed)
    cfg = pool.config(bkv, heads)
    K, V = pool.fresh(slots, seed + 100, fill=5.0), pool.fresh(slots, seed + 200, fill=5.0)
    total = sum(lens) + extra
    x = randn((total, heads + 2 * kv, D), seed + 300)
    q, k, v = x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:]
    if in_place:
        q = q.contiguous()
    q0 = q.clone()
    rope = bkv.make_rope(theta=theta, rotary_dim=r, interleaved=interleaved, scaling=scaling, factor=factor, original_len=4096)
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    pos = i32([pos0 + 5 * b for b in range(len(lens))])
    depth = torch.randint(0, 30, (total,), dtype=torch.int32, device="cuda") if depths else None
    q_rot = q if in_place else torch.full((total, heads, D), 7.0, dtype=torch.bfloat16, device="cuda")
    K0, V0, status = K.clone(), V.clone(), new_status()
    bkv.bkv_store_paged(cfg, rope, q, k, v, i32(cu), i32(first), pos, q_rot, K, V, table=pool.table, depth=depth, status=status,
                        stream=stream())
    assert int(status) == 0
    f, scale = frequencies(theta, r, scaling, factor, 4096)
    worst = -math.inf
    for b, (n, start) in enumerate(zip(lens, first)):
        a = cu[b]
        where = pos[b].long() + (depth[a:a + n] if depths else torch.arange(n, device="cuda"))
        if n:
            worst = max(worst, ref.close(q_rot[a:a + n], *turned(q0[a:a + n], where, f, scale, interleaved)))
            want, tol = turned(k[a:a + n], where, f, scale, interleaved)
            page_, place = pool.at(b, start + n, start)
            worst = max(worst, ref.close(K[page_, :, place], want, tol))
            assert torch.equal(V[page_, :, place], v[a:a + n])
            K0[page_, :, place], V0[page_, :, place] = K[page_, :, place], V[page_, :, place]
    assert torch.equal(K, K0) and torch.equal(V, V0)  # no other slot
    behind = q_rot[sum(lens):]
    assert torch.equal(behind, q0[sum(lens):]) if in_place else bool((behind == 7).all())
    return worst


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("r", [0, 16, 32, 64, 80, 96, 128])
@pytest.mark.parametrize("heads,kv,page", [(4, 1, None), (40, 8, 16), (28, 4, 48)])
def test_store_layouts(bkv, heads, kv, page, r, interleaved):
    assert store_case(bkv, heads, kv, [3, 0, 1, 70], [0, 4, 15, 30], page, 20, r=r, interleaved=interleaved) <= 0


@pytest.mark.parametrize("scaling,factor", [("linear", 4.0), ("ntk", 2.5), ("yarn", 8.0), ("yarn", 1.0)])
@pytest.mark.parametrize("pos0", [0, 131071, 2 ** 31 - 200])
def test_store_scalings_and_far_positions(bkv, scaling, factor, pos0):
    for r, interleaved in ((128, False), (64, True)):
        assert store_case(bkv, 8, 2, [20, 9], [0, 3], 16, 21, r=r, interleaved=interleaved, scaling=scaling, factor=factor, pos0=pos0) <= 0


@pytest.mark.parametrize("lens", [[1] * 50, [1500], [700, 0, 900]])
def test_store_few_and_many_tokens(bkv, lens):
    assert store_case(bkv, 32, 8, lens, [3] * len(lens), 64, 22, depths=True) <= 0


def test_store_in_place(bkv):
    assert store_case(bkv, 8, 2, [20, 9], [0, 3], 16, 23, in_place=True) <= 0


def test_store_of_own_frequencies(bkv):
    """The rotate-half layout with theta's own frequencies is bkv_store_kv's, up to a rounding."""
    heads, kv, n = 8, 2, 33
    cfg = bkv.make_config(heads=heads, kv_heads=kv, d=D, budget=1, period=16, prefix=0, recent=0, layers=1, batch=1, max_cache=64,
                          rope_theta=1e4)
    x = randn((n, heads + 2 * kv, D), 24)
    args = (x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:], i32([0, n]), i32([5]), i32([77]))
    got = []
    for new in (False, True):
        K, V = torch.zeros((1, kv, 64, D), dtype=torch.bfloat16, device="cuda"), torch.zeros((1, kv, 64, D), dtype=torch.bfloat16, device="cuda")
        q = torch.empty((n, heads, D), dtype=torch.bfloat16, device="cuda")
        if new:
            rope = bkv.make_rope(rotary_dim=128, inv_freq=[1e4 ** (-2.0 * i / 128) for i in range(64)])
            bkv.bkv_store_paged(cfg, rope, *args, q, K, V, stream=stream())
        else:
            bkv.bkv_store_kv(cfg, *args, q, K, V, stream=stream())
        got.append((q, K, V))
    assert torch.equal(got[0][2], got[1][2])
    for a, b in zip(got[0][:2], got[1][:2]):
        assert float((a.float() - b.float()).abs().max()) <= 2.0 ** -7 * 4  # a frequency's last bit may move a rounding by a step
