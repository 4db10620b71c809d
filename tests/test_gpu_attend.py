"""The model-side calls over the caches (bkv_store_kv, bkv_attend_prompt,
bkv_attend_tree, bkv_commit_tree) against 64-bit statements of them."""

from __future__ import annotations

import math

import numpy as np
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


def config(bkv, heads, kv_heads, batch, max_cache, layers=1, theta=1e6):
    return bkv.make_config(heads=heads, kv_heads=kv_heads, d=D, budget=1, period=16, prefix=0, recent=0, layers=layers,
                           batch=batch, max_cache=max_cache, rope_theta=theta)


def randn(shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, device="cuda", generator=g) * scale).to(torch.bfloat16)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def new_status():
    return torch.full((1,), 77, dtype=torch.int32, device="cuda")


def prompt_case(bkv, heads, kv, lens, first, seed, *, extra=0, scale=1.0, status=None, slack=3):
    """Runs a packed prompt whose unused slots hold NaN; returns the largest excesses."""
    batch = len(lens)
    max_cache = max(max(a + b for a, b in zip(lens, first)) + slack, 2)
    total = sum(lens) + extra
    cfg = config(bkv, heads, kv, batch, max_cache)
    K, V = randn((batch, kv, max_cache, D), seed), randn((batch, kv, max_cache, D), seed + 1)
    for b in range(batch):
        K[b, :, first[b] + lens[b]:] = math.nan
        V[b, :, first[b] + lens[b]:] = math.nan
    wide = randn((total, heads + 3, D), seed + 2, scale)
    q = wide[:, 1:1 + heads]  # tokens (heads + 3) * d elements apart
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    out = torch.full((total, heads, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((total, heads), 7.0, dtype=torch.float32, device="cuda")
    status = new_status() if status is None else status
    bkv.bkv_attend_prompt(cfg, q, K, V, i32(cu), i32(first), out, lse=lse, status=status,
                          stream=torch.cuda.current_stream())
    worst = -math.inf
    for b in range(batch):
        n, f = lens[b], first[b]
        see = torch.arange(f + n, device="cuda")[None] <= f + torch.arange(n, device="cuda")[:, None]
        want, wlse, tol, ltol = ref.attention(q[cu[b]:cu[b + 1]], K[b, :, :f + n], V[b, :, :f + n], see)
        worst = max(worst, ref.close(out[cu[b]:cu[b + 1]], want, tol), ref.close(lse[cu[b]:cu[b + 1]], wlse, ltol))
    assert int(status) == 0
    assert bool((out[sum(lens):] == 7).all()) and bool((lse[sum(lens):] == 7).all())  # rows of no sequence stay
    return worst


@pytest.mark.parametrize("heads,kv", [(4, 1), (6, 6), (10, 2), (7, 1), (16, 1), (128, 1), (96, 1)])
def test_prompt_lengths_and_groups(bkv, heads, kv):
    """Lengths around the tile and token-block borders, empty sequences, cached slots in front."""
    lens = [33, 0, 1, 127, 128, 0, 129, 31]
    first = [0, 5, 0, 1, 0, 0, 130, 127]
    assert prompt_case(bkv, heads, kv, lens, first, 10 + heads, extra=3) <= 0


@pytest.mark.parametrize("lens,first", [([1], [0]), ([1], [300]), ([700], [0]), ([5, 260], [0, 0]), ([64] * 40, [0] * 40)])
def test_prompt_few_and_many_sequences(bkv, lens, first):
    assert prompt_case(bkv, 32, 8, lens, first, 3) <= 0


@pytest.mark.parametrize("heads,kv", [(32, 8), (40, 8), (28, 4)])
def test_prompt_two_tiles_per_block(bkv, heads, kv):
    """Enough row blocks for the two-tile kernel: ragged ends in the first and the second tile."""
    lens = [300, 257, 64, 65, 1, 17, 0, 191, 450, 33, 96, 128]
    first = [0, 129, 3, 0, 0, 0, 9, 64, 0, 500, 0, 1]
    assert prompt_case(bkv, heads, kv, lens, first, 5, extra=1) <= 0


@pytest.mark.parametrize("heads,kv", [(7, 1), (32, 8)])
@pytest.mark.parametrize("lens,first", [([1], [4000]), ([5, 0, 3], [3000, 900, 0]), ([40, 70], [1500, 127])])
def test_prompt_chunks_behind_a_long_context(bkv, heads, kv, lens, first):
    """Few row blocks: their keys are split over clusters."""
    assert prompt_case(bkv, heads, kv, lens, first, 6, extra=2) <= 0


def test_prompt_large_logits(bkv):
    """Logits of some hundreds, whose running maximum moves from tile to tile."""
    assert prompt_case(bkv, 8, 2, [400, 90], [0, 200], 8, scale=40.0) <= 0


def random_mask(batch, n, seed, empty=True):
    """Random trees' ancestor bits; some rows see nothing of the tree."""
    rs = np.random.RandomState(seed)
    bits = np.zeros((batch, n), np.uint64)
    for b in range(batch):
        for i in range(n):
            p = rs.randint(-1, i) if i else -1
            bits[b, i] = (bits[b, p] if p >= 0 else np.uint64(0)) | np.uint64(1 << i)
        if empty and n > 2:
            bits[b, rs.randint(0, n)] = 0
    return torch.from_numpy(bits.view(np.int64)).cuda()


def tree_case(bkv, heads, kv, n, lens, seed, *, mask=None, nodes=None, max_cache=None, scale=1.0, contiguous=True):
    batch = len(lens)
    max_cache = max_cache or max(lens) + n + 5
    cfg = config(bkv, heads, kv, batch, max_cache)
    used = nodes or [n] * batch
    K, V = randn((batch, kv, max_cache, D), seed), randn((batch, kv, max_cache, D), seed + 1)
    for b in range(batch):
        K[b, :, lens[b] + used[b]:] = math.nan
        V[b, :, lens[b] + used[b]:] = math.nan
    q = randn((batch, n, heads, D), seed + 2, scale)
    if not contiguous:
        wide = torch.zeros((batch, n, heads + 2, D), dtype=torch.bfloat16, device="cuda")
        wide[:, :, 2:] = q
        q = wide[:, :, 2:]
    out = torch.full((batch, n, heads, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((batch, n, heads), 7.0, dtype=torch.float32, device="cuda")
    status = new_status()
    bkv.bkv_attend_tree(cfg, q, K, V, i32(lens), out, mask=mask, nodes=None if nodes is None else i32(nodes), lse=lse,
                        status=status, stream=torch.cuda.current_stream())
    worst = -math.inf
    for b in range(batch):
        m, L = used[b], lens[b]
        see = torch.ones((m, L + m), dtype=torch.bool, device="cuda")
        for i in range(m):
            word = (int(mask[b, i]) & (2 ** 64 - 1)) if mask is not None else (1 << (i + 1)) - 1
            see[i, L:] = torch.tensor([bool((word >> j) & 1) for j in range(m)], device="cuda")
        want, wlse, tol, ltol = ref.attention(q[b, :m], K[b, :, :L + m], V[b, :, :L + m], see)
        worst = max(worst, ref.close(out[b, :m], want, tol), ref.close(lse[b, :m], wlse, ltol))
        assert bool((out[b, m:] == 7).all()) and bool((lse[b, m:] == 7).all())
    assert int(status) == 0
    return worst


@pytest.mark.parametrize("heads,kv", [(4, 1), (8, 8), (10, 2), (14, 2), (128, 1)])
@pytest.mark.parametrize("lens", [[0, 1, 126, 127], [128, 1000, 2063, 250]])
def test_decode(bkv, heads, kv, lens):
    assert tree_case(bkv, heads, kv, 1, lens, heads) <= 0


@pytest.mark.parametrize("n", [2, 7, 31, 33, 64])
@pytest.mark.parametrize("heads,kv", [(4, 1), (14, 2)])
def test_tree_masks(bkv, n, heads, kv):
    lens = [0, 3, 127, 128 - n, 700]
    assert tree_case(bkv, heads, kv, n, lens, 20 + n, mask=random_mask(5, n, n), contiguous=False) <= 0


@pytest.mark.parametrize("n,heads,kv", [(5, 8, 2), (64, 40, 8)])
def test_tree_ragged_node_counts(bkv, n, heads, kv):
    nodes = [n, 0, 1, n - 1, n // 2]
    assert tree_case(bkv, heads, kv, n, [50, 60, 0, 127, 513], 31, mask=random_mask(5, n, 2), nodes=nodes) <= 0


def test_tree_chain_without_a_mask_and_bits_behind_the_nodes(bkv):
    assert tree_case(bkv, 8, 2, 9, [0, 64, 300], 41) <= 0
    mask = random_mask(3, 9, 4) | torch.tensor(-1 << 40, device="cuda")  # bits 40..63: no such nodes
    assert tree_case(bkv, 8, 2, 9, [0, 64, 300], 42, mask=mask) <= 0


def test_tree_row_that_sees_nothing(bkv):
    """Empty cache and an empty mask: zeros and a log-sum-exp of -inf, also across a split."""
    for max_cache in (64, 4096):
        mask = torch.zeros((2, 3), dtype=torch.int64, device="cuda")
        mask[:, 1] = 2
        assert tree_case(bkv, 4, 1, 3, [0, 0], 51, mask=mask, max_cache=max_cache) <= 0


@pytest.mark.parametrize("batch,kv,max_cache", [(1, 1, 8192), (1, 8, 8192), (3, 8, 4096), (40, 8, 300)])
def test_tree_key_splits(bkv, batch, kv, max_cache):
    """From sixteen CTAs per row block down to one; a share may have no tile."""
    lens = [(7919 * (b + 1)) % (max_cache - 8) for b in range(batch)]
    lens[0] = max_cache - 4
    assert tree_case(bkv, 4 * kv, kv, 4, lens, 61, mask=random_mask(batch, 4, 1), max_cache=max_cache) <= 0


def test_tree_results_do_not_vary(bkv):
    cfg = config(bkv, 8, 2, 1, 5000)
    K, V, q = randn((1, 2, 5000, D), 1), randn((1, 2, 5000, D), 2), randn((1, 1, 8, D), 3)
    outs = []
    for _ in range(20):
        out, lse = torch.empty_like(q), torch.empty((1, 1, 8), dtype=torch.float32, device="cuda")
        bkv.bkv_attend_tree(cfg, q, K, V, i32([4900]), out, lse=lse, stream=torch.cuda.current_stream())
        outs.append((out, lse))
    assert all(torch.equal(o, outs[0][0]) and torch.equal(l, outs[0][1]) for o, l in outs)


@pytest.mark.parametrize("theta,positions", [(1e6, [0, 7, 40000]), (1e4, [2_000_000_000, -1000, 131071])])
@pytest.mark.parametrize("depths", [False, True])
def test_store(bkv, theta, positions, depths):
    heads, kv, lens, first, max_cache = 10, 2, [5, 0, 38], [3, 0, 9], 64
    total, slack = sum(lens), 2
    cfg = config(bkv, heads, kv, 3, max_cache, theta=theta)
    qkv = randn((total + slack, heads + 2 * kv, D), 5)
    q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
    K, V = randn((3, kv, max_cache, D), 6), randn((3, kv, max_cache, D), 7)
    K0, V0 = K.clone(), V.clone()
    q_rot = torch.full((total + slack, heads, D), 7.0, dtype=torch.bfloat16, device="cuda")
    depth = torch.randint(0, 9, (total + slack,), dtype=torch.int32, device="cuda") if depths else None
    status = new_status()
    cu = [0, 5, 5, 43]
    bkv.bkv_store_kv(cfg, q, k, v, i32(cu), i32(first), i32(positions), q_rot, K, V, depth=depth, status=status,
                     stream=torch.cuda.current_stream())
    assert int(status) == 0
    for b in range(3):
        s = slice(cu[b], cu[b + 1])
        at = torch.arange(lens[b], device="cuda") if depth is None else depth[s].long()
        pos = positions[b] + at.long()
        # fp32 pairs: the angle's error, in turns of 2 pi, moves a component by as much of the pair's
        # norm: 2^-25 turns from the fp32 fraction, |pos| 2^-52 from the reference's own fp64 angle
        # and this one's fraction; sine, cosine and two products add 2^-21. Then one bf16 rounding.
        angle = 2 * math.pi * 2.0 ** -25 + float(pos.abs().max() if lens[b] else 0) * 2.0 ** -51
        for x, y in ((q[s], q_rot[s]), (k[s], K[b, :, first[b]:first[b] + lens[b]].transpose(0, 1))):
            want = ref.rope(x, pos, theta)
            lo, hi = x.double()[..., :64], x.double()[..., 64:]
            norm = torch.sqrt(lo ** 2 + hi ** 2).repeat(1, 1, 2) * (angle + 2.0 ** -21)
            assert ref.close(y, want, norm + ref.BF16 * (want.abs() + norm)) <= 0
        assert torch.equal(V[b, :, first[b]:first[b] + lens[b]].transpose(0, 1), v[s])
        for now, before in ((K, K0), (V, V0)):  # other slots stay
            assert torch.equal(now[b, :, :first[b]], before[b, :, :first[b]])
            assert torch.equal(now[b, :, first[b] + lens[b]:], before[b, :, first[b] + lens[b]:])
    assert bool((q_rot[total:] == 7).all())


def test_store_in_place_and_slots_out_of_range(bkv):
    heads, kv, max_cache = 4, 1, 16
    cfg = config(bkv, heads, kv, 2, max_cache)
    q, k, v = randn((6, heads, D), 1), randn((6, kv, D), 2), randn((6, kv, D), 3)
    K, V = randn((2, kv, max_cache, D), 4), randn((2, kv, max_cache, D), 5)
    K0 = K.clone()
    cu, pos = i32([0, 3, 6]), i32([0, 100])
    apart, status = torch.empty_like(q), new_status()
    args = (cfg, q, k, v, cu, i32([14, -1]), pos)
    bkv.bkv_store_kv(*args, apart, K, V, status=status, stream=torch.cuda.current_stream())
    assert int(status) == bkv.BKV_ERR_INVALID_ARG
    kr = ref.rope(k, torch.tensor([0, 1, 2, 100, 101, 102], device="cuda"), 1e6)
    assert torch.equal(K[0, :, :14], K0[0, :, :14]) and torch.equal(K[1, :, 2:], K0[1, :, 2:])
    assert float((K[0, 0, 14:].double() - kr[:2, 0]).abs().max()) < 0.05
    assert float((K[1, 0, :2].double() - kr[4:6, 0]).abs().max()) < 0.05
    bkv.bkv_store_kv(*args, q, K, V, status=status, stream=torch.cuda.current_stream())
    assert torch.equal(q, apart)


@pytest.mark.parametrize("n", [1, 5, 64])
def test_commit(bkv, n):
    layers, batch, kv, max_cache = 3, 4, 2, 100
    cfg = config(bkv, 2 * kv, kv, batch, max_cache, layers=layers)
    lens = [0, 20, max_cache - n, 7]
    rs = np.random.RandomState(n)
    path = np.stack([np.sort(rs.permutation(n)), rs.permutation(n), np.arange(n), rs.randint(0, n, n)]).astype(np.int32)
    count = [max(1, n // 2), n, n, n]
    K = [randn((batch, kv, max_cache, D), 10 + l) for l in range(layers)]
    V = [randn((batch, kv, max_cache, D), 20 + l) for l in range(layers)]
    want = [[t.clone() for t in ts] for ts in (K, V)]
    for ts, old in zip(want, (K, V)):
        for l in range(layers):
            for b in range(batch):
                for i in range(count[b]):
                    ts[l][b, :, lens[b] + i] = old[l][b, :, lens[b] + int(path[b, i])]
    path[0, count[0]:] = 99  # not read
    status = new_status()
    bkv.bkv_commit_tree(cfg, K, V, i32(lens), torch.from_numpy(path).cuda(), i32(count), status=status,
                        stream=torch.cuda.current_stream())
    assert int(status) == 0
    for got, ts in zip((K, V), want):
        assert all(torch.equal(a, b) for a, b in zip(got, ts))


def test_lengths_out_of_range_are_latched_and_nothing_else_is_touched(bkv):
    """The kernels clamp them: the outputs stay in the tensors, the status names the error."""
    cs = torch.cuda.current_stream()
    cfg = config(bkv, 4, 1, 2, 32)
    K, V = randn((2, 1, 32, D), 1), randn((2, 1, 32, D), 2)
    for lens, nodes in (([-5, 3], None), ([31, 3], None), ([40, 3], None), ([3, 3], [9, -1])):
        q = randn((2, 4, 4, D), 3)
        out, status = torch.zeros_like(q), new_status()
        bkv.bkv_attend_tree(cfg, q, K, V, i32(lens), out, nodes=None if nodes is None else i32(nodes), status=status, stream=cs)
        assert int(status) == bkv.BKV_ERR_INVALID_ARG
    for cu, first in (([0, 4, 9], [0, 0]), ([0, 6, 4], [0, 0]), ([-2, 2, 4], [0, 0]), ([0, 4, 8], [30, 0]), ([0, 4, 8], [0, -1])):
        q = randn((8, 4, D), 3)
        out, status = torch.zeros_like(q), new_status()
        bkv.bkv_attend_prompt(cfg, q, K, V, i32(cu), i32(first), out, status=status, stream=cs)
        assert int(status) == bkv.BKV_ERR_INVALID_ARG
    for lens, path, count in (([0, 0], [0, 4], [2, 2]), ([0, 0], [-1, 0], [2, 2]), ([31, 0], [1, 0], [2, 2]), ([-1, 0], [1, 0], [2, 2]), ([0, 0], [1, 0], [3, 2]), ([0, 0], [1, 0], [-1, 2])):
        K1, V1, status = K.clone(), V.clone(), new_status()
        bkv.bkv_commit_tree(cfg, [K1], [V1], i32(lens), i32([path, [0, 1]]), i32(count), status=status, stream=cs)
        assert int(status) == bkv.BKV_ERR_INVALID_ARG
        assert torch.equal(K1[1], K[1]) and torch.equal(V1[1], V[1])


@pytest.mark.parametrize("poison", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("where", ["K", "V", "q"])
def test_visible_non_finite_values_are_latched(bkv, poison, where):
    cs = torch.cuda.current_stream()
    cfg = config(bkv, 4, 1, 1, 300)
    t = {"K": randn((1, 1, 300, D), 1), "V": randn((1, 1, 300, D), 2), "q": randn((1, 1, 4, D), 3)}
    if where == "q":
        t["q"][0, 0, 2, 5] = poison
    else:
        t[where][0, 0, 17, 5] = poison
    out, status = torch.empty_like(t["q"]), new_status()
    bkv.bkv_attend_tree(cfg, t["q"], t["K"], t["V"], i32([250]), out, status=status, stream=cs)
    if not (where == "K" and poison == -math.inf) and not (where == "K" and poison == math.inf):
        assert int(status) == bkv.BKV_ERR_NONFINITE
    else:  # q * inf is +inf for some heads and -inf for others, which then give the key no weight
        finite = bool(torch.isfinite(out).all())
        assert (int(status) == 0) == finite


def test_empty_calls(bkv):
    cs = torch.cuda.current_stream()
    cfg = config(bkv, 4, 1, 2, 32)
    K, V = randn((2, 1, 32, D), 1), randn((2, 1, 32, D), 2)
    K0, V0 = K.clone(), V.clone()
    e = lambda h: torch.empty((0, h, D), dtype=torch.bfloat16, device="cuda")
    status = new_status()
    bkv.bkv_store_kv(cfg, e(4), e(1), e(1), i32([0, 0, 0]), i32([0, 0]), i32([0, 0]), e(4), K, V, status=status, stream=cs)
    assert int(status) == 0 and torch.equal(K, K0) and torch.equal(V, V0)
    bkv.bkv_attend_prompt(cfg, e(4), K, V, i32([0, 0, 0]), i32([0, 0]), e(4), stream=cs)
    q = randn((2, 3, 4, D), 1)
    out = torch.full_like(q, 7.0)
    bkv.bkv_attend_tree(cfg, q, K, V, i32([4, 4]), out, nodes=i32([0, 0]), stream=cs)
    assert bool((out == 7).all())
    bkv.bkv_commit_tree(cfg, [K], [V], i32([4, 4]), i32([[0], [0]]), i32([0, 0]), stream=cs)
    assert torch.equal(K, K0) and torch.equal(V, V0)


@pytest.mark.parametrize("poison", [math.nan, math.inf])
def test_query_rows_of_nobody_reach_no_other_row(bkv, poison):
    """Rows of unused nodes, of tokens around the sequences and of a neighbour sequence lie in
    the same 128-row tiles: whatever they hold, the others' results keep their bits."""
    cs = torch.cuda.current_stream()
    for heads, kv, n, used in ((8, 2, 5, [2, 0, 5]), (40, 8, 64, [1, 40, 64])):
        cfg = config(bkv, heads, kv, 3, 700)
        K, V, q = randn((3, kv, 700, D), 1), randn((3, kv, 700, D), 2), randn((3, n, heads, D), 3)
        outs = []
        for fill in (0.0, poison):
            x = q.clone()
            for b, m in enumerate(used):
                x[b, m:] = fill
            out, lse, status = torch.full_like(q, 7.0), torch.full((3, n, heads), 7.0, device="cuda"), new_status()
            bkv.bkv_attend_tree(cfg, x, K, V, i32([0, 300, 620]), out, nodes=i32(used), lse=lse, status=status, stream=cs)
            assert int(status) == 0
            outs.append((out, lse))
        assert all(torch.equal(a, b) for a, b in zip(*outs))
        assert all(bool((outs[0][0][b, m:] == 7).all()) for b, m in enumerate(used))
    for heads, kv, lens in ((8, 2, [20, 11, 30]), (32, 8, [200, 170, 65])):
        cfg = config(bkv, heads, kv, 3, 700)
        cu = [3, 3 + lens[0], 3 + lens[0] + lens[1], 3 + sum(lens)]
        total = cu[-1] + 9
        K, V, q = randn((3, kv, 700, D), 1), randn((3, kv, 700, D), 2), randn((total, heads, D), 3)
        outs = []
        for fill in (0.0, poison):
            x = q.clone()
            x[:cu[0]] = fill
            x[cu[1]:cu[2]] = fill  # the sequence between the two that are compared
            x[cu[3]:] = fill
            out, status = torch.full_like(q, 7.0), new_status()
            bkv.bkv_attend_prompt(cfg, x, K, V, i32(cu), i32([0, 5, 100]), out, status=status, stream=cs)
            assert int(status) == (0 if fill == 0.0 else bkv.BKV_ERR_NONFINITE)
            outs.append(torch.cat((out[:cu[1]], out[cu[2]:])))
        assert torch.equal(*outs)


@pytest.mark.parametrize("heads,kv", [(32, 8), (28, 4), (2, 1), (5, 5)])
def test_prompt_last_tiles_end_anywhere(bkv, heads, kv):
    """Blocks of one and of two row tiles, whose keys end in every quarter of a tile, one after
    the other on the same SM (more row blocks than SMs)."""
    rng = torch.Generator().manual_seed(heads)
    lens = [int(x) for x in torch.randint(1, 300, (48,), generator=rng)]
    first = [int(x) for x in torch.randint(0, 200, (48,), generator=rng)]
    first[::3] = [0] * len(first[::3])
    assert prompt_case(bkv, heads, kv, lens, first, 5) <= 0


@pytest.mark.parametrize("n,heads,kv", [(1, 8, 2), (9, 8, 2), (40, 28, 4), (64, 28, 4)])
def test_tree_last_tiles_end_anywhere(bkv, n, heads, kv):
    ends = [n, 127, 128, 129, 159, 160, 161, 191, 192, 193, 223, 224, 225, 255, 256, 257]
    lens = [max(e - n, 0) for e in ends] * 4
    assert tree_case(bkv, heads, kv, n, lens, 6, mask=random_mask(len(lens), n, 7)) <= 0


@pytest.mark.parametrize("heads,kv", [(28, 4), (40, 8), (3, 1)])
def test_results_do_not_depend_on_what_ran_before(bkv, heads, kv):
    """Rows of a tile behind its last one hold what an earlier call left on the SM; a row
    keeps its bits whatever they are."""
    cs = torch.cuda.current_stream()
    cfg = config(bkv, heads, kv, 20, 900)
    K, V, q = randn((20, kv, 900, D), 1), randn((20, kv, 900, D), 2), randn((20, 40, heads, D), 3)
    K2, q2 = randn((20, kv, 900, D), 4, 30.0), randn((20, 40, heads, D), 5, 30.0)
    lens, cu = i32([40 * b for b in range(20)]), i32([40 * b for b in range(21)])
    flat = lambda t: t.view(-1, heads, D)
    tree, prompt = [torch.zeros_like(q) for _ in range(5)], [torch.zeros_like(q) for _ in range(5)]
    for i in range(4):
        bkv.bkv_attend_tree(cfg, q, K, V, lens, tree[i], stream=cs)
        bkv.bkv_attend_prompt(cfg, flat(q), K, V, cu, lens, flat(prompt[i]), stream=cs)
        if i % 2 == 0:
            bkv.bkv_attend_tree(cfg, q2, K2, V, lens, tree[4], stream=cs)
            bkv.bkv_attend_prompt(cfg, flat(q2), K2, V, cu, lens, flat(prompt[4]), stream=cs)
    assert all(torch.equal(t, tree[0]) for t in tree[1:4]) and all(torch.equal(t, prompt[0]) for t in prompt[1:4])
