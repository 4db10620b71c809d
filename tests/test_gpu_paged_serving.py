"""The calls over paged caches as a program uses them: a prompt's weights, decode steps that
keep the account, evictions by it, in dense caches and in pages; in captured graphs and on
several streams; pools that 32-bit offsets do not reach; the bounds-checked build."""

from __future__ import annotations

import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from tests import attend_ref as ref
from tests.paged_ref import D, Pool, i32, keep_set, new_status, probabilities, randn, weight_sums

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def bkv():
    from kv_cache_eviction_head_gb300.build import build
    build()
    from kv_cache_eviction_head_gb300 import bkv as mod
    return mod


def stream():
    return torch.cuda.current_stream()


@pytest.mark.parametrize("page", [None, 16, 32])
def test_prompt_decode_and_eviction_together(bkv, page):
    """Two ragged prompts are stored, attended (over dense caches; copied to the pages where the
    program has pages) and weighed, evicted by weight, and decoded for three rounds of steps with an
    eviction after each. Every output, weight and keep set is checked against 64 bits on the
    caches as they are; nothing is waited for inside a round."""
    layers, heads, kv, budget, period, prefix, recent = 2, 8, 2, 48, 8, 2, 4
    prompts = [60, 37]
    batch, cap = 2, 96
    pool = Pool(batch, kv, [cap] * batch, page, 1)
    if page is None:
        pool.size = cap
        pool.where = [np.full(cap, b) for b in range(batch)], [np.arange(cap)] * batch
    cfg = pool.config(bkv, heads, budget=budget, period=period, prefix=prefix, recent=recent, layers=layers, max_cache=cap)
    rope = bkv.make_rope(theta=1e4, rotary_dim=64, interleaved=True, scaling="yarn", factor=4.0, original_len=64)
    K = [torch.full(pool.shape() + (D,), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(layers)]
    V = [torch.full_like(K[0], math.nan) for _ in range(layers)]
    W = [torch.full(pool.shape(), math.nan, device="cuda") for _ in range(layers)]
    ws = [torch.empty(bkv.bkv_attend_paged_bytes(cfg, K[0], pool.table, weighed=True), dtype=torch.uint8, device="cuda") for _ in range(layers)]
    kept, status = torch.empty((layers, batch, kv, budget), dtype=torch.int32, device="cuda"), new_status()
    kw = dict(table=pool.table, stream=stream())
    seed = iter(range(1000, 9000))
    total = sum(prompts)
    cu, zero = i32([0, prompts[0], total]), i32([0, 0])
    for l in range(layers):
        x = randn((total, heads + 2 * kv, D), next(seed))
        q, out, lse = torch.empty((total, heads, D), dtype=torch.bfloat16, device="cuda"), torch.empty((total, heads, D), dtype=torch.bfloat16, device="cuda"), torch.empty((total, heads), device="cuda")
        bkv.bkv_store_paged(cfg, rope, x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:], cu, zero, zero, q, K[l], V[l], **kw)
        if page is None:
            bkv.bkv_attend_prompt(cfg, q, K[l], V[l], cu, zero, out, lse=lse, stream=stream())
        else:
            dense = [torch.zeros((batch, kv, cap, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
            bkv.bkv_store_paged(cfg, rope, x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:], cu, zero, zero, q, *dense, stream=stream())
            bkv.bkv_attend_prompt(cfg, q, *dense, cu, zero, out, lse=lse, stream=stream())
        bkv.bkv_weigh_prompt(cfg, q, lse, K[l], cu, zero, W[l], decay=0.0, status=status, **kw)
        for b, n in enumerate(prompts):
            rows = q[int(cu[b]):int(cu[b + 1])]
            see = torch.ones((n, n), dtype=torch.bool, device="cuda").tril()
            p, rel, wlse = probabilities(rows, pool.get(K[l], b, n), see)
            s, tol = weight_sums(p, rel + 2.0 ** -22 * wlse.abs(), kv)
            # the log-sum-exps are the attention kernel's, within their own bound
            _, _, _, ltol = ref.attention(rows, pool.get(K[l], b, n), pool.get(V[l], b, n), see)
            assert ref.close(pool.get(W[l], b, n), s, tol + s * float(ltol.max())) <= 0
            want, _, otol, _ = ref.attention(rows, pool.get(K[l], b, n), pool.get(V[l], b, n), see)
            assert ref.close(out[int(cu[b]):int(cu[b + 1])], want, otol) <= 0
    lens = list(prompts)
    position = list(prompts)
    for round_ in range(4):
        before = [[t.clone() for t in ts] for ts in (K, V, W)]
        left = i32([0] * batch)
        bkv.bkv_evict_weight(cfg, K, V, W, i32(lens), kept, new_lens=left, status=status, **kw)
        assert int(status) == 0 and left.tolist() == [min(n, budget) for n in lens]
        for l in range(layers):
            for b, n in enumerate(lens):
                w = pool.get(before[2][l], b, n)
                for h in range(kv):
                    i = kept[l, b, h, :min(n, budget)].cpu().numpy()
                    assert np.array_equal(i, keep_set(w[h].cpu().numpy(), budget, prefix, recent) if n > budget else np.arange(n))
                    for now, old in zip((K, V, W), before):
                        assert torch.equal(pool.get(now[l], b, len(i))[h], pool.get(old[l], b, n)[h, torch.from_numpy(i.astype(np.int64)).cuda()])
        lens = [min(n, budget) for n in lens]
        if round_ == 3:
            break
        for _ in range(period):
            first, pos = i32(lens), i32(position)
            lens, position = [n + 1 for n in lens], [n + 1 for n in position]
            now = i32(lens)
            old_w = [w.clone() for w in W]
            got = []
            for l in range(layers):
                x = randn((batch, heads + 2 * kv, D), next(seed))
                q, out = torch.empty((batch, heads, D), dtype=torch.bfloat16, device="cuda"), torch.empty((batch, heads, D), dtype=torch.bfloat16, device="cuda")
                bkv.bkv_store_paged(cfg, rope, x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:], i32([0, 1, 2]), first, pos, q, K[l], V[l], **kw)
                bkv.bkv_attend_paged(cfg, q, K[l], V[l], now, out, ws[l], weights=W[l], decay=0.9, status=status, **kw)
                got.append((q, out))
            assert int(status) == 0
            for l, (q, out) in enumerate(got):
                for b, n in enumerate(lens):
                    see = torch.ones((1, n), dtype=torch.bool, device="cuda")
                    want, _, tol, _ = ref.attention(q[b:b + 1], pool.get(K[l], b, n), pool.get(V[l], b, n), see)
                    assert ref.close(out[b:b + 1], want, tol) <= 0
                    p, rel, _ = probabilities(q[b:b + 1], pool.get(K[l], b, n), see)
                    s, stol = weight_sums(p, rel, kv)
                    old = pool.get(old_w[l], b, n).double()
                    old[:, n - 1] = 0
                    assert ref.close(pool.get(W[l], b, n), 0.9 * old + s, stol + 2.0 ** -22 * (old + s)) <= 0


def step_state(bkv, seed, page=16, lens=(70, 33, 0, 129), heads=8, kv=2):
    """A decode step, a prompt chunk's weights and an eviction over one pool, ready to be called."""
    lens = list(lens)
    pool = Pool(len(lens), kv, [n + 40 for n in lens], page, seed)
    cfg = pool.config(bkv, heads, budget=60, prefix=2, recent=4)
    s = dict(pool=pool, cfg=cfg, K=pool.fresh([n + 40 for n in lens], seed), V=pool.fresh([n + 40 for n in lens], seed + 50), lens=i32(lens),
             q=randn((len(lens), heads, D), seed + 90), W=torch.rand(pool.shape(), device="cuda"), status=new_status(),
             x=randn((len(lens), heads + 2 * kv, D), seed + 91), kept=torch.zeros((1, len(lens), kv, 60), dtype=torch.int32, device="cuda"),
             cu=i32(list(range(0, 10 * len(lens) + 1, 10))), qp=randn((10 * len(lens), heads, D), seed + 92),
             lse=torch.full((10 * len(lens), heads), 5.0, device="cuda"), rope=bkv.make_rope(), heads=heads, kv=kv)
    s["out"], s["q_rot"] = torch.zeros_like(s["q"]), torch.zeros_like(s["q"])
    s["ws"] = torch.empty(bkv.bkv_attend_paged_bytes(cfg, s["K"], pool.table, weighed=True), dtype=torch.uint8, device="cuda")
    return s


def step(bkv, s, cs):
    h, kv, kw = s["heads"], s["kv"], dict(table=s["pool"].table, status=s["status"], stream=cs)
    x = s["x"]
    bkv.bkv_store_paged(s["cfg"], s["rope"], x[:, :h], x[:, h:h + kv], x[:, h + kv:], i32_range(len(x)), s["lens"], s["lens"], s["q_rot"], s["K"], s["V"], **kw)
    bkv.bkv_weigh_prompt(s["cfg"], s["qp"], s["lse"], s["K"], s["cu"], s["lens"], s["W"], decay=0.5, **kw)
    bkv.bkv_attend_paged(s["cfg"], s["q"], s["K"], s["V"], s["lens"], s["out"], s["ws"], weights=s["W"], decay=0.5, **kw)
    bkv.bkv_evict_weight(s["cfg"], [s["K"]], [s["V"]], [s["W"]], s["lens"], s["kept"], **kw)


_ranges = {}


def i32_range(n):
    if n not in _ranges:
        _ranges[n] = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    return _ranges[n]


def results(s):
    return [s[x].clone() for x in ("K", "V", "W", "out", "q_rot", "kept", "status")]


def same(a, b):
    return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)) for x, y in zip(a, b))


def test_captured_and_replayed_with_other_lengths(bkv):
    """Lengths and tables are read at replay; the bits are those of plain calls, every time."""
    s = step_state(bkv, 3)
    saved = {x: s[x].clone() for x in ("K", "V", "W", "lens")}
    table = s["pool"].table
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    i32_range(4)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(bkv, s, side)
    other = torch.stack([table[1], table[0], table[3], table[2]])  # two pairs of sequences change their pages
    for lens, pages in (([70, 33, 0, 129], table.clone()), ([5, 66, 1, 60], other), ([0, 0, 0, 0], table.clone()), ([72, 1, 9, 100], table.clone())):
        got = []
        for replay in (True, True, False):
            for x in ("K", "V", "W"):
                s[x].copy_(saved[x])
            s["out"].zero_(), s["q_rot"].zero_(), s["kept"].zero_()
            s["lens"].copy_(i32(lens))
            table.copy_(pages)
            torch.cuda.synchronize()
            if replay:
                graph.replay()
            else:
                step(bkv, s, torch.cuda.current_stream())
            torch.cuda.synchronize()
            got.append(results(s))
        assert same(got[0], got[1]) and same(got[0], got[2])


def test_several_streams_and_graphs_at_once(bkv):
    """Six states on six streams, a workspace each, give what they give alone."""
    states = [step_state(bkv, 20 + k, page=[None, 16, 64][k % 3]) for k in range(6)]
    first = [{x: s[x].clone() for x in ("K", "V", "W")} for s in states]
    i32_range(4)
    alone = []
    for s in states:
        step(bkv, s, torch.cuda.current_stream())
        torch.cuda.synchronize()
        alone.append(results(s))
    for _ in range(3):
        for s, f in zip(states, first):
            for x, t in f.items():
                s[x].copy_(t)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in states]
        for s, cs in zip(states, streams):
            step(bkv, s, cs)
        torch.cuda.synchronize()
        for s, want in zip(states, alone):
            assert same(results(s), want)


FIRST = r"""
import torch
from kv_cache_eviction_head_gb300 import bkv
from tests import test_gpu_paged_serving as t
torch.zeros(1, device="cuda")
s, plain = t.step_state(bkv, 5), None
t.i32_range(4)
saved = {x: s[x].clone() for x in ("K", "V", "W")}
side = torch.cuda.Stream()
side.wait_stream(torch.cuda.current_stream())
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g, stream=side):
    t.step(bkv, s, side)
g.replay()
torch.cuda.synchronize()
got = t.results(s)
for x, v in saved.items():
    s[x].copy_(v)
t.step(bkv, s, torch.cuda.current_stream())
torch.cuda.synchronize()
assert t.same(got, t.results(s))
print("FIRST_OK")
"""


def test_prompt_layers_back_to_back(bkv):
    """Attention and weights of one layer after the other, nothing between them: each launch starts
    while the one before it drains, and both take TMEM. The results are those of calls that were
    waited for one by one."""
    heads, kv, lens = 8, 2, [700, 129]
    pool = Pool(2, kv, lens, None, 6)
    cfg, total, n = pool.config(bkv, heads), sum(lens), 12
    cu, zero = i32([0, lens[0], total]), i32([0, 0])
    K, V = ([pool.fresh(lens, 10 * l + s) for l in range(n)] for s in (1, 2))
    q = [randn((total, heads, D), 900 + l) for l in range(n)]
    out, lse = torch.empty_like(q[0]), [torch.empty((total, heads), device="cuda") for _ in range(n)]

    def run(wait):
        W = [torch.zeros(pool.shape(), device="cuda") for _ in range(n)]
        for l in range(n):
            bkv.bkv_attend_prompt(cfg, q[l], K[l], V[l], cu, zero, out, lse=lse[l], stream=stream())
            if wait:
                torch.cuda.synchronize()
            bkv.bkv_weigh_prompt(cfg, q[l], lse[l], K[l], cu, zero, W[l], decay=0.0, stream=stream())
            if wait:
                torch.cuda.synchronize()
        return torch.stack(W)

    want = run(True)
    for _ in range(10):
        assert torch.equal(run(False), want)


def test_first_calls_of_a_process_are_captured(bkv):
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "FIRST_OK" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]


def test_rows_do_not_depend_on_other_sequences_contents(bkv):
    """NaN, infinities and long tails elsewhere in the batch change no bit of a sequence's results."""
    a, b = step_state(bkv, 7), step_state(bkv, 7)
    pool = a["pool"]
    b["W"].copy_(a["W"])
    for x in ("K", "V", "W"):
        page, place = pool.at(3, 100)
        b[x][page, :, place] = math.nan
    for s in (a, b):
        bkv.bkv_attend_paged(s["cfg"], s["q"], s["K"], s["V"], s["lens"], s["out"], s["ws"], table=pool.table, weights=s["W"], stream=stream())
    assert torch.equal(a["out"][:3], b["out"][:3])
    for seq, n in ((0, 70), (1, 33)):
        assert torch.equal(pool.get(a["W"], seq, n), pool.get(b["W"], seq, n))


def test_beyond_32_bit_offsets(bkv):
    """A pool of 2^32 elements and more: sequences at its far end, in every call."""
    heads, kv, size = 8, 4, 256
    pages = (1 << 32) // (kv * size * D) + 40
    K = torch.empty((pages, kv, size, D), dtype=torch.bfloat16, device="cuda")
    V = torch.empty_like(K)
    W = torch.zeros((pages, kv, size), device="cuda")
    slots, lens = [1500, 700], [1400, 600]
    pool = Pool(2, kv, slots, size, 3)
    shift = pages - pool.pages
    pool.table[pool.table >= 0] += shift
    pool.where = ([w + shift for w in pool.where[0]], pool.where[1])
    pool.pages = pages
    for x, seed in ((K, 5), (V, 6)):
        x[shift:] = math.nan
        for b, n in enumerate(lens):
            pool.put(x, b, n, randn((kv, n, D), seed + 10 * b))
    cfg = pool.config(bkv, heads, budget=500, prefix=4, recent=8, max_cache=2048)
    kw = dict(table=pool.table, stream=stream())
    status = new_status()
    x = randn((2, heads + 2 * kv, D), 8)
    q = torch.empty((2, heads, D), dtype=torch.bfloat16, device="cuda")
    bkv.bkv_store_paged(cfg, bkv.make_rope(), x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:], i32([0, 1, 2]), i32(lens), i32([0, 0]), q, K, V,
                        status=status, **kw)
    assert int(status) == 0
    for b, n in enumerate(lens):
        assert torch.equal(pool.get(V, b, n + 1)[:, n], x[b, heads + kv:])
    lens = [n + 1 for n in lens]
    qp, cu = randn((20, heads, D), 9), i32([0, 10, 20])
    first = [n - 10 for n in lens]
    lse = torch.full((20, heads), 9.0, device="cuda")
    bkv.bkv_weigh_prompt(cfg, qp, lse, K, cu, i32(first), W, decay=0.0, status=status, **kw)
    assert int(status) == 0
    for b, n in enumerate(lens):
        k = pool.get(K, b, n)
        see = torch.arange(n, device="cuda")[None] <= first[b] + torch.arange(10, device="cuda")[:, None]
        want = torch.zeros((kv, n), dtype=torch.float64, device="cuda")
        for h in range(heads):
            l = qp[10 * b:10 * b + 10, h].double() @ k[h // 2].double().T / math.sqrt(D) - 9.0
            want[h // 2] += torch.exp(l.masked_fill(~see, -math.inf)).sum(dim=0)
        assert float(((pool.get(W, b, n).double() - want).abs() / want).max()) < 1e-5
    ws = torch.empty(bkv.bkv_attend_paged_bytes(cfg, K, pool.table, weighed=True), dtype=torch.uint8, device="cuda")
    out, old = torch.empty_like(q), W.clone()
    bkv.bkv_attend_paged(cfg, q, K, V, i32(lens), out, ws, weights=W, status=status, **kw)
    assert int(status) == 0
    for b, n in enumerate(lens):
        see = torch.ones((1, n), dtype=torch.bool, device="cuda")
        want, _, tol, _ = ref.attention(q[b:b + 1], pool.get(K, b, n), pool.get(V, b, n), see)
        assert ref.close(out[b:b + 1], want, tol) <= 0
        p, rel, _ = probabilities(q[b:b + 1], pool.get(K, b, n), see)
        s, stol = weight_sums(p, rel, kv)
        o = pool.get(old, b, n).double()
        o[:, n - 1] = 0
        assert ref.close(pool.get(W, b, n), o + s, stol + 2.0 ** -22 * (o + s)) <= 0
    rows = [[pool.get(t, b, n).clone() for b, n in enumerate(lens)] for t in (K, V, W)]
    kept = torch.empty((1, 2, kv, 500), dtype=torch.int32, device="cuda")
    bkv.bkv_evict_weight(cfg, [K], [V], [W], i32(lens), kept, status=status, **kw)
    assert int(status) == 0
    for b, n in enumerate(lens):
        for h in range(kv):
            i = torch.from_numpy(keep_set(rows[2][b][h].cpu().numpy(), 500, 4, 8)).cuda()
            assert torch.equal(kept[0, b, h].long(), i)
            for t, old in zip((K, V, W), rows):
                assert torch.equal(pool.get(t, b, 500)[h], old[b][h, i])


def test_far_slots(bkv):
    """2^17 slots of one sequence: aligned keys at the borders of shares and pages all count."""
    n, heads, kv = (1 << 17) - 3, 8, 1
    for page in (None, 256):
        pool = Pool(1, kv, [n], page, 4)
        cfg = pool.config(bkv, heads)
        g = torch.Generator(device="cuda").manual_seed(6)
        u = torch.randn(D, device="cuda", generator=g)
        u *= math.sqrt(D) / u.norm()
        k = torch.empty((kv, n, D), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
        v = torch.empty_like(k).normal_(generator=g)
        q = (u + 0.1 * torch.randn((1, heads, D), device="cuda", generator=g)).to(torch.bfloat16)
        at = [0, 15, 16, 255, 256, 4095, 4096, n // 2, n - 257, n - 17, n - 2, n - 1]
        k[:, at] = (25 * math.sqrt(D) / D * u + 0.02 * torch.randn((kv, len(at), D), device="cuda", generator=g)).to(torch.bfloat16)
        K, V = (torch.full(pool.shape() + (D,), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        pool.put(K, 0, n, k), pool.put(V, 0, n, v)
        W, out, lse, status = torch.zeros(pool.shape(), device="cuda"), torch.empty_like(q), torch.empty((1, heads), device="cuda"), new_status()
        ws = torch.empty(bkv.bkv_attend_paged_bytes(cfg, K, pool.table, weighed=True), dtype=torch.uint8, device="cuda")
        bkv.bkv_attend_paged(cfg, q, K, V, i32([n]), out, ws, table=pool.table, lse=lse, weights=W, status=status, stream=stream())
        assert int(status) == 0
        see = torch.ones((1, n), dtype=torch.bool, device="cuda")
        want, wlse, tol, ltol = ref.attention(q, k, v, see)
        assert ref.close(out, want, tol) <= 0 and ref.close(lse, wlse, ltol) <= 0
        p, rel, _ = probabilities(q, k, see)
        s, stol = weight_sums(p, rel, kv)
        assert ref.close(pool.get(W, 0, n), s, stol + 2.0 ** -22 * s) <= 0


CHECKED = r"""
import torch
from kv_cache_eviction_head_gb300 import bkv
assert bkv.library_path().endswith("libbkv_checked.so"), bkv.library_path()
from tests import test_gpu_paged as t, test_gpu_paged_serving as s
for heads, kv in ((8, 2), (24, 1)):
    for page in (None, 16, 48):
        assert t.attend_case(bkv, heads, kv, [33, 0, 1, 250, 129], page, 3) <= 0
        assert t.weigh_case(bkv, heads, kv, [33, 0, 129], [0, 5, 130], page, 4) <= 0
        assert t.store_case(bkv, heads, kv, [3, 0, 70], [0, 4, 30], page, 5, interleaved=page == 16, r=64) <= 0
for order_free in (False, True):
    t.evict_case(bkv, 4, 2, [300, 0, 90, 1, 160], 16, 6, budget=90, prefix=4, recent=16, order_free=order_free)
s.test_prompt_decode_and_eviction_together(bkv, 16)
print("CHECKED_OK")
"""


def test_checked_build(bkv):
    from kv_cache_eviction_head_gb300.build import build
    build(checked=True)
    r = subprocess.run([sys.executable, "-c", CHECKED], cwd=ROOT, env={**os.environ, "BKV_LIBRARY": "checked"}, capture_output=True, text=True,
                       timeout=900)
    assert r.returncode == 0 and "CHECKED_OK" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]
