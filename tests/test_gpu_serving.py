"""The model-side calls as a program uses them: together with the eviction
handle, in captured graphs, on several streams at once, on caches larger than
32-bit offsets reach, and in the bounds-checked build."""

from __future__ import annotations

import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from tests import attend_ref as ref

pytestmark = pytest.mark.gpu
D = 128
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def bkv():
    from kv_cache_eviction_head_gb300.build import build
    build()
    from kv_cache_eviction_head_gb300 import bkv as mod
    return mod


def randn(shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, device="cuda", generator=g) * scale).to(torch.bfloat16)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def check_rows(q, K, V, see, out):
    want, _, tol, _ = ref.attention(q, K, V, see)
    assert ref.close(out, want, tol) <= 0


def chain(n, past):
    return torch.arange(past + n, device="cuda")[None] <= past + torch.arange(n, device="cuda")[:, None]


def test_prompt_tree_commit_decode_and_eviction_together(bkv):
    """A prompt is stored, attended and used to start the query state; it is evicted down to
    the budget; a draft tree is attended and its accepted path kept; decode steps follow up
    to the next eviction. Every attention is checked against 64 bits on the caches as they
    then are, and the handle's own count of the cache agrees at the end."""
    layers, batch, heads, kv, P = 2, 2, 8, 2, 70
    cfg = bkv.make_config(heads=heads, kv_heads=kv, d=D, budget=64, period=16, prefix=4, recent=16, layers=layers,
                          batch=batch, max_cache=88, rope_theta=1e4)
    cs = torch.cuda.current_stream()
    h = bkv.bkv_create(cfg, torch.empty(bkv.bkv_workspace_bytes(cfg), dtype=torch.uint8, device="cuda"), cs)
    K = [torch.full((batch, kv, 88, D), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(layers)]
    V = [torch.full_like(K[0], math.nan) for _ in range(layers)]
    kept = torch.zeros((layers, batch, kv, 64), dtype=torch.int32, device="cuda")
    seed = iter(range(1000, 2000))

    def tokens(n):
        """A layer's projections of n packed tokens, as one fused output."""
        return randn((n, heads + 2 * kv, D), next(seed))

    def evict(step, length):
        before = [[t.clone() for t in ts] for ts in (K, V)]
        bkv.bkv_evict(h, K, V, length, step, kept)
        bkv.bkv_sync(h)
        for now, old in zip((K, V), before):
            for l in range(layers):
                at = kept[l].long()[..., None].expand(-1, -1, -1, D)
                assert torch.equal(now[l][:, :, :64], torch.gather(old[l], 2, at))

    try:
        q_prompt = torch.empty((P, layers, batch, heads, D), dtype=torch.bfloat16, device="cuda")
        cu, zero = i32([0, P, 2 * P]), i32([0, 0])
        for l in range(layers):
            x = tokens(batch * P)
            q = torch.empty((batch * P, heads, D), dtype=torch.bfloat16, device="cuda")
            out = torch.empty_like(q)
            bkv.bkv_store_kv(cfg, x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:], cu, zero, zero, q, K[l], V[l], stream=cs)
            bkv.bkv_attend_prompt(cfg, q, K[l], V[l], cu, zero, out, stream=cs)
            q_prompt[:, l] = x[:, :heads].view(batch, P, heads, D).transpose(0, 1)
            for b in range(batch):
                check_rows(q[b * P:(b + 1) * P], K[l][b, :, :P], V[l][b, :, :P], chain(P, 0), out[b * P:(b + 1) * P])
        bkv.bkv_prefill(h, q_prompt, 0)
        evict(P - 1, P)

        # a draft of five nodes: 0 - 1 - 3 and 0 - 2 - 4; the path 0, 2, 4 is accepted
        n, parent, path = 5, [-1, 0, 0, 1, 2], [0, 2, 4]
        bits, depth = [], []
        for i, p in enumerate(parent):
            bits.append((bits[p] if p >= 0 else 0) | 1 << i)
            depth.append(depth[p] + 1 if p >= 0 else 0)
        mask = torch.tensor([bits] * batch, dtype=torch.int64, device="cuda")
        lens, pos = i32([64, 64]), i32([P, P])
        drafted = torch.empty((n, layers, batch, heads, D), dtype=torch.bfloat16, device="cuda")
        see = torch.ones((n, 64 + n), dtype=torch.bool, device="cuda")
        for i in range(n):
            see[i, 64:] = torch.tensor([bool(bits[i] >> j & 1) for j in range(n)], device="cuda")
        for l in range(layers):
            x = tokens(batch * n)
            q = torch.empty((batch, n, heads, D), dtype=torch.bfloat16, device="cuda")
            out = torch.empty_like(q)
            bkv.bkv_store_kv(cfg, x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:], i32([0, n, 2 * n]), lens, pos,
                             q.view(batch * n, heads, D), K[l], V[l], depth=i32(depth * batch), stream=cs)
            bkv.bkv_attend_tree(cfg, q, K[l], V[l], lens, out, mask=mask, stream=cs)
            drafted[:, l] = x[:, :heads].view(batch, n, heads, D).transpose(0, 1)
            for b in range(batch):
                check_rows(q[b], K[l][b, :, :64 + n], V[l][b, :, :64 + n], see, out[b])
        tree = [t[:, :, 64:64 + n].clone() for t in K + V]
        bkv.bkv_commit_tree(cfg, K, V, lens, i32([path + [-1] * (n - 3)] * batch), i32([3, 3]), stream=cs)
        for t, old in zip(K + V, tree):
            assert torch.equal(t[:, :, 64:67], old[:, :, path])
        for k, node in enumerate(path):
            bkv.bkv_append_queries(h, drafted[node], P + k)

        # decode up to the next eviction
        length, step = 67, P + 3
        while length < 80:
            lens, pos, one = i32([length] * batch), i32([step] * batch), i32([0, 1, 2])
            q_step = torch.empty((layers, batch, heads, D), dtype=torch.bfloat16, device="cuda")
            for l in range(layers):
                x = tokens(batch)
                q = torch.empty((batch, 1, heads, D), dtype=torch.bfloat16, device="cuda")
                out = torch.empty_like(q)
                bkv.bkv_store_kv(cfg, x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:], one, lens, pos,
                                 q.view(batch, heads, D), K[l], V[l], stream=cs)
                bkv.bkv_attend_tree(cfg, q, K[l], V[l], lens, out, stream=cs)
                q_step[l] = x[:, :heads]
                for b in range(batch):
                    check_rows(q[b], K[l][b, :, :length + 1], V[l][b, :, :length + 1], chain(1, length), out[b])
            bkv.bkv_append_queries(h, q_step, step)
            length, step = length + 1, step + 1
        assert bkv.bkv_get_stats(h).cache_len == length
        evict(step - 1, length)
        assert bkv.bkv_get_stats(h).cache_len == 64
    finally:
        bkv.bkv_destroy(h)


def serving_state(bkv, seed, batch=3, heads=8, kv=2, slots=700, n=4):
    cfg = bkv.make_config(heads=heads, kv_heads=kv, d=D, budget=1, period=16, prefix=0, recent=0, layers=1, batch=batch,
                          max_cache=slots, rope_theta=1e6)
    s = dict(cfg=cfg, K=randn((batch, kv, slots, D), seed), V=randn((batch, kv, slots, D), seed + 1),
             x=randn((batch * n, heads + 2 * kv, D), seed + 2), cu=i32([i * n for i in range(batch + 1)]),
             lens=i32([5 + 100 * b for b in range(batch)]), path=i32([[0, 2, 3, 3]] * batch), count=i32([3] * batch),
             q=torch.zeros((batch, n, heads, D), dtype=torch.bfloat16, device="cuda"), n=n, heads=heads, kv=kv)
    s["out"], s["prompt"] = torch.zeros_like(s["q"]), torch.zeros((batch * n, heads, D), dtype=torch.bfloat16, device="cuda")
    s["status"] = torch.zeros((1,), dtype=torch.int32, device="cuda")
    return s


def serve(bkv, s, stream):
    h, kv = s["heads"], s["kv"]
    flat = s["q"].view(-1, h, D)
    bkv.bkv_store_kv(s["cfg"], s["x"][:, :h], s["x"][:, h:h + kv], s["x"][:, h + kv:], s["cu"], s["lens"], s["lens"], flat,
                     s["K"], s["V"], status=s["status"], stream=stream)
    bkv.bkv_attend_tree(s["cfg"], s["q"], s["K"], s["V"], s["lens"], s["out"], status=s["status"], stream=stream)
    bkv.bkv_attend_prompt(s["cfg"], flat, s["K"], s["V"], s["cu"], s["lens"], s["prompt"], stream=stream)
    bkv.bkv_commit_tree(s["cfg"], [s["K"]], [s["V"]], s["lens"], s["path"], s["count"], stream=stream)


def results(s):
    return [s[k] for k in ("q", "out", "prompt", "K", "V")]


def test_captured_calls_read_their_lengths_at_replay(bkv):
    a, b = serving_state(bkv, 10), serving_state(bkv, 10)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        serve(bkv, serving_state(bkv, 10), stream)
        torch.cuda.synchronize()
        graph.capture_begin()
        serve(bkv, a, stream)
        graph.capture_end()
    for lens in ([5, 105, 205], [600, 0, 333]):
        for s in (a, b):
            s["lens"].copy_(i32(lens))
            s["x"].copy_(randn(s["x"].shape, 77))
        graph.replay()
        serve(bkv, b, torch.cuda.current_stream())
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(results(a), results(b)))
        # mask NULL is a chain: the tree and the prompt see the same slots
        assert float((a["out"].view(-1, 8, D).float() - a["prompt"].float()).abs().max()) < 0.05


def test_calls_on_several_streams_at_once(bkv):
    """No workspace is shared: eight streams' calls, interleaved, give what each gives alone."""
    states = [serving_state(bkv, 100 + 10 * i, slots=700 + 600 * i) for i in range(8)]
    alone = [serving_state(bkv, 100 + 10 * i, slots=700 + 600 * i) for i in range(8)]
    for s in alone:
        for _ in range(5):
            serve(bkv, s, torch.cuda.current_stream())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    for _ in range(5):
        for s, stream in zip(states, streams):
            serve(bkv, s, stream)
    torch.cuda.synchronize()
    for s, t in zip(states, alone):
        assert int(s["status"]) == 0
        assert all(torch.equal(x, y) for x, y in zip(results(s), results(t)))


def test_caches_beyond_32_bit_offsets(bkv):
    """The last of 16 heads of 2^21 slots starts behind element 2^31."""
    kv, slots, n = 16, 1 << 21, 3
    cfg = bkv.make_config(heads=kv, kv_heads=kv, d=D, budget=1, period=16, prefix=0, recent=0, layers=1, batch=1,
                          max_cache=slots, rope_theta=1e6)
    K = torch.empty((1, kv, slots, D), dtype=torch.bfloat16, device="cuda")
    V = torch.empty_like(K)
    cs = torch.cuda.current_stream()
    for length in (150, slots - n):
        K[:, :, max(0, length - 150):length] = randn((1, kv, 150, D), 1)
        V[:, :, max(0, length - 150):length] = randn((1, kv, 150, D), 2)
        x = randn((n, 3 * kv, D), 3)
        q = torch.empty((1, n, kv, D), dtype=torch.bfloat16, device="cuda")
        lens = i32([length])
        bkv.bkv_store_kv(cfg, x[:, :kv], x[:, kv:2 * kv], x[:, 2 * kv:], i32([0, n]), lens, lens, q[0], K, V, stream=cs)
        want = ref.rope(x[:, kv:2 * kv], length + torch.arange(n, device="cuda"), 1e6)
        assert float((K[0, :, length:length + n].transpose(0, 1).double() - want).abs().max()) < 0.05
        assert torch.equal(V[0, :, length:length + n].transpose(0, 1), x[:, 2 * kv:])
        if length == 150:
            out = torch.empty_like(q)
            bkv.bkv_attend_tree(cfg, q, K, V, lens, out, stream=cs)
            check_rows(q[0], K[0, :, :153], V[0, :, :153], chain(n, 150), out[0])
            bkv.bkv_attend_prompt(cfg, q[0], K, V, i32([0, n]), lens, out[0], stream=cs)
            check_rows(q[0], K[0, :, :153], V[0, :, :153], chain(n, 150), out[0])
        rows = K[0, :, length:length + n].clone()
        bkv.bkv_commit_tree(cfg, [K], [V], lens, i32([[2, 1, 0]]), i32([3]), stream=cs)
        assert torch.equal(K[0, :, length:length + n], rows.flip(1))


def test_many_short_sequences(bkv):
    """More sequences than the block search looks at in one step, most of one token, some empty."""
    batch, heads, kv, slots = 300, 4, 1, 40
    lens = [(b * 7) % 5 for b in range(batch)]
    lens[271] = 33
    first = [(b * 3) % 6 for b in range(batch)]
    cfg = bkv.make_config(heads=heads, kv_heads=kv, d=D, budget=1, period=16, prefix=0, recent=0, layers=1, batch=batch,
                          max_cache=slots, rope_theta=1e6)
    total = sum(lens)
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    K, V = randn((batch, kv, slots, D), 1), randn((batch, kv, slots, D), 2)
    x = randn((total, heads + 2 * kv, D), 3)
    q = torch.empty((total, heads, D), dtype=torch.bfloat16, device="cuda")
    out, cs = torch.empty_like(q), torch.cuda.current_stream()
    bkv.bkv_store_kv(cfg, x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:], i32(cu), i32(first), i32(first), q, K, V, stream=cs)
    bkv.bkv_attend_prompt(cfg, q, K, V, i32(cu), i32(first), out, stream=cs)
    for b in range(batch):
        f, n = first[b], lens[b]
        if n:
            assert torch.equal(V[b, :, f:f + n].transpose(0, 1), x[cu[b]:cu[b + 1], heads + kv:])
            check_rows(q[cu[b]:cu[b + 1]], K[b, :, :f + n], V[b, :, :f + n], chain(n, f), out[cu[b]:cu[b + 1]])


def test_store_of_a_long_prompt(bkv):
    """The two-token form of the kernel, an odd number of tokens, against the one-token form."""
    heads, kv, n = 6, 2, 1301
    cfg = bkv.make_config(heads=heads, kv_heads=kv, d=D, budget=1, period=16, prefix=0, recent=0, layers=1, batch=1,
                          max_cache=n, rope_theta=1e4)
    x, cs = randn((n, heads + 2 * kv, D), 1), torch.cuda.current_stream()

    def store(lo, hi, q, K, V):
        y = x[lo:hi]
        bkv.bkv_store_kv(cfg, y[:, :heads], y[:, heads:heads + kv], y[:, heads + kv:], i32([0, hi - lo]), i32([lo]),
                         i32([lo + 50000]), q[lo:hi], K, V, stream=cs)
    got, want = [], []
    for parts, to in (([(0, n)], got), ([(0, 700), (700, n)], want)):
        q = torch.empty((n, heads, D), dtype=torch.bfloat16, device="cuda")
        K, V = torch.zeros((1, kv, n, D), dtype=torch.bfloat16, device="cuda"), torch.zeros((1, kv, n, D), dtype=torch.bfloat16, device="cuda")
        for lo, hi in parts:
            store(lo, hi, q, K, V)
        to += [q, K, V]
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_checked_build(bkv):
    """The bounds-checked library runs a selection of the cases with no latched status."""
    from kv_cache_eviction_head_gb300.build import build
    build(checked=True)
    cases = ["test_gpu_attend.py::" + c for c in (
        "test_prompt_lengths_and_groups[7-1]", "test_prompt_two_tiles_per_block[40-8]", "test_tree_masks[14-2-33]",
        "test_decode[lens0-10-2]", "test_tree_key_splits[1-8-8192]", "test_store[True-10000.0-positions1]", "test_commit[5]")]
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-m", "gpu"] + ["tests/" + c for c in cases], cwd=ROOT,
                       env={**os.environ, "BKV_LIBRARY": "checked"}, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and f"{len(cases)} passed" in r.stdout, r.stdout[-3000:] + r.stderr[-2000:]


def test_two_captured_graphs_replayed_at_once(bkv):
    """Two-tile kernels behind one another in two graphs, replayed on two streams at a time,
    give what the same calls give eagerly."""
    shape = dict(batch=20, heads=28, kv=4, slots=900, n=40)

    def state(seed):
        s = serving_state(bkv, seed, **shape)
        s["lens"].copy_(i32([40 * b for b in range(20)]))
        s["path"] = i32([list(range(3, 40)) + [0, 1, 2]] * 20)
        s["count"] = i32([b + 1 for b in range(20)])
        return s

    states, eager = [state(20), state(30)], [state(20), state(30)]
    streams, graphs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for s, stream in zip(states, streams):
        stream.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(stream):
            serve(bkv, state(1), stream)
            torch.cuda.synchronize()
            graph.capture_begin()
            serve(bkv, s, stream)
            serve(bkv, s, stream)
            graph.capture_end()
        graphs.append(graph)
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    for s in eager:
        for _ in range(6):
            serve(bkv, s, torch.cuda.current_stream())
    torch.cuda.synchronize()
    for s, t in zip(states, eager):
        assert int(s["status"]) == 0
        assert all(torch.equal(x, y) for x, y in zip(results(s), results(t)))


def test_calls_from_several_threads_at_once(bkv):
    """Four host threads, each with a stream and a state of its own."""
    import threading

    states, alone = ([serving_state(bkv, 200 + 10 * i, n=4 + 12 * i) for i in range(4)] for _ in range(2))
    for s in states + alone:
        s["path"] = i32([list(range(s["n"]))[::-1]] * 3)
    for s in alone:
        for _ in range(20):
            serve(bkv, s, torch.cuda.current_stream())
    torch.cuda.synchronize()
    errors = []

    def work(s, stream):
        try:
            for _ in range(20):
                serve(bkv, s, stream)
        except Exception as e:  # shown by the assertion below
            errors.append(e)

    threads = [threading.Thread(target=work, args=(s, torch.cuda.Stream())) for s in states]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for s, t in zip(states, alone):
        assert int(s["status"]) == 0
        assert all(torch.equal(x, y) for x, y in zip(results(s), results(t)))
