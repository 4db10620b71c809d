"""Attention calls whose waits run out. In the bounds-checked build the bound of a wait can be
lowered to anything (bkv_checked_wait_cycles), so that some warp gives up while copies and
products of its block are under way: at once, in front of the first logits, in the middle of
the key loop, between two row blocks. The call must end, say so in its status, and leave the
GPU's tensor memory, shared memory and barriers to the next calls as if nothing had been."""

from __future__ import annotations

import os
import subprocess
import sys
import textwrap

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = textwrap.dedent('''
    import ctypes
    import torch
    from kv_cache_eviction_head_gb300 import bkv
    assert bkv.library_path().endswith("libbkv_checked.so"), bkv.library_path()
    lib = ctypes.CDLL(bkv.library_path())
    D, WHOLE = 128, 2_000_000_000

    def bound(cycles):
        torch.cuda.synchronize()
        assert lib.bkv_checked_wait_cycles(ctypes.c_uint32(cycles)) == 0

    def randn(shape, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        return torch.randn(shape, device="cuda", generator=g).to(torch.bfloat16)

    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    def make(kind, heads, kv, batch, n, past):
        """n tokens (nodes) of each sequence behind `past` slots."""
        cfg = bkv.make_config(heads=heads, kv_heads=kv, d=D, budget=1, period=16, prefix=0, recent=0, layers=1,
                              batch=batch, max_cache=past + n + 3, rope_theta=1e6)
        K, V = randn((batch, kv, past + n + 3, D), 1), randn((batch, kv, past + n + 3, D), 2)
        q, first = randn((batch, n, heads, D), 3), i32([past] * batch)
        cu = i32([n * b for b in range(batch + 1)])

        def call():
            out, lse = torch.zeros_like(q), torch.zeros((batch, n, heads), device="cuda")
            status = torch.zeros((1,), dtype=torch.int32, device="cuda")
            s = torch.cuda.current_stream()
            if kind == "tree":
                bkv.bkv_attend_tree(cfg, q, K, V, first, out, lse=lse, status=status, stream=s)
            else:
                bkv.bkv_attend_prompt(cfg, q.view(-1, heads, D), K, V, cu, first, out.view(-1, heads, D),
                                      lse=lse.view(-1, heads), status=status, stream=s)
            return out, lse, status
        return call

    cases = {
        "prompt, one tile, split": make("prompt", 32, 8, 1, 3, 3000),
        "prompt, one tile": make("prompt", 32, 8, 1, 300, 700),
        "prompt, two tiles": make("prompt", 32, 8, 12, 300, 500),
        "decode, split": make("tree", 32, 8, 1, 1, 2063),
        "tree, two tiles, split": make("tree", 28, 4, 2, 64, 2000),
        "tree, two tiles": make("tree", 28, 4, 24, 64, 1500),
        "decode": make("tree", 32, 8, 60, 1, 2063),
    }
    for name, call in cases.items():
        want = call()
        assert int(want[2]) == 0, name
        gave_up = []
        for cycles in (0, 100, 300, 600, 900, 1200, 1600, 2000, 3000, 5000, 10000, 20000, 50000):
            bound(cycles)
            short = [call() for _ in range(3)]  # one behind the other on the same SMs
            bound(WHOLE)
            for got in short:
                code = int(got[2])
                assert code in (0, bkv.BKV_ERR_TIMEOUT), (name, cycles, code)
                if code == 0:
                    assert all(torch.equal(a, b) for a, b in zip(got, want)), (name, cycles)
            gave_up.append(sum(int(got[2]) != 0 for got in short))
            got = call()
            assert all(torch.equal(a, b) for a, b in zip(got, want)), (name, cycles, int(got[2]))
        print(name, gave_up, flush=True)
        assert gave_up[0] == 3, name
    print("WAITS_OK")
''')


def test_waits_that_run_out_end_the_call_and_leave_nothing_behind():
    from kv_cache_eviction_head_gb300.build import build
    build(checked=True)
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env={**os.environ, "BKV_LIBRARY": "checked"},
                       capture_output=True, text=True, timeout=300)
    print(r.stdout)
    assert r.returncode == 0 and "WAITS_OK" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]
