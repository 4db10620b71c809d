"""The first calls that a process makes, captured into a graph: no warm-up has loaded a kernel,
set an attribute or looked up the tensor-map encoder before."""

from __future__ import annotations

import os
import subprocess
import sys
import textwrap

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = textwrap.dedent('''
    import torch
    from kv_cache_eviction_head_gb300 import bkv
    from tests.test_gpu_serving import results, serve, serving_state
    a, b = serving_state(bkv, 10), serving_state(bkv, 10)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        graph.capture_begin()
        serve(bkv, a, stream)
        graph.capture_end()
        graph.replay()
        serve(bkv, b, stream)
    torch.cuda.synchronize()
    assert int(a["status"]) == 0 and int(b["status"]) == 0
    assert all(torch.equal(x, y) for x, y in zip(results(a), results(b)))
    assert bool(b["out"].any()) and bool(b["prompt"].any())
    print("CAPTURED_OK")
''')


def test_a_process_s_first_calls_can_be_captured():
    from kv_cache_eviction_head_gb300.build import build
    build()
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env={**os.environ}, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "CAPTURED_OK" in r.stdout, r.stdout[-2000:] + r.stderr[-3000:]
