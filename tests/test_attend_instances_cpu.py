"""Every compiled instance of the attention kernel is one that some call reaches: the launch
rule, swept over head shapes, batches, lengths and caches, against the names in the library."""

from __future__ import annotations

import itertools
import re
import shutil
import subprocess

import pytest

SMS = 152


def splits(items, ctas, max_cache):
    most = [7 * ctas, 32 if ctas == 2 else 15, 36 * ctas, 76 * ctas]
    for i in range(4):
        if items <= most[i] and 16 >> i <= (max_cache + 127) // 128:
            return 16 >> i
    return 1


def instance(tree, heads, kv, batch, tokens, max_cache):
    """(row tiles, trees, clusters) of a call; tokens: nodes per sequence, or a prompt call's total."""
    group = heads // kv
    per_tile = min(128 // group, tokens)
    if tree:
        tiles = 2 if per_tile < tokens else 1
        items = batch * kv * -(-tokens // (tiles * per_tile))
    else:
        blocks = lambda nq: (tokens // (nq * per_tile) + batch) * kv
        tiles = 2 if blocks(2) > SMS // 2 and per_tile < tokens else 1
        items = blocks(tiles)
    ctas = 2 if tiles == 1 and group * per_tile <= 32 else 1
    return tiles, tree, splits(items, ctas, max_cache) > 1


def test_no_instance_is_out_of_reach():
    from kv_cache_eviction_head_gb300 import build
    nm = shutil.which("nm")
    if not nm:
        pytest.skip("nm is not installed")
    names = subprocess.run([nm, "-C", build.build()], capture_output=True, text=True, check=True).stdout
    built = {(int(q), t == "true", c == "true") for q, t, c in re.findall(r"attend_kernel<(\d), (true|false), (true|false)>", names)}
    shapes = [(4, 1), (32, 8), (40, 8), (28, 4), (128, 1), (96, 1), (7, 7), (16, 16), (64, 32)]
    caches = [40, 300, 2064, 8192]
    reached = {instance(True, h, kv, b, n, m) for (h, kv), b, n, m in itertools.product(shapes, [1, 2, 7, 30, 64, 192], range(1, 65), caches)}
    reached |= {instance(False, h, kv, b, t, m) for (h, kv), b, t, m in
                itertools.product(shapes, [1, 2, 7, 30, 64, 192], [*range(1, 700, 3), 2000, 9001], caches)}
    assert built == reached
