"""Host-only checks of the calls over paged caches: refusals before anything is
enqueued (fake, aligned device addresses are enough: nothing is dereferenced),
frequencies, workspace sizes. Nothing here touches a GPU."""

from __future__ import annotations

import ctypes
import math

import pytest
import torch

A = 1 << 20  # an aligned address that no call reaches


@pytest.fixture(scope="module")
def bkv():
    from kv_cache_eviction_head_gb300.build import build
    build()
    from kv_cache_eviction_head_gb300 import bkv as mod
    return mod


def cfg_for(bkv, **over):
    base = dict(heads=8, kv_heads=2, d=128, budget=16, period=16, prefix=0, recent=0, layers=2, batch=3, max_cache=64,
                rope_theta=1e6)
    base.update(over)
    return bkv.make_config(**base)


def layers(*ptrs):
    return (ctypes.c_void_p * len(ptrs))(*ptrs)


p, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
KINDS = {
    "bkv_store_paged": [p, i64, p, i64, p, i64, i32] + [p] * 9,
    "bkv_attend_paged": [p, i64, p, p, p, p, p, p, f32, p, sz, p, p],
    "bkv_weigh_prompt": [p, i64, p, p, p, p, i32, p, f32, p, p],
    "bkv_evict_weight": [p] * 8,
}
GOOD = {
    "bkv_store_paged": dict(q=A, qs=1024, k=A, ks=256, v=A, vs=256, total=5, cu=A, first=A, pos=A, depth=0, q_rot=A, K=A, V=A,
                            status=0, stream=0),
    "bkv_attend_paged": dict(q=A, qs=1024, K=A, V=A, lens=A, out=A, lse=0, weights=A, decay=1.0, ws=A, size=1 << 40, status=0, stream=0),
    "bkv_weigh_prompt": dict(q=A, qs=1024, lse=A, K=A, cu=A, first=A, total=5, weights=A, decay=1.0, status=0, stream=0),
    "bkv_evict_weight": dict(K=layers(A, A), V=layers(A, A), W=layers(A, A), lens=A, kept=A, new=0, status=0, stream=0),
}
BAD = {
    "bkv_store_paged": [dict(q=0), dict(q=A + 8), dict(qs=1016), dict(qs=1028), dict(k=0), dict(ks=128), dict(v=A + 2), dict(vs=260),
                        dict(total=-1), dict(cu=0), dict(cu=A + 2), dict(first=0), dict(pos=0), dict(depth=A + 2), dict(q_rot=0),
                        dict(q_rot=A + 8), dict(K=0), dict(V=A + 4), dict(status=A + 2)],
    "bkv_attend_paged": [dict(q=0), dict(q=A + 8), dict(qs=512), dict(qs=1025), dict(K=0), dict(V=A + 8), dict(lens=0), dict(lens=A + 1),
                         dict(out=0), dict(out=A + 4), dict(lse=A + 2), dict(weights=A + 2), dict(decay=-0.1), dict(decay=1.5),
                         dict(decay=math.nan), dict(status=A + 1)],
    "bkv_weigh_prompt": [dict(q=0), dict(qs=1025), dict(lse=0), dict(lse=A + 2), dict(K=0), dict(cu=0), dict(first=A + 2), dict(total=-1),
                         dict(weights=0), dict(weights=A + 1), dict(decay=2.0), dict(decay=math.nan), dict(status=A + 2)],
    "bkv_evict_weight": [dict(K=layers(A, 0)), dict(V=layers(A + 8, A)), dict(W=layers(A, A + 2)), dict(W=layers(0, A)), dict(lens=0),
                         dict(lens=A + 2), dict(kept=0), dict(kept=A + 1), dict(new=A), dict(new=A + 2), dict(status=A + 2)],
}


def call(bkv, name, cfg, args, pages=None, rope="good"):
    good = bkv.make_rope()
    head = [ctypes.byref(cfg) if cfg is not None else None, ctypes.byref(pages) if pages is not None else None]
    if name == "bkv_store_paged":
        head.append(ctypes.byref(good if rope == "good" else rope) if rope is not None else None)
    args = list(args)
    assert len(KINDS[name]) == len(args)
    return bkv.raw_status(name, *head, *[k(a) if not isinstance(a, ctypes.Array) else a for k, a in zip(KINDS[name], args)])


@pytest.mark.parametrize("name,over", [(n, o) for n, os in BAD.items() for o in os],
                         ids=lambda v: v if isinstance(v, str) else ",".join(f"{k}={x}" for k, x in v.items() if not isinstance(x, ctypes.Array)))
def test_invalid_arguments(bkv, name, over):
    assert call(bkv, name, cfg_for(bkv), {**GOOD[name], **over}.values()) == bkv.BKV_ERR_INVALID_ARG


@pytest.mark.parametrize("name", GOOD)
def test_configs(bkv, name):
    args = GOOD[name].values()
    assert call(bkv, name, None, args) == bkv.BKV_ERR_INVALID_ARG
    assert call(bkv, name, cfg_for(bkv, heads=9), args) == bkv.BKV_ERR_INVALID_ARG
    assert call(bkv, name, cfg_for(bkv, d=64), args) == bkv.BKV_ERR_UNSUPPORTED
    assert call(bkv, name, cfg_for(bkv, heads=258, kv_heads=2), args) == bkv.BKV_ERR_UNSUPPORTED


@pytest.mark.parametrize("name", GOOD)
@pytest.mark.parametrize("pages,code", [((0, 16, 4, A), 1), ((9, 0, 4, A), 1), ((9, 16, 0, A), 1), ((9, 16, 4, 0), 1), ((9, 16, 4, A + 2), 1),
                                        ((9, 8, 4, A), 7), ((9, 24, 4, A), 7), ((9, 1 << 20, 1 << 11, A), 7), ((9, 16, 1 << 28, A), 7)])
def test_pages(bkv, name, pages, code):
    assert call(bkv, name, cfg_for(bkv), GOOD[name].values(), bkv.BkvPages(*pages)) == code


def test_attend_workspace(bkv):
    args = GOOD["bkv_attend_paged"]
    c = cfg_for(bkv)
    n = sz(0)
    for weights in (0, A):
        assert bkv.raw_status("bkv_attend_paged_bytes", ctypes.byref(c), None, 1 if weights else 0, ctypes.byref(n)) == 0
        for bad in (dict(size=n.value - 1), dict(ws=0), dict(ws=A + 128)):
            assert call(bkv, "bkv_attend_paged", c, {**args, "weights": weights, "size": n.value, **bad}.values()) == bkv.BKV_ERR_WORKSPACE
    assert bkv.raw_status("bkv_attend_paged_bytes", ctypes.byref(c), None, 1, None) == bkv.BKV_ERR_INVALID_ARG
    # the logits of every slot that the pool has, and not of every slot that the tables could name
    size = lambda pages, weighed: (bkv.raw_status("bkv_attend_paged_bytes", ctypes.byref(c), ctypes.byref(pages), weighed, ctypes.byref(n)), n.value)[1]
    small, large = bkv.BkvPages(10, 16, 1 << 20, A), bkv.BkvPages(20, 16, 1 << 20, A)
    assert size(small, 0) == size(large, 0)
    assert size(large, 1) - size(small, 1) == 10 * 16 * 8 * 4


def test_unsupported(bkv):
    assert call(bkv, "bkv_weigh_prompt", cfg_for(bkv, heads=97, kv_heads=1), {**GOOD["bkv_weigh_prompt"], "qs": 97 * 128}.values()) == 7
    big = cfg_for(bkv, budget=(1 << 19) + 1, max_cache=1 << 20, flags=2)
    assert call(bkv, "bkv_evict_weight", big, GOOD["bkv_evict_weight"].values()) == 7
    far = cfg_for(bkv, budget=2 ** 31 - 4096, max_cache=2 ** 31 - 1)
    assert call(bkv, "bkv_evict_weight", far, GOOD["bkv_evict_weight"].values(), pages=bkv.BkvPages(10, 16, 4, A)) == 7


def test_ropes(bkv):
    from tests.test_gpu_paged import frequencies
    for r in (0, 16, 96, 128):
        for scaling, factor in (("none", 1.0), ("linear", 4.0), ("ntk", 3.0), ("yarn", 5.5)):
            rope = bkv.make_rope(theta=5e5, rotary_dim=r, interleaved=True, scaling=scaling, factor=factor, original_len=4096)
            want, scale = frequencies(5e5, r, scaling, factor, 4096)
            assert rope.rotary_dim == r and rope.interleaved == 1
            assert list(rope.inv_freq[:r // 2]) == pytest.approx(want, rel=1e-14) and not any(rope.inv_freq[r // 2:])
            if r:
                assert rope.scale == pytest.approx(scale, rel=1e-15)
    for over, code in ((dict(theta=0.0), 1), (dict(theta=math.inf), 1), (dict(rotary_dim=-16), 1), (dict(rotary_dim=144), 7), (dict(rotary_dim=24), 7),
                       (dict(scaling="linear", factor=0.5), 1), (dict(scaling="ntk", factor=math.nan), 1), (dict(scaling="yarn", factor=2.0), 1)):
        with pytest.raises(bkv.BkvError) as e:
            bkv.make_rope(**over)
        assert e.value.code == code
    for over in (dict(scaling="linear2"), dict(inv_freq=[1.0]), dict(inv_freq=[1.0] * 64, scaling="yarn", factor=2.0)):
        with pytest.raises(ValueError):
            bkv.make_rope(**over)
    bad = bkv.make_rope()
    bad.inv_freq[3] = math.nan
    args = GOOD["bkv_store_paged"].values()
    assert call(bkv, "bkv_store_paged", cfg_for(bkv), args, rope=bad) == bkv.BKV_ERR_INVALID_ARG
    assert call(bkv, "bkv_store_paged", cfg_for(bkv), args, rope=None) == bkv.BKV_ERR_INVALID_ARG
    for field, value, code in (("rotary_dim", 24, 7), ("rotary_dim", -16, 1), ("rotary_dim", 144, 7), ("interleaved", 2, 1), ("scale", math.inf, 1)):
        bad = bkv.make_rope()
        setattr(bad, field, value)
        assert call(bkv, "bkv_store_paged", cfg_for(bkv), args, rope=bad) == code


def test_the_binding_refuses_what_does_not_match(bkv, monkeypatch):
    """CPU tensors, wrong types and shapes raise ValueError before the library is called."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    c = cfg_for(bkv)
    t = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)
    K, b, ws = t(3, 2, 64, 128), t(3, dtype=torch.int32), t(100, dtype=torch.uint8)
    table = t(3, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="table:"):
        bkv.bkv_attend_paged_bytes(c, K, b)
    with pytest.raises(ValueError, match="table:"):
        bkv.bkv_attend_paged_bytes(c, K, table)
    with pytest.raises(ValueError, match="K:"):
        bkv.bkv_attend_paged_bytes(c, b, table)
    with pytest.raises(ValueError, match="q:"):
        bkv.bkv_attend_paged(c, t(3, 8, 128), K, K, b, t(3, 8, 128), ws)
    with pytest.raises(ValueError, match="q:"):
        bkv.bkv_weigh_prompt(c, t(8, 128), None, K, b, b, None)
    with pytest.raises(ValueError, match="q_pre:"):
        bkv.bkv_store_paged(c, bkv.make_rope(), None, None, None, b, b, b, None, K, K)
    with pytest.raises(ValueError, match="K:"):
        bkv.bkv_evict_weight(c, [K], [K, K], [K, K], b, b)
    with pytest.raises(ValueError, match="K"):
        bkv.bkv_evict_weight(c, [K, K], [K, K], [K, K], b, b)
