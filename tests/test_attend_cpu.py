"""Host-only checks of the model-side calls over the caches: every argument
error comes back before anything is enqueued (fake, aligned device addresses
are enough: nothing is dereferenced), and the binding refuses tensors that do
not match the config. Nothing here touches a GPU."""

from __future__ import annotations

import ctypes

import pytest
import torch

A = 1 << 20  # a 16-byte aligned address that no call reaches


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


def call(bkv, name, cfg, args):
    p = ctypes.c_void_p
    ptr = lambda v: p(v) if not isinstance(v, ctypes.Array) else v
    i64, i32 = ctypes.c_int64, ctypes.c_int32
    kinds = {
        "bkv_store_kv": [ptr, i64, ptr, i64, ptr, i64, i32] + [ptr] * 9,
        "bkv_attend_prompt": [ptr, i64, ptr, ptr, ptr, ptr, i32] + [ptr] * 4,
        "bkv_attend_tree": [ptr, i64, ptr, ptr, ptr, i32] + [ptr] * 6,
        "bkv_commit_tree": [ptr, ptr, ptr, ptr, ptr, i32, ptr, ptr],
    }[name]
    assert len(kinds) == len(args)
    return bkv.raw_status(name, ctypes.byref(cfg) if cfg is not None else None, *[k(a) for k, a in zip(kinds, args)])


def layers(*ptrs):
    return (ctypes.c_void_p * len(ptrs))(*ptrs)


GOOD = {
    "bkv_store_kv": dict(q=A, qs=1024, k=A, ks=256, v=A, vs=256, total=5, cu=A, first=A, pos=A, depth=0, q_rot=A, K=A, V=A,
                         status=0, stream=0),
    "bkv_attend_prompt": dict(q=A, qs=1024, K=A, V=A, cu=A, first=A, total=5, out=A, lse=0, status=0, stream=0),
    "bkv_attend_tree": dict(q=A, qs=1024, K=A, V=A, lens=A, n=4, mask=0, nodes=0, out=A, lse=0, status=0, stream=0),
    "bkv_commit_tree": dict(K=layers(A, A), V=layers(A, A), lens=A, path=A, count=A, n=4, status=0, stream=0),
}
BAD = {
    "bkv_store_kv": [dict(q=0), dict(q=A + 8), dict(qs=1016), dict(qs=1028), dict(k=0), dict(ks=128), dict(v=A + 2),
                     dict(vs=260), dict(vs=-256), dict(total=-1), dict(cu=0), dict(cu=A + 2), dict(first=0), dict(pos=0),
                     dict(pos=A + 1), dict(depth=A + 2), dict(q_rot=0), dict(q_rot=A + 8), dict(K=0), dict(V=0),
                     dict(V=A + 4), dict(status=A + 2)],
    "bkv_attend_prompt": [dict(q=0), dict(q=A + 8), dict(qs=512), dict(qs=1025), dict(K=0), dict(K=A + 8), dict(V=0),
                          dict(cu=0), dict(cu=A + 1), dict(first=0), dict(total=-3), dict(out=0), dict(out=A + 4),
                          dict(lse=A + 2), dict(status=A + 1)],
    "bkv_attend_tree": [dict(q=0), dict(q=A + 2), dict(qs=1020), dict(qs=0), dict(K=0), dict(V=A + 2), dict(lens=0),
                        dict(lens=A + 2), dict(n=0), dict(n=-1), dict(mask=A + 4), dict(nodes=A + 1), dict(out=0),
                        dict(lse=A + 1), dict(status=A + 3)],
    "bkv_commit_tree": [dict(K=layers(A, 0)), dict(V=layers(A + 8, A)), dict(lens=0), dict(path=0), dict(path=A + 2),
                        dict(count=0), dict(n=0), dict(status=A + 2)],
}


@pytest.mark.parametrize("name,over", [(n, o) for n, os in BAD.items() for o in os],
                         ids=lambda v: v if isinstance(v, str) else ",".join(v))
def test_invalid_arguments(bkv, name, over):
    assert call(bkv, name, cfg_for(bkv), {**GOOD[name], **over}.values()) == bkv.BKV_ERR_INVALID_ARG


@pytest.mark.parametrize("name", GOOD)
def test_configs(bkv, name):
    args = GOOD[name].values()
    assert call(bkv, name, None, args) == bkv.BKV_ERR_INVALID_ARG
    assert call(bkv, name, cfg_for(bkv, heads=9), args) == bkv.BKV_ERR_INVALID_ARG
    assert call(bkv, name, cfg_for(bkv, max_cache=16), args) == bkv.BKV_ERR_INVALID_ARG
    assert call(bkv, name, cfg_for(bkv, d=64), args) == bkv.BKV_ERR_UNSUPPORTED
    assert call(bkv, name, cfg_for(bkv, heads=258, kv_heads=2), args) == bkv.BKV_ERR_UNSUPPORTED


@pytest.mark.parametrize("name", ["bkv_attend_tree", "bkv_commit_tree"])
def test_more_nodes_than_mask_bits(bkv, name):
    assert call(bkv, name, cfg_for(bkv), {**GOOD[name], "n": 65}.values()) == bkv.BKV_ERR_UNSUPPORTED


def test_the_binding_refuses_what_does_not_match(bkv, monkeypatch):
    """CPU tensors, wrong types, shapes and strides raise ValueError before the library is called."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    c = cfg_for(bkv)
    t = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)
    K = t(3, 2, 64, 128)
    cu, b = t(4, dtype=torch.int32), t(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="q:"):
        bkv.bkv_attend_prompt(c, t(5, 8, 128), K, K, cu, b, t(5, 8, 128))
    with pytest.raises(ValueError, match="q:"):
        bkv.bkv_attend_prompt(c, t(8, 128), K, K, cu, b, t(5, 8, 128))
    with pytest.raises(ValueError, match="q:"):
        bkv.bkv_attend_tree(c, t(3, 8, 128), K, K, b, t(3, 1, 8, 128))
    with pytest.raises(ValueError, match="q_pre:"):
        bkv.bkv_store_kv(c, None, None, None, cu, b, b, None, K, K)
    with pytest.raises(ValueError, match="path:"):
        bkv.bkv_commit_tree(c, [K, K], [K, K], b, b, b)
    with pytest.raises(ValueError, match="K:"):
        bkv.bkv_commit_tree(c, [K], [K, K], b, t(3, 4, dtype=torch.int32), b)


class FakeCuda(torch.Tensor):
    """A CPU tensor that says it is on a device, for the binding's checks."""
    is_cuda = True

    def get_device(self):
        return self.at


def test_packed_strides_and_devices(bkv):
    def fake(x, at=0):
        f = x.as_subclass(FakeCuda)
        f.at = at
        return f
    bkv._load()
    wide = torch.zeros((5, 12, 128), dtype=torch.bfloat16)
    assert bkv._check_packed(fake(wide[:, :8]), "q", (5, 8, 128), 0)[1] == 12 * 128
    assert bkv._check_packed(fake(wide[:1, :8]), "q", (1, 8, 128), 0)[1] == 8 * 128  # one token: any spacing
    tree = torch.zeros((3, 4, 12, 128), dtype=torch.bfloat16)
    assert bkv._check_packed(fake(tree[:, :, 4:]), "q", (3, 4, 8, 128), 0)[1] == 12 * 128
    assert bkv._check_packed(fake(tree[:, :1, :8]), "q", (3, 1, 8, 128), 0)[1] == 4 * 12 * 128
    for bad, shape in ((wide.transpose(0, 1)[:8], (8, 5, 128)), (wide[:, ::2], (5, 6, 128)), (wide[..., ::2], (5, 12, 64)),
                       (tree[:, :3], (3, 3, 12, 128)), (wide.float(), (5, 12, 128)), (wide, (4, 12, 128))):
        with pytest.raises(ValueError, match="q:"):
            bkv._check_packed(fake(bad), "q", shape, 0)
    with pytest.raises(ValueError, match="current device"):
        bkv._check_packed(fake(wide, at=1), "q", (5, 12, 128), 0)
    with pytest.raises(ValueError, match="current device"):
        bkv._check_on_device(fake(wide, at=1), "q", torch.bfloat16, (5, 12, 128), 0)
