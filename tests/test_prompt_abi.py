"""Prompt attention, its column sums and tree verification without a GPU: what is refused, before
anything is enqueued (host tensors; no kernel is launched)."""

import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def T():
    from tiered_mixed_precision_gb300 import build

    build.build()
    import tiered_mixed_precision_gb300 as T

    return T


class _S:  # a stream handle that is never used (no launch happens)
    cuda_stream = 0


def _cfg(T, **kw):
    return T.Config(**{**dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=64, mid_capacity=8), **kw})


def _z(*s, dt=torch.float16):
    return torch.zeros(s, dtype=dt)


def _prompt(T, status, sums=False, **kw):
    c = kw.pop("cfg", None) or _cfg(T)
    n_q, n_kv = kw.pop("n_q", 5), kw.pop("n_kv", 9)
    a = dict(q=_z(2, n_q, 8, 64), k=_z(2, n_kv, 2, 64), v=_z(2, n_kv, 2, 64), out=_z(2, n_q, 8, 64),
             lse=_z(2, n_q, 8, dt=torch.float32), mass=_z(2, 2, n_kv, dt=torch.float32),
             ws=_z(1 << 24, dt=torch.uint8))
    a.update({x: kw.pop(x) for x in list(kw) if x in a})
    with pytest.raises((T.FadeError, ValueError)) as e:
        if sums:
            T.fade_prompt_mass(c, a["q"], a["k"], a["lse"], a["mass"], ws=a["ws"], stream=_S(), **kw)
        else:
            T.fade_prompt_attention(c, a["q"], a["k"], a["v"], a["out"], a["lse"], ws=a["ws"],
                                    stream=_S(), **kw)
    if status is None:
        assert isinstance(e.value, ValueError), e.value
    else:
        assert isinstance(e.value, T.FadeError) and e.value.status == status, e.value
    return str(e.value)


@pytest.mark.parametrize("mass", [False, True])
def test_lengths_windows_and_sinks(T, mass):
    for q_len, kv_len in (([6, 1], None), ([-1, 1], None), (None, [10, 9]), ([5, 5], [4, 9]),
                          (None, [-1, 9]), (None, [4, 9])):
        assert "row" in _prompt(T, 1, mass, q_len=q_len, kv_len=kv_len)
    for q_len in ([1], [1, 1, 1], [[1, 1]]):
        _prompt(T, None, mass, q_len=q_len)
    _prompt(T, 1, mass, n_sink=-1)
    _prompt(T, 1, mass, window=-1)
    _prompt(T, 1, mass, n_q=9, n_kv=5)   # more queries than tokens


@pytest.mark.parametrize("mass", [False, True])
def test_shapes_types_and_layouts(T, mass):
    big = _z(2, 5, 8, 65)
    _prompt(T, None, mass, q=_z(2, 5, 7, 64))
    _prompt(T, None, mass, q=_z(5, 8, 64))
    _prompt(T, None, mass, q=_z(2, 5, 8, 64, dt=torch.bfloat16))
    _prompt(T, None, mass, k=_z(2, 9, 3, 64))
    _prompt(T, None, mass, lse=_z(2, 5, 8))
    _prompt(T, None, mass, lse=_z(2, 8, 5, dt=torch.float32).transpose(1, 2))
    assert "16-byte" in _prompt(T, 1, mass, q=big[..., 1:])        # off the boundary
    assert "16-byte" in _prompt(T, 1, mass, q=big[..., :64])       # strides of 65 elements
    assert "every token" in _prompt(T, 2, mass, k=_z(2, 1, 2, 64).expand(2, 9, 2, 64))
    assert "every token or head" in _prompt(T, 2, mass, q=_z(2, 5, 1, 64).expand(2, 5, 8, 64))
    _prompt(T, None, mass, q=_z(2, 5, 64, 8).transpose(2, 3))      # channels apart
    _prompt(T, 2, mass, cfg=_cfg(T, num_q_heads=6), q=_z(2, 5, 6, 64), out=_z(2, 5, 6, 64),
            lse=_z(2, 5, 6, dt=torch.float32))                     # 3 query heads a KV head
    if mass:
        _prompt(T, None, mass, lse=None)
        _prompt(T, None, mass, mass=None)
        _prompt(T, None, mass, mass=_z(2, 2, 9))
        _prompt(T, None, mass, mass=_z(2, 9, 2, dt=torch.float32).transpose(1, 2))
    else:
        _prompt(T, None, v=_z(2, 8, 2, 64))
        _prompt(T, None, out=_z(2, 5, 8, 64, dt=torch.float32))
        assert "16-byte" in _prompt(T, 1, out=big[..., :64])
        assert "every token" in _prompt(T, 2, v=_z(2, 1, 2, 64).expand(2, 9, 2, 64))
        for one in ((1, 5, 8, 64), (2, 1, 8, 64), (2, 5, 1, 64)):   # results over each other
            assert "share vectors" in _prompt(T, 1, out=_z(*one).expand(2, 5, 8, 64))


@pytest.mark.parametrize("mass", [False, True])
def test_workspaces(T, mass):
    need = T.fade_prompt_ws_bytes(_cfg(T), 5, 9)
    assert need > 0 and need % 16 == 0
    flat = _z(need + 16, dt=torch.uint8)
    at = (-flat.data_ptr()) % 16
    _prompt(T, 3, mass, ws=flat[at:at + 64])
    assert "16-byte" in _prompt(T, 1, mass, ws=flat[at + 1:at + need - 15])
    for bad in ((0, 9), (5, 0), (-1, 9), (5, 1 << 25)):
        with pytest.raises(T.FadeError) as e:
            T.fade_prompt_ws_bytes(_cfg(T), *bad)
        assert e.value.status == 1


def test_null_pointers(T):
    import ctypes

    from tiered_mixed_precision_gb300 import fade as F

    L, c = T.lib(), ctypes.byref(_cfg(T).c())
    x = _z(2, 9, 8, 64)
    f = _z(2, 9, 8, dt=torch.float32)
    h, n = F._heads(x), None
    none = ctypes.byref(F.HeadsT(None, 0, 0, 0))
    p = F._ptr(f)
    assert L.fade_prompt_attention(c, h, h, h, 9, 9, n, n, 0, 0, h, p, n, n, 0, n) == 1      # no ws
    assert L.fade_prompt_attention(c, h, h, n, 9, 9, n, n, 0, 0, h, p, n, p, 1 << 30, n) == 1
    assert L.fade_prompt_attention(c, h, h, h, 9, 9, n, n, 0, 0, none, p, n, p, 1 << 30, n) == 1
    assert L.fade_prompt_attention(n, h, h, h, 9, 9, n, n, 0, 0, h, p, n, p, 1 << 30, n) == 1
    assert L.fade_prompt_mass(c, h, h, 9, 9, n, n, 0, 0, n, 0, p, n, p, 1 << 30, n) == 1
    assert L.fade_prompt_mass(c, h, h, 9, 9, n, n, 0, 0, p, 0, n, n, p, 1 << 30, n) == 1
    neg = ctypes.byref(F.HeadsT(x.data_ptr() + 4096, -64, 64, 64))
    assert L.fade_prompt_mass(c, neg, h, 9, 9, n, n, 0, 0, p, 0, p, n, p, 1 << 30, n) == 2
    assert b"negative" in L.fade_last_error()


def _verify(T, status, **kw):
    B, N, V = 2, 5, 40
    i32, f32 = torch.int32, torch.float32
    a = dict(parents=_z(B, N, dt=i32), n_nodes=None, tokens=_z(B, N, dt=i32), target=_z(B, N, V),
             target_root=_z(B, V), draft=_z(B, N, V), draft_root=_z(B, V),
             temperature=_z(B, dt=f32), u=_z(B, N, dt=f32), noise=_z(B, V, dt=f32),
             path=_z(B, N, dt=i32), n_path=_z(B, dt=i32), next_token=_z(B, dt=i32))
    a.update(kw)
    with pytest.raises((T.FadeError, ValueError)) as e:
        T.fade_tree_verify(_cfg(T), *a.values(), stream=_S())
    if status is None:
        assert isinstance(e.value, ValueError), e.value
    else:
        assert isinstance(e.value, T.FadeError) and e.value.status == status, e.value
    return str(e.value)


def test_verify_refuses(T):
    i32, f32 = torch.int32, torch.float32
    _verify(T, None, target=None)
    _verify(T, None, parents=None)
    _verify(T, None, target=_z(2, 5, 40, dt=torch.float64))
    _verify(T, None, target=_z(2, 4, 40))
    _verify(T, None, target=_z(5, 40))
    _verify(T, None, target=_z(2, 40, 5).transpose(1, 2))
    _verify(T, None, target_root=_z(2, 41))
    _verify(T, None, draft=_z(2, 5, 40, dt=torch.bfloat16))      # not the target's type
    _verify(T, None, u=_z(2, 4, dt=f32))
    _verify(T, None, u=_z(2, 5))
    _verify(T, None, noise=_z(2, 41, dt=f32))
    _verify(T, None, noise=_z(40, 2, dt=f32).t())
    _verify(T, None, temperature=_z(1, dt=f32))
    _verify(T, None, tokens=_z(2, 5, dt=torch.int64))
    _verify(T, None, path=_z(2, 6, dt=i32))
    _verify(T, None, n_path=_z(3, dt=i32))
    assert "uniform" in _verify(T, 1, u=None)
    assert "drafter logits" in _verify(T, 1, draft_root=None)
    assert "drafter logits" in _verify(T, 1, draft=None)
    assert "drafter logits" in _verify(T, 1, target_root=None)
    _verify(T, 1, parents=_z(2, 65, dt=i32), tokens=_z(2, 65, dt=i32), target=_z(2, 65, 40),
            draft=_z(2, 65, 40), u=_z(2, 65, dt=f32), path=_z(2, 65, dt=i32))
    _verify(T, 1, target=_z(2, 5, 0), draft=_z(2, 5, 0), target_root=_z(2, 0), draft_root=_z(2, 0),
            noise=_z(2, 0, dt=f32))


def test_verify_null_and_misaligned(T):
    import ctypes

    from tiered_mixed_precision_gb300 import fade as F

    L, c = T.lib(), ctypes.byref(_cfg(T).c())
    i, x = F._ptr(_z(2, 5, dt=torch.int32)), _z(2, 5, 40)
    t = ctypes.byref(F.LogitsT(x.data_ptr(), 200, 40))
    odd = ctypes.byref(F.LogitsT(x.data_ptr() + 1, 200, 40))
    n = None
    args = lambda **k: [c, 5, 40, k.get("ty", 0), k.get("par", i), n, i, k.get("t", t), n, n, n, n, n,
                        n, k.get("path", i), i, i, n]
    assert L.fade_tree_verify(*args(par=n)) == 1
    assert L.fade_tree_verify(*args(path=n)) == 1
    assert L.fade_tree_verify(*args(t=n)) == 1
    assert L.fade_tree_verify(*args(t=odd)) == 1
    assert L.fade_tree_verify(*args(ty=3)) == 1
    assert L.fade_tree_verify(*args(ty=-1)) == 1
    assert L.fade_tree_verify(*args(path=ctypes.c_void_p(i.value + 2))) == 1


def test_the_cache_refuses_a_prompt_attention_without_queries(T):
    from tiered_mixed_precision_gb300.model import FadeCache

    cache = FadeCache.__new__(FadeCache)   # (no CUDA buffers: the checks come first)
    cache.cfg, cache.qk_norm = _cfg(T), [None]
    k = _z(2, 2, 9, 64)
    with pytest.raises(ValueError, match="q_raw"):
        cache.prefill(0, k, k, out=_z(2, 8, 9, 64))
    with pytest.raises(ValueError, match="q_raw"):
        cache.prefill(0, k, k, window=4)
    with pytest.raises(ValueError, match="out"):
        cache.prefill(0, k, k, q_raw=_z(2, 8, 9, 64), window=4)
