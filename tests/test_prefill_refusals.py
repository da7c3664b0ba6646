"""Without a GPU: a prefill looks at all its arguments before it rotates or resets anything."""

import ctypes
from types import SimpleNamespace

import numpy as np
import pytest
import torch


class _Written(Exception):
    pass


@pytest.fixture()
def cache(monkeypatch):
    from tiered_mixed_precision_gb300 import build

    build.build()
    from tiered_mixed_precision_gb300 import fade as F
    from tiered_mixed_precision_gb300.model import FadeCache

    def written(*a, **kw):
        raise _Written

    for name in ("fade_rope_apply", "fade_qk_norm_rope", "fade_cache_reset"):
        monkeypatch.setattr(F, name, written)
    F._device(None)   # (imports torch for the argument checks)
    monkeypatch.setattr(F, "_device", lambda stream: None)   # host tensors pass
    monkeypatch.setattr(F, "_stream", lambda stream: ctypes.c_void_p(0))
    c = FadeCache.__new__(FadeCache)
    c.cfg = F.Config(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=64, mid_capacity=64, policy="h2o")
    c.qk_norm, c.table, c.max_pos, c.device = [None], None, 64, torch.device("cpu")
    c.layers = [SimpleNamespace(status=torch.zeros(F.STATUS_WORDS, dtype=torch.int32))]
    return c


def _z(*s, dt=torch.float16):
    return torch.zeros(s, dtype=dt)


def _prompt(**kw):
    return {**dict(k_raw=_z(2, 2, 9, 64), v=_z(2, 2, 9, 64), q_raw=_z(2, 8, 9, 64),
                   prompt_len=np.array([9, 4], np.int32), out=_z(2, 8, 9, 64)), **kw}


@pytest.mark.parametrize("kw", [{}, dict(window=3), dict(out=None), dict(prompt_len=None),
                                dict(prompt_len=[0, 9]),
                                dict(out=_z(2, 9, 8, 64).transpose(1, 2))], ids=str)
@pytest.mark.parametrize("norm", [False, True])
def test_what_is_in_order_comes_to_the_rotation(cache, kw, norm):
    if norm:
        cache.qk_norm = [(_z(64), _z(64), 1e-6)]
    with pytest.raises(_Written):
        cache.prefill(0, **_prompt(**kw))


@pytest.mark.parametrize("kw", [
    dict(out=_z(2, 8, 8, 64)), dict(out=_z(2, 8, 9, 64, dt=torch.bfloat16)), dict(out=_z(2, 8, 9, 65)[..., :64]),
    dict(out=_z(2, 8, 64, 9).transpose(2, 3)), dict(out=_z(2, 8, 1, 64).expand(2, 8, 9, 64)),
    dict(window=-1), dict(prompt_len=[9, 10]), dict(prompt_len=[-1, 9]), dict(prompt_len=[9]),
    dict(out=None, prompt_len=[9, 10]), dict(out=None, prompt_len=[9]),
    dict(q_raw=_z(2, 8, 8, 64)), dict(out=None, q_raw=_z(2, 8, 8, 64)), dict(q_raw=_z(2, 9, 8, 64).transpose(1, 2)),
    dict(k_raw=_z(2, 9, 2, 64).transpose(1, 2)), dict(k_raw=_z(1, 2, 9, 64)), dict(v=_z(2, 2, 10, 64)),
    dict(v=_z(2, 2, 9, 64, dt=torch.float32))], ids=str)
def test_what_is_not_is_refused_before(cache, kw):
    from tiered_mixed_precision_gb300 import FadeError

    with pytest.raises((FadeError, ValueError)):
        cache.prefill(0, **_prompt(**kw))
