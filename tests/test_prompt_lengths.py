"""Numbers of a prompt call that a 32-bit integer does not hold are not taken modulo 2^32: lengths are
refused, and so are windows and sinks below 0; larger ones hide, or keep, what all tokens' would."""

import ctypes

import numpy as np
import pytest
import torch


class _S:  # a stream handle that is never used (no launch happens)
    cuda_stream = 0


@pytest.fixture(scope="module")
def T():
    from tiered_mixed_precision_gb300 import build

    build.build()
    import tiered_mixed_precision_gb300 as T

    return T


def _z(*s, dt=torch.float16):
    return torch.zeros(s, dtype=dt)


def _call(T, mass, **lens):
    cfg = T.Config(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=64, mid_capacity=8)
    q, k, ws = _z(2, 5, 8, 64), _z(2, 9, 2, 64), _z(1 << 24, dt=torch.uint8)
    lse = _z(2, 5, 8, dt=torch.float32)
    if mass:
        T.fade_prompt_mass(cfg, q, k, lse, _z(2, 2, 9, dt=torch.float32), ws=ws, stream=_S(), **lens)
    else:
        T.fade_prompt_attention(cfg, q, k, k, q.clone(), lse, ws=ws, stream=_S(), **lens)


@pytest.mark.parametrize("mass", [False, True])
@pytest.mark.parametrize("lens", [np.array([2 ** 32 + 5, 1]), np.array([1, -2 ** 32]),
                                  np.array([2 ** 40, 0], np.uint64), np.array([1.5, 2.0]),
                                  np.array([np.nan, 1.0]), torch.tensor([2 ** 32, 3])], ids=str)
@pytest.mark.filterwarnings("ignore:invalid value")
def test_lengths_that_do_not_fit(T, mass, lens):
    with pytest.raises(ValueError, match="q_len"):
        _call(T, mass, q_len=lens)
    with pytest.raises(ValueError, match="kv_len"):
        _call(T, mass, kv_len=lens)


@pytest.mark.parametrize("zero", [[0, 0], np.zeros(2), np.zeros(2, np.int64), np.zeros(2, np.uint8),
                                  torch.zeros(2, dtype=torch.int64), np.zeros(4, np.int32)[::2]], ids=str)
def test_integers_of_any_type_are_taken(T, zero):
    """(without queries an attention call looks at its arguments and does nothing)"""
    _call(T, False, q_len=zero)


@pytest.mark.parametrize("mass", [False, True])
@pytest.mark.parametrize("kw", [dict(window=-2 ** 32), dict(n_sink=-2 ** 32), dict(window=-2 ** 32 + 3),
                                dict(n_sink=1 - 2 ** 33)], ids=str)
def test_far_below_0(T, mass, kw):
    with pytest.raises(T.FadeError, match="below 0"):
        _call(T, mass, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("wide,same", [(dict(window=2 ** 32 + 3), {}), (dict(window=2 ** 31), {}),
                                       (dict(window=7, n_sink=2 ** 32), dict(window=7, n_sink=300)),
                                       (dict(window=7, n_sink=2 ** 32 + 2), dict(window=7, n_sink=300))],
                         ids=str)
def test_more_than_any_prompt_has(T, wide, same):
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn((2, 300, n, 64), generator=g).half().cuda() for n in (8, 2, 2))
    cfg = T.Config(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=64, mid_capacity=8)
    got = []
    for see in (wide, same):
        out, lse = torch.zeros_like(q), torch.zeros((2, 300, 8), device="cuda")
        mass = torch.zeros((2, 2, 300), device="cuda")
        T.fade_prompt_attention(cfg, q, k, v, out, lse, **see)
        T.fade_prompt_mass(cfg, q, k, lse, mass, **see)
        got.append((out, lse, mass))
    for x, y in zip(*got):
        assert torch.equal(x, y)
