"""Values and keys that are not finite and that a query sees, in shares of an item whose weight beside the
others is nothing: they reach the query's result however its tokens are divided among CTAs."""

import math

import numpy as np
import pytest
import torch

from test_gpu_prompt import F, _cfg, _draw  # noqa: F401  (F: the fixture)

pytestmark = pytest.mark.gpu


def _inputs(B, n_q, n_kv, hq, h, d):
    """Queries of 2 in every channel. Keys of +-1/8 and, in a row's first 512 tokens, of -8: their logits
    lie 16 sqrt(d) - 1/4 sqrt(d) > 126 below the others', so that e^.. and 2^.. of that are 0 in fp32."""
    q = torch.full((B, n_q, hq, d), 2.0, dtype=torch.float16, device="cuda")
    k = _draw((B, n_kv, h, d), 1).sign() / 8
    k[:, :512] = -8
    return q, k.half(), _draw((B, n_kv, h, d), 2)


def _attend(F, q, k, v, **see):
    B, n_q, hq, d = q.shape
    out = torch.full_like(q, 7.0)
    lse = torch.full((B, n_q, hq), 7.0, device="cuda")
    F.fade_prompt_attention(_cfg(F, B, hq, k.shape[2], d), q, k, v, out, lse, **see)
    torch.cuda.synchronize()
    return out, lse


# rows: one is divided among the CTAs; of 40 x 4 units the longest (row 0) is taken whole
@pytest.mark.parametrize("B", [1, 40])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n_q", [1, 3, 130])
@pytest.mark.parametrize("sink,window", [(0, 0), (600, 100)])
def test_values_that_are_not_finite(F, B, d, n_q, sink, window):
    hq, h, n_kv = 8, 4, 4096
    q, k, v = _inputs(B, n_q, n_kv, hq, h, d)
    kv_len = np.full(B, n_kv, np.int32)
    kv_len[1:] -= 200
    see = dict(kv_len=kv_len, n_sink=sink, window=window)
    plain, plain_lse = _attend(F, q, k, v, **see)
    assert bool(torch.isfinite(plain).all())
    v[0, 10, :, 3] = math.nan
    v[0, 20, :, 5] = math.inf
    v[0, 300, :, 7] = -math.inf
    v[0, 301, 1, 9] = math.inf
    out, lse = _attend(F, q, k, v, **see)
    bad = torch.zeros((hq, d), dtype=torch.bool, device="cuda")
    bad[:, [3, 5, 7]] = True
    bad[2:4, 9] = True     # the query heads of KV head 1
    assert torch.equal(~torch.isfinite(out[0]), bad.expand(n_q, hq, d))
    assert bool(torch.isnan(out[0, :, :, 3]).all())
    assert torch.equal(out[0][:, ~bad], plain[0][:, ~bad]) and torch.equal(lse, plain_lse)
    assert torch.equal(out[1:], plain[1:])


@pytest.mark.parametrize("B", [1, 40])
@pytest.mark.parametrize("d", [64, 128])
def test_a_key_that_is_not_a_number(F, B, d):
    """Its logit is NaN: so are the row's results."""
    hq, h, n_q, n_kv = 8, 4, 3, 4096
    q, k, v = _inputs(B, n_q, n_kv, hq, h, d)
    kv_len = np.full(B, n_kv, np.int32)
    kv_len[1:] -= 200
    k[0, 30, 1, 2] = math.nan
    out, lse = _attend(F, q, k, v, kv_len=kv_len)
    assert bool(torch.isnan(out[0, :, 2:4]).all()) and bool(torch.isnan(lse[0, :, 2:4]).all())
    assert bool(torch.isfinite(out[0, :, [0, 1, 4, 5, 6, 7]]).all()) and bool(torch.isfinite(out[1:]).all())
