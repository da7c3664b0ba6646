"""Verification where runs of the drafter's logits are NaN (a smaller drafter's vocabulary whose padding was
never written): q is 0 there, so that all of p is left of those tokens after a refusal."""

import math

import numpy as np
import pytest
import torch

from test_gpu_verify import F, _call, _compare, _inputs  # noqa: F401  (F: the fixture)

pytestmark = pytest.mark.gpu

DTYPES = [torch.float16, torch.bfloat16, torch.float32]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V,start,n", [(64, 0, 16), (64, 48, 16), (1000, 0, 64), (1000, 936, 64),
                                       (4096, 2048, 64), (16384, 16320, 64), (40001, 0, 39000)])
def test_the_residual_keeps_what_the_drafter_does_not_have(F, V, start, n, dtype):
    """p = 1 / V everywhere, q = 1 / (V - n) outside the run: two drafts outside it are refused (u is
    above the ratio, 0.9961 at most), r is 1 / V in the run and 0 outside, where the noise is least."""
    B, T = 3, 2
    zero = lambda *s: torch.zeros(s, dtype=dtype)
    outside = start - 1 if start else n
    st = dict(parents=torch.full((B, T), -1, dtype=torch.int32), n_nodes=None,
              tokens=torch.full((B, T), outside, dtype=torch.int32), target=zero(B, T, V),
              target_root=zero(B, V), draft=zero(B, T, V), draft_root=zero(B, V), temperature=None,
              u=torch.full((B, T), 0.999), noise=torch.ones((B, V)))
    st["draft_root"][:, start:start + n] = math.nan
    st["draft_root"][1, start:start + n:2] = -math.inf   # (row 1: NaN and -inf in turn)
    st["noise"][:, outside] = 1e-3
    want = [start, start + n // 2, start + n - 1]
    for b, w in enumerate(want):
        st["noise"][b, w] = 0.5
    path, n_path, nxt = _call(F, st, B, T)
    assert n_path.tolist() == [0] * B and nxt.tolist() == want


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [777, 4096, 20001, 70001])
def test_runs_of_nan_in_the_drafter(F, V, dtype):
    """Siblings that are refused now and then, the drafter's runs at the start, in the middle, at the end, of
    8 to 64 tokens, some of NaN and -inf in turn: against the definition."""
    B, T = 24, 6
    for seed in (1, 2, 3):
        st = _inputs(B, T, V, dtype, 100 * seed + V, vary=False)
        st["temperature"][:] = torch.from_numpy(
            np.random.default_rng(seed).choice([0.6, 1.0, 1.7], B).astype(np.float32))
        st["parents"][:, :4] = -1
        st["u"] = 0.5 + 0.5 * st["u"]
        rng = np.random.default_rng(V + seed)
        for b in range(B):
            n = int(rng.integers(8, 65))
            start = [0, int(rng.integers(0, V - n)), V - n][b % 3]
            for x in (st["draft"][b], st["draft_root"][b]):
                x[..., start:start + n] = math.nan
                if b % 4 == 3:
                    x[..., start:start + n:3] = -math.inf
        _compare(F, st, B, T, near=0.1)
