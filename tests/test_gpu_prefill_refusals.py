"""A refused prefill leaves prompt, layer and counts as they were."""

import numpy as np
import pytest
import torch

from test_gpu_prompt import _draw
from test_gpu_request import F, _cache  # noqa: F401  (F: the fixture)

pytestmark = pytest.mark.gpu

B, HQ, H, D, P = 2, 8, 2, 64, 300


def _state(cache):
    L = cache.layers[0]
    bufs = [t.clone() for n in cache._STATE_BUFFERS
            for t in (getattr(L, n) if isinstance(getattr(L, n), list) else [getattr(L, n)])]
    return bufs, [getattr(L, n).copy() for n in ("h_n_sink", "h_n_mid", "h_n_recent")]


def _new(*s, dtype=torch.float16):
    return torch.zeros(s, dtype=dtype, device="cuda")


REFUSED = {
    "out of another shape": lambda: dict(out=_new(B, HQ, P - 1, D)),
    "out of another type": lambda: dict(out=_new(B, HQ, P, D, dtype=torch.bfloat16)),
    "out with its channels apart": lambda: dict(out=_new(B, HQ, D, P).transpose(2, 3)),
    "out off the boundary": lambda: dict(out=_new(B, HQ, P, D + 1)[..., :D]),
    "out on the host": lambda: dict(out=torch.zeros((B, HQ, P, D), dtype=torch.float16)),
    "out that shares vectors": lambda: dict(out=_new(B, HQ, 1, D).expand(B, HQ, P, D)),
    "a window below 0": lambda: dict(window=-1),
    "a length past the prompt": lambda: dict(prompt_len=np.array([P, P + 1])),
    "a length below 0": lambda: dict(prompt_len=np.array([P, -1])),
    "one length": lambda: dict(prompt_len=np.array([P])),
    "queries of another shape": lambda: dict(q_raw=_new(B, HQ, P - 1, D)),
    "queries of another type": lambda: dict(q_raw=_new(B, HQ, P, D, dtype=torch.float32)),
    "queries in another order": lambda: dict(q_raw=_new(B, P, HQ, D).transpose(1, 2)),
    "keys in another order": lambda: dict(k_raw=_new(B, P, H, D).transpose(1, 2)),
    "values in another order": lambda: dict(v=_new(B, P, H, D).transpose(1, 2)),
    "values of another shape": lambda: dict(v=_new(B, H, P + 1, D)),
}


OF_ATTENTION = [w for w in REFUSED if "out" in w.split() or "window" in w]


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("what,attends", [(w, True) for w in REFUSED] +
                         [(w, False) for w in REFUSED if w not in OF_ATTENTION])
def test_a_refused_prefill_changes_nothing(F, what, attends, norm):
    bad = REFUSED[what]()
    cache, other = (_cache(F, "h2o", 1) for _ in range(2))
    if norm:
        w = [(1 + 0.2 * _draw((D,), 50 + i)).half() for i in range(2)]
        cache.set_qk_norm(*w)
        other.set_qk_norm(*w)

    def prompt():
        a = dict(k_raw=_draw((B, H, P, D), 2), v=_draw((B, H, P, D), 3), q_raw=_draw((B, HQ, P, D), 1),
                 prompt_len=np.array([P, 171], np.int32))
        return {**a, **(dict(out=torch.full((B, HQ, P, D), 7.0, dtype=torch.float16, device="cuda"))
                        if attends else {})}

    cache.prefill(0, **{**prompt(), "v": _draw((B, H, P, D), 4)})
    before = _state(cache)
    a = {**prompt(), **bad}
    with pytest.raises((F.FadeError, ValueError)):
        cache.prefill(0, **a)
    fresh = prompt()
    for name in ("k_raw", "v", "q_raw", "out"):
        if name not in bad and name in fresh:
            assert torch.equal(a[name], fresh[name]), name
    for x, y in zip(_state(cache)[0] + before[1], before[0] + _state(cache)[1]):
        assert (np.array_equal(x, y) if isinstance(x, np.ndarray) else torch.equal(x, y))
    # the same prompt again, as it should be: what a cache that never refused has
    a, b = prompt(), prompt()
    cache.prefill(0, **a)
    other.prefill(0, **b)
    L, M = cache.layers[0], other.layers[0]
    for n in ("sink_k", "recent_k", "recent_v", "sink_scores", "recent_scores"):
        assert torch.equal(getattr(L, n), getattr(M, n)), n
    assert torch.equal(a["k_raw"], b["k_raw"]) and torch.equal(a["q_raw"], b["q_raw"])
    if attends:
        assert torch.equal(a["out"], b["out"])
