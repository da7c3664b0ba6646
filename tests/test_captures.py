"""Captured steps while the program leaves cycles that Python's collector would take apart."""

import contextlib
import gc

import pytest
import torch


@pytest.mark.parametrize("collects", [True, False])
def test_no_collection_while_a_capture_is_open(monkeypatch, collects):
    from tiered_mixed_precision_gb300 import model

    seen = []

    @contextlib.contextmanager
    def graph(g):
        seen.append((g, gc.isenabled()))
        yield
        seen.append((g, gc.isenabled()))

    monkeypatch.setattr(torch.cuda, "graph", graph)
    was = gc.isenabled()
    (gc.enable if collects else gc.disable)()
    try:
        with model._capturing("one"):
            seen.append(gc.isenabled())
        assert seen == [("one", False), False, ("one", False)] and gc.isenabled() == collects
        with pytest.raises(KeyError):
            with model._capturing("two"):
                raise KeyError
        assert gc.isenabled() == collects
    finally:
        (gc.enable if was else gc.disable)()


@pytest.mark.gpu
@pytest.mark.parametrize("growing", [False, True])
def test_a_graph_left_in_a_cycle(growing):
    """A graph in a cycle of garbage, and containers enough to call the collector, inside the capture."""
    from tiered_mixed_precision_gb300 import build

    build.build()
    from tiered_mixed_precision_gb300 import fade as F
    from tiered_mixed_precision_gb300.model import FadeCache

    B, hq, h, d, P = 2, 8, 2, 64, 300
    cfg = F.Config(batch=B, num_q_heads=hq, num_kv_heads=h, head_dim=d, n_sink=4, recent_window=32,
                   int4_budget=-1 if growing else 100, mid_capacity=P + 200,
                   policy="none" if growing else "position")
    cache = FadeCache(cfg, 1, P, 4096)
    draw = lambda *s: torch.randn(s, device="cuda").half()
    cache.prefill(0, draw(B, h, P, d), draw(B, h, P, d))
    q, k, v, out = draw(1, B, hq, d), draw(1, B, h, d), draw(1, B, h, d), draw(1, B, hq, d)
    for _ in range(2):   # to the steady state
        cache.set_positions(cache.next_positions())
        cache.step_all(q, k, v, out)
    other, x = torch.cuda.CUDAGraph(), torch.zeros(4, device="cuda")
    with torch.cuda.graph(other):
        x += 1

    class Box:
        pass

    box = Box()
    box.me, box.graph = box, other
    left = [box]
    del box, other
    step = cache.step_layer

    def leaving(*a):
        left.clear()
        kept = [[i] for i in range(100000)]
        assert len(kept) == 100000
        return step(*a)

    cache.step_layer = leaving
    cache.set_positions(cache.next_positions())
    g = (cache.capture_growing_step if growing else cache.capture_step)(q, k, v, out)
    cache.step_layer = step
    gc.collect()
    if growing:
        cache.replay_growing(g)
    else:
        g.replay()
    torch.cuda.synchronize()
    assert bool(torch.isfinite(out).all())
    F.fade_check_status(cache.layers[0])
