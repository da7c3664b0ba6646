"""A request's two ends together, through FadeCache: the prompt attends and fills the cache, trees are
drafted, attended to, verified and committed."""

import numpy as np
import pytest
import torch

from test_gpu_prompt import _check, _draw
from test_gpu_verify import _definition

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def F():
    from tiered_mixed_precision_gb300 import build

    build.build()
    from tiered_mixed_precision_gb300 import fade

    return fade


def _cache(F, policy, layers, B=2, hq=8, h=2, d=64, P=300, **kw):
    from tiered_mixed_precision_gb300.model import FadeCache

    cfg = F.Config(batch=B, num_q_heads=hq, num_kv_heads=h, head_dim=d, n_sink=4, recent_window=32,
                   int4_budget=100 if policy != "none" else -1, mid_capacity=P + 200, policy=policy, **kw)
    return FadeCache(cfg, num_layers=layers, max_prompt=P, max_pos=4096)


def _layers_equal(a, b):
    for x, y in zip(a.layers, b.layers):
        for name in a._STATE_BUFFERS:
            u, v = getattr(x, name), getattr(y, name)
            for s, t in zip(u, v) if isinstance(u, list) else [(u, v)]:
                assert torch.equal(s, t), name


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("policy,window", [("h2o", 0), ("h2o", 90), ("position", 132), ("none", 0)])
def test_prefill_attends(F, policy, window, norm):
    """The attention's outputs, its mass, and the cache that a prefill with that mass makes."""
    B, hq, h, d, P = 2, 8, 2, 64, 300
    lens = np.array([300, 171], np.int32)
    cache, other = (_cache(F, policy, 1) for _ in range(2))
    if norm:
        w = [(1 + 0.2 * _draw((d,), 50 + i)).half() for i in range(2)]
        cache.set_qk_norm(*w)
        other.set_qk_norm(*w)
    q, k, v = _draw((B, hq, P, d), 1), _draw((B, h, P, d), 2), _draw((B, h, P, d), 3)
    q2, k2 = q.clone(), k.clone()
    out = torch.full_like(q, 7.0)
    mass = cache.prefill(0, k, v, lens, q_raw=q, out=out, window=window)
    cfg = cache.cfg
    # (q and k are rotated now)
    ref = _check(F, cfg, q.transpose(1, 2), k.transpose(1, 2), v.transpose(1, 2), lens, lens, 4, window)
    assert torch.equal(out.transpose(1, 2), ref[0])
    if policy == "h2o":
        assert torch.equal(mass, ref[2])
        if not window:   # what the prefill without attention would have used
            rows = torch.empty_like(mass)
            F.fade_prefill_mass(cfg, q, k, P, lens, rows)
            assert bool(((mass - rows).abs() <= 2.0 ** -14 * rows).all())
    else:
        assert mass is None
    other.prefill(0, k2, v, lens, mass=mass)
    _layers_equal(cache, other)
    assert torch.equal(k, k2)
    F.fade_check_status(cache.layers[0])


@pytest.mark.parametrize("mode", ["sampled", "certain", "greedy"])
@pytest.mark.parametrize("policy", ["h2o", "position", "none"])
def test_request(F, policy, mode):
    """Prompt, then three drafted trees: layers attend, a head makes logits of the last one's output, the
    kept paths are committed. Verification against its definition, the cache's counts against the paths;
    a second cache that commits the same paths by hand ends in the same state."""
    B, hq, h, d, P, T, V, layers = 2, 8, 2, 64, 300, 7, 101, 2
    lens = np.array([300, 171], np.int32)
    cache, other = (_cache(F, policy, layers) for _ in range(2))
    for c in (cache, other):
        for layer in range(layers):
            q, k, v = (_draw((B, n, P, d), 10 * layer + i) for i, n in enumerate((hq, h, h)))
            c.prefill(layer, k, v, lens, q_raw=q, out=torch.empty_like(q))
    head = _draw((hq * d, V), 90, 0.3).float()
    g = torch.Generator(device="cuda").manual_seed(7)
    rng = np.random.default_rng(7)
    for step in range(3):
        par = np.full((B, T), -1, np.int32)
        for i in range(1, T):
            par[:, i] = rng.integers(max(0, i - 3), i, B)
        parents = torch.from_numpy(par).cuda()
        n_nodes = torch.tensor([T, T - step], dtype=torch.int32, device="cuda")
        outs, trees = [], []
        for c in (cache, other):
            tree = c.tree_begin(parents, n_nodes)
            out = torch.zeros((B, T, hq, d), dtype=torch.float16, device="cuda")
            for layer in range(layers):
                q, k, v = (_draw((B, T, n, d), 1000 * step + 10 * layer + i)
                           for i, n in enumerate((hq, h, h)))
                c.tree_attend(layer, tree, q, k, v, out)
            outs.append(out)
            trees.append(tree)
        assert torch.equal(*outs)
        target = (outs[0].float().reshape(B, T, hq * d) @ head).half()
        draft = (target.float() + torch.randn(target.shape, generator=g, device="cuda")).half()
        q = torch.softmax(draft.float(), -1)
        at = parents.clamp(min=0).long()
        tokens = torch.multinomial(q[torch.arange(B, device="cuda")[:, None], at].reshape(B * T, V), 1,
                                   generator=g).reshape(B, T).int()
        if mode == "greedy":   # the first drafts are the target's own
            tokens[:, 1:3] = target[torch.arange(B, device="cuda")[:, None], at[:, 1:3]].argmax(-1).int()
        u = None if mode == "greedy" else 0.5 * torch.rand((B, T), generator=g, device="cuda")
        noise = torch.empty((B, V), device="cuda").exponential_(generator=g)
        path, n_path, nxt = cache.tree_verify(trees[0], tokens, target,
                                              draft=draft if mode == "sampled" else None, u=u,
                                              noise=noise)
        n = n_path.tolist()
        host = lambda x, b: None if x is None else x[b].float().cpu().numpy()
        for b in range(B):
            want, token, margin = _definition(
                par[b], int(n_nodes[b]), tokens[b].cpu().numpy(), host(target, b), None,
                host(draft, b) if mode == "sampled" else None, None, 1.0, host(u, b), host(noise, b))
            if margin > 1e-4:
                assert path[b, :n[b]].tolist() == want and int(nxt[b]) == token
        assert all(x >= 1 for x in n)
        held = [cache.layers[0].h_n_mid + cache.layers[0].h_n_recent + cache.layers[0].h_n_sink]
        cache.tree_commit(trees[0], path, n)
        other.tree_commit(trees[1], path.clone(), np.array(n, np.int32))
        L = cache.layers[0]
        assert (L.h_n_mid + L.h_n_recent + L.h_n_sink - held[0] == n).all()
    _layers_equal(cache, other)
    for L in cache.layers:
        F.fade_check_status(L)


def test_captured_draft_step(F):
    """Attention and verification of a tree captured into one graph, replayed with other inputs."""
    B, hq, h, d, T, V = 2, 8, 2, 64, 5, 1000
    cache = _cache(F, "none", 1)
    q, k, v = _draw((B, hq, 300, d), 1), _draw((B, h, 300, d), 2), _draw((B, h, 300, d), 3)
    cache.prefill(0, k, v)
    parents = torch.tensor([[-1, 0, 0, 1, 3]] * B, dtype=torch.int32, device="cuda")
    tree = cache.tree_begin(parents)
    qs, ks, vs = _draw((B, T, hq, d), 4), _draw((B, T, h, d), 5), _draw((B, T, h, d), 6)
    out = torch.zeros_like(qs)
    head = _draw((hq * d, V), 7, 0.2)
    tokens = torch.randint(V, (B, T), device="cuda").int()
    u, noise = torch.rand((B, T), device="cuda") * 1e-3, torch.rand((B, V), device="cuda") + 0.1

    def step():
        cache.tree_attend(0, tree, qs, ks, vs, out)
        return cache.tree_verify(tree, tokens, out.reshape(B, T, hq * d) @ head, u=u, noise=noise)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        res = step()
    for seed in (20, 21):
        qs.copy_(_draw((B, T, hq, d), seed))
        tokens.copy_(torch.randint(V, (B, T), device="cuda").int())
        g.replay()
        got = [x.clone() for x in res]
        for x, y in zip(got, step()):
            assert torch.equal(x, y)


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs a second GPU")
def test_other_device_is_refused(F):
    cfg = F.Config(batch=1, num_q_heads=4, num_kv_heads=2, head_dim=64, mid_capacity=8)
    x = torch.zeros((1, 3, 4, 64), dtype=torch.float16, device="cuda:1")
    with pytest.raises(ValueError, match="current CUDA device"):
        F.fade_prompt_attention(cfg, x, x[:, :, :2], x[:, :, :2], x)
