"""Verification of drafted trees on a GPU against the definition in 64 bits, and what it is for: the
tokens that come out are distributed as the target's own."""

import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def F():
    from tiered_mixed_precision_gb300 import build

    build.build()
    from tiered_mixed_precision_gb300 import fade

    return fade


def _cfg(F, B):
    return F.Config(batch=B, num_q_heads=4, num_kv_heads=2, head_dim=64, mid_capacity=64)


def _softmax(x, t):
    x = np.where(np.isnan(x), -np.inf, np.minimum(x.astype(np.float64), np.finfo(np.float32).max))
    if not (x > -np.inf).any():
        return np.zeros_like(x)
    e = np.exp((x - x.max()) / t)
    return e / e.sum()


def _definition(parents, n, tokens, target, root, draft, draft_root, temp, u, noise):
    """One row in 64 bits: (path, next, the smallest margin by which something was decided)."""
    V = target.shape[-1]
    path, cur, margin = [], -1, math.inf
    if root is None:
        if n == 0:
            return [], -1, margin
        path, cur = [0], 0
    greedy = u is None or not temp > 0
    while True:
        x = root if cur < 0 else target[cur]
        kids = [i for i in range(max(cur, -1) + 1, n)
                if (parents[i] if 0 <= parents[i] < i else -1) == cur]
        take = None
        if greedy:
            p = _softmax(x, 1.0)
            clean = np.where(np.isnan(x), -np.inf, x)
            nxt = int(np.argmax(clean)) if p.any() else -1
            take = next((i for i in kids if nxt >= 0 and tokens[i] == nxt), None)
        else:
            p, r, w = _softmax(x, temp), None, 1.0
            q = None if draft is None else _softmax(draft_root if cur < 0 else draft[cur], temp)
            r = p.copy()
            for i in kids:
                inside = 0 <= tokens[i] < V
                rx = r[tokens[i]] if inside else 0.0
                qx = (q[tokens[i]] if inside else 0.0) if q is not None else 1.0
                lhs = u[i] * qx * w
                if max(lhs, rx) > 0:
                    margin = min(margin, abs(lhs - rx) / max(lhs, rx))
                if lhs < rx:
                    take = i
                    break
                if q is not None:
                    r = np.maximum(r - w * q, 0.0)
                    w = r.sum()
                elif inside:
                    w -= r[tokens[i]]
                    r[tokens[i]] = 0.0
            if take is None:
                if not w > 1e-300:
                    r = p
                s = r / noise if noise is not None else r
                nxt = int(np.argmax(s)) if s.max() > 0 else -1
                top = np.sort(s)[-2:]
                if len(top) == 2 and top[1] > 0:
                    margin = min(margin, (top[1] - top[0]) / top[1])
        if take is None:
            return path, nxt, margin
        path.append(take)
        cur = take


def _inputs(B, T, V, dtype, seed, mode="sampled", root=True, scale=3.0, vary=True):
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    target = torch.randn((B, T + 1, V), generator=g) * scale
    draft = target + torch.randn((B, T + 1, V), generator=g)
    parents = np.full((B, T), -1, np.int32)
    for i in range(1, T):
        parents[:, i] = rng.integers(-1 if root else 0, i, B)
    target, draft = target.to(dtype), draft.to(dtype)
    at = torch.from_numpy(parents).long() + 1
    rows = torch.arange(B)[:, None]
    probs = torch.softmax(draft[rows, at].float(), -1).reshape(B * T, V)
    tokens = torch.multinomial(probs, 1, generator=g).reshape(B, T).int()
    st = dict(parents=torch.from_numpy(parents), tokens=tokens,
              n_nodes=torch.from_numpy(rng.integers(0, T + 1, B).astype(np.int32)) if vary else None,
              target=target[:, 1:], target_root=target[:, 0] if root else None,
              draft=draft[:, 1:] if mode == "sampled" else None,
              draft_root=draft[:, 0] if mode == "sampled" and root else None,
              temperature=torch.from_numpy(rng.choice([0.0, 0.6, 1.0, 1.7], B).astype(np.float32)),
              u=torch.rand((B, T), generator=g),
              noise=torch.empty((B, V)).exponential_(generator=g))
    if mode == "greedy":
        st["u"] = st["noise"] = st["temperature"] = None
    return st


def _call(F, st, B, T, cuda=None):
    d = cuda or {k: None if x is None else x.cuda() for k, x in st.items()}
    path = torch.full((B, T), 77, dtype=torch.int32, device="cuda")
    n_path, nxt = (torch.full((B,), 77, dtype=torch.int32, device="cuda") for _ in range(2))
    F.fade_tree_verify(_cfg(F, B), d["parents"], d["n_nodes"], d["tokens"], d["target"],
                       d["target_root"], d["draft"], d["draft_root"], d["temperature"], d["u"],
                       d["noise"], path, n_path, nxt)
    torch.cuda.synchronize()
    return path.cpu().numpy(), n_path.cpu().numpy(), nxt.cpu().numpy()


def _compare(F, st, B, T, near=0.02):
    """Decisions whose margin in 64 bits is below 1e-4 (fp32 sums are off by 1e-5 at most) may go either
    way: rows with such a one are left out, and few."""
    path, n_path, nxt = _call(F, st, B, T)
    f = lambda x, b: None if x is None else x[b].float().numpy() if x.dtype != torch.int32 else x[b].numpy()
    left_out = 0
    for b in range(B):
        n = T if st["n_nodes"] is None else int(st["n_nodes"][b])
        temp = 1.0 if st["temperature"] is None else float(st["temperature"][b])
        want, token, margin = _definition(
            f(st["parents"], b), n, f(st["tokens"], b), f(st["target"], b), f(st["target_root"], b),
            f(st["draft"], b), f(st["draft_root"], b), temp, f(st["u"], b), f(st["noise"], b))
        if margin < 1e-4:
            left_out += 1
            continue
        assert n_path[b] == len(want) and list(path[b, :len(want)]) == want and nxt[b] == token, \
            (b, want, token, path[b], n_path[b], nxt[b])
        assert (path[b, len(want):] == 0).all()
    assert left_out <= max(1, near * B)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("mode", ["sampled", "certain", "greedy"])
@pytest.mark.parametrize("B,T,V,root", [(1, 1, 1, True), (3, 1, 2, False), (5, 7, 31, True),
                                        (16, 64, 1000, True), (4, 16, 50257, False),
                                        (2, 9, 32768, True), (33, 5, 2049, False)])
def test_against_definition(F, B, T, V, root, mode, dtype):
    _compare(F, _inputs(B, T, V, dtype, B * 7 + T, mode, root), B, T)


def test_wide_vocabulary_and_many_rows(F):
    _compare(F, _inputs(3, 4, 150001, torch.bfloat16, 1), 3, 4)
    _compare(F, _inputs(256, 3, 500, torch.float16, 2), 256, 3)


def test_flat_and_sharp_distributions(F):
    for scale in (0.0, 0.01, 30.0):
        for mode in ("sampled", "certain", "greedy"):
            _compare(F, _inputs(8, 12, 3001, torch.float32, 5, mode, scale=scale), 8, 12)


def test_masked_logits(F):
    """-inf, NaN and +inf among the logits, rows without any, tokens outside the vocabulary."""
    B, T, V = 8, 6, 777
    for mode in ("sampled", "certain", "greedy"):
        for dtype in (torch.float16, torch.float32):
            st = _inputs(B, T, V, dtype, 9, mode, vary=False)
            low = torch.finfo(dtype).min
            for x in (st["target"], st["draft"]):
                if x is None:
                    continue
                x[0, :, ::2] = -math.inf
                x[1, :, 1::3] = math.nan
                x[2, :, 5] = math.inf
                x[3] = -math.inf
                x[4] = math.nan
                x[5, :, 100:] = low
            st["target_root"][6] = -math.inf
            st["tokens"][7] = torch.tensor([-1, V, 2 ** 31 - 1, -2 ** 31, 3, V + 5], dtype=torch.int32)
            _compare(F, st, B, T, near=0.2)
    nothing = _inputs(2, 3, 50, torch.float16, 3, "certain", vary=False)
    nothing["target"][:] = -math.inf
    nothing["target_root"][:] = -math.inf
    path, n_path, nxt = _call(F, nothing, 2, 3)
    assert (path == 0).all() and (n_path == 0).all() and (nxt == -1).all()


def test_ties_go_to_the_lowest_token(F):
    B, T, V = 2, 2, 5000
    st = _inputs(B, T, V, torch.float16, 3, "greedy", root=False, vary=False)
    st["target"][:] = 0
    st["target"][0, 0, [4999, 1234, 77]] = 5.0
    st["parents"][:] = torch.tensor([-1, 0])
    st["tokens"][:, 1] = 77
    path, n_path, nxt = _call(F, st, B, T)
    assert list(n_path) == [2, 1] and list(nxt) == [0, 0]
    st["target_root"] = None
    st["u"], st["noise"] = torch.full((B, T), 0.999), torch.ones((B, V))
    st["tokens"][:] = 4000
    path, n_path, nxt = _call(F, st, B, T)
    assert list(n_path) == [1, 1] and list(nxt) == [77, 0]


def test_no_nodes_strides_and_alignment(F):
    B, T, V = 6, 5, 1001
    for dtype in (torch.float16, torch.float32):
        st = _inputs(B, T, V, dtype, 21)
        plain = _call(F, st, B, T)
        dev = {k: None if x is None else x.cuda() for k, x in st.items()}
        # target and drafter rows on different boundaries, nodes before rows, broadcast rows
        for pad in (1, 2, 3, 5):
            t = torch.zeros((T, B, V + pad), dtype=dtype, device="cuda")
            t[:, :, pad:] = dev["target"].transpose(0, 1)
            d = torch.zeros((B, T, V + 2 * pad), dtype=dtype, device="cuda")
            d[:, :, :V] = dev["draft"]
            got = _call(F, st, B, T, {**dev, "target": t[:, :, pad:].transpose(0, 1), "draft": d[:, :, :V]})
            for x, y in zip(got, plain):
                assert np.array_equal(x, y)
    st = _inputs(B, T, V, torch.float32, 22, root=False)
    st["n_nodes"][:] = torch.tensor([0, 1, 5, 0, 2, 9], dtype=torch.int32)
    st["n_nodes"] = st["n_nodes"].clamp(max=T)
    _compare(F, st, B, T, near=0.2)
    st["parents"][0, 0], st["parents"][2, 3] = 4, 3   # outside [0, i): read as -1
    _compare(F, st, B, T, near=0.2)


def test_nothing_is_left_of_equal_distributions(F):
    """p = q: every child is kept; made to be refused (u = 1), the token is drawn from p itself."""
    B, T, V = 4, 3, 300
    st = _inputs(B, T, V, torch.float32, 4, vary=False)
    st["draft"], st["draft_root"] = st["target"].clone(), st["target_root"].clone()
    st["parents"][:] = torch.tensor([-1, -1, -1])
    st["temperature"][:] = 1.0
    path, n_path, nxt = _call(F, st, B, T)
    assert (n_path == 1).all() and (path[:, 0] == 0).all()
    st["u"][:] = 1.0
    path, n_path, nxt = _call(F, st, B, T)
    p = torch.softmax(st["target_root"].double(), -1) / st["noise"].double()
    assert (n_path == 0).all() and np.array_equal(nxt, p.argmax(-1).numpy())


@pytest.mark.parametrize("mode", ["sampled", "certain"])
def test_tokens_are_distributed_as_the_targets(F, mode):
    """The first token that comes out (a kept child's, or the drawn one) over many runs: within six
    standard deviations of the target's probabilities."""
    B, T, V, runs = 256, 3, 6, 60
    g = torch.Generator(device="cuda").manual_seed(5)
    target = torch.tensor([1.0, 0.2, -1.0, 0.7, -math.inf, 2.0], device="cuda")
    draft = torch.tensor([0.0, 1.5, 0.5, -0.5, 0.3, 0.9], device="cuda")
    q = torch.softmax(draft, -1)
    one = lambda x: x.expand(B, V).contiguous()
    many = lambda x: x.expand(B, T, V)
    cfg = _cfg(F, B)
    parents = torch.full((B, T), -1, dtype=torch.int32, device="cuda")
    count = torch.zeros(V, dtype=torch.long, device="cuda")
    path = torch.zeros((B, T), dtype=torch.int32, device="cuda")
    n_path, nxt = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
    for _ in range(runs):
        if mode == "sampled":   # children drawn independently of each other
            tokens = torch.multinomial(q.expand(B * T, V), 1, generator=g).reshape(B, T).int()
        else:                   # any distinct ones
            tokens = torch.tensor([5, 1, 0], device="cuda").expand(B, T).contiguous().int()
        u = torch.rand((B, T), generator=g, device="cuda")
        noise = torch.empty((B, V), device="cuda").exponential_(generator=g)
        d = (many(draft), one(draft)) if mode == "sampled" else (None, None)
        F.fade_tree_verify(cfg, parents, None, tokens, many(target), one(target), *d, None, u, noise,
                           path, n_path, nxt)
        first = torch.where(n_path > 0, tokens.gather(1, path[:, :1].long())[:, 0], nxt)
        count += torch.bincount(first.long(), minlength=V)
    p = torch.softmax(target.double(), -1)
    N = B * runs
    off = (count.double() - N * p).abs()
    assert bool((off <= 6 * (N * p * (1 - p)).sqrt()).all()), (count.tolist(), (N * p).tolist())


def test_same_bits_and_graphs(F):
    B, T, V = 16, 8, 20000
    st = _inputs(B, T, V, torch.bfloat16, 31)
    d = {k: None if x is None else x.cuda() for k, x in st.items()}
    plain = _call(F, st, B, T, d)
    cfg = _cfg(F, B)
    outs, graphs = [], []
    for _ in range(2):
        path = torch.full((B, T), 77, dtype=torch.int32, device="cuda")
        n_path, nxt = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            F.fade_tree_verify(cfg, d["parents"], d["n_nodes"], d["tokens"], d["target"],
                               d["target_root"], d["draft"], d["draft_root"], d["temperature"],
                               d["u"], d["noise"], path, n_path, nxt)
        graphs.append(g)
        outs.append((path, n_path, nxt))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o in outs:
        for x, y in zip(o, plain):
            assert np.array_equal(x.cpu().numpy(), y)


@pytest.mark.parametrize("mode", ["sampled", "certain", "greedy"])
def test_largest_vocabulary(F, mode):
    """2^24 tokens: the last one is likeliest by far (probability 1 - 2^24 e^-40), is kept where it is the
    draft, and comes next where it is not."""
    B, T, V = 2, 1, 1 << 24
    target = torch.zeros((B, T + 1, V), dtype=torch.float16, device="cuda")
    target[:, :, -1] = 40
    d = dict(parents=torch.full((B, T), -1, dtype=torch.int32, device="cuda"), n_nodes=None,
             tokens=torch.tensor([[V - 1], [V // 2]], dtype=torch.int32, device="cuda"),
             target=target[:, 1:], target_root=target[:, 0],
             draft=target[:, 1:] if mode == "sampled" else None,
             draft_root=target[:, 0] if mode == "sampled" else None,
             temperature=None, u=None if mode == "greedy" else torch.full((B, T), 0.5, device="cuda"),
             noise=None if mode == "greedy" else torch.ones((B, V), device="cuda"))
    if mode == "sampled":   # the drafter's likeliest token is another one
        d["draft"], d["draft_root"] = d["draft"].clone(), d["draft_root"].clone()
        for x in (d["draft"], d["draft_root"]):
            x[1:, ..., V // 2], x[1:, ..., -1] = 40, 0
    path, n_path, nxt = _call(F, None, B, T, d)
    assert n_path.tolist() == [1, 0] and path[0, 0] == 0 and nxt.tolist() == [V - 1, V - 1]
