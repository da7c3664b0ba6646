"""Prompt attention and its column sums on a GPU against a plain implementation in 64 bits."""

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


def _cfg(F, B, hq, h, d):
    return F.Config(batch=B, num_q_heads=hq, num_kv_heads=h, head_dim=d, mid_capacity=64)


def _draw(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).half().cuda()


def _sees(q_len, kv_len, sink, window):
    """[queries][tokens] of one row."""
    pos = torch.arange(kv_len - q_len, kv_len, device="cuda")[:, None]
    j = torch.arange(kv_len, device="cuda")
    see = j <= pos
    if window:
        see &= (j > pos - window) | (j < sink)
    return see


def _reference(q, k, v, q_len, kv_len, sink, window):
    """float64 out, lse, mass and, for the bounds, sum p|v| and the largest sum |q||k| / sqrt(d)."""
    B, nq, hq, d = q.shape
    nk, h = k.shape[1], k.shape[2]
    out = torch.zeros((B, nq, hq, d), dtype=torch.float64, device="cuda")
    absv = torch.zeros_like(out)
    lse = torch.zeros((B, nq, hq), dtype=torch.float64, device="cuda")
    mass = torch.zeros((B, h, nk), dtype=torch.float64, device="cuda")
    big = 0.0
    for b in range(B):
        a, n = int(q_len[b]), int(kv_len[b])
        if a == 0:
            continue
        see = _sees(a, n, sink, window)
        for x in range(hq):
            kk, vv = k[b, :n, x * h // hq].double(), v[b, :n, x * h // hq].double()
            qq = q[b, :a, x].double()
            s = torch.where(see, qq @ kk.T / math.sqrt(d), -math.inf)
            p = torch.softmax(s, -1)
            out[b, :a, x], absv[b, :a, x] = p @ vv, p @ vv.abs()
            lse[b, :a, x] = torch.logsumexp(s, -1)
            mass[b, x * h // hq, :n] += p.sum(0)
            big = max(big, float((qq.abs() @ kk.abs().T).max()) / math.sqrt(d))
    return out, lse, mass, absv, big


def _lens(B, q_len, kv_len, nq, nk):
    return (np.full(B, nq, np.int32) if q_len is None else np.asarray(q_len, np.int32),
            np.full(B, nk, np.int32) if kv_len is None else np.asarray(kv_len, np.int32))


def _check(F, cfg, q, k, v, q_len=None, kv_len=None, sink=0, window=0, ws=None):
    """Runs both calls on (q, k, v) and holds them to the reference. The bounds: a probability is off by
    half a step of fp16 (2^-11) where it meets V, and by what its fp32 logit is: the product's sum of
    d terms (8 roundings of 2^-23 of the terms' absolute sum: the tensor cores add 16 or more terms a
    step), its scaling and ex2 (2^-16 for |logit| up to 2^6, more in proportion); out rounds by 2^-11, or
    2^-25 near 0. Logits' errors reach lse as they are, and mass relative to each term; a term of mass
    below fp32's least normal number, 2^-126, may be flushed: that much a query row."""
    B, nq, hq, d = q.shape
    nk, h = k.shape[1], k.shape[2]
    out = torch.full((B, nq, hq, d), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((B, nq, hq), 7.0, device="cuda")
    mass = torch.full((B, h, nk), 7.0, device="cuda")
    see = dict(q_len=q_len, kv_len=kv_len, n_sink=sink, window=window, ws=ws)
    F.fade_prompt_attention(cfg, q, k, v, out, lse, **see)
    F.fade_prompt_mass(cfg, q, k, lse, mass, **see)
    torch.cuda.synchronize()
    ql, kl = _lens(B, q_len, kv_len, nq, nk)
    ro, rl, rm, absv, big = _reference(q, k, v, ql, kl, sink, window)
    logit = 8 * 2.0 ** -23 * big + 2.0 ** -16 * max(1.0, big / 64)
    for b in range(B):
        a = int(ql[b])
        assert bool((out[b, a:] == 7).all()) and bool((lse[b, a:] == 7).all())
        off = (out[b, :a].double() - ro[b, :a]).abs()
        bound = (2.0 ** -11 + 2 * logit) * absv[b, :a] + 2.0 ** -11 * ro[b, :a].abs() + 2.0 ** -25
        worst = float((off / bound).max()) if a else 0.0
        assert worst <= 1, f"row {b}: out off by {worst} bounds"
        off = (lse[b, :a].double() - rl[b, :a]).abs()
        assert bool((off <= logit + 2.0 ** -22 * rl[b, :a].abs()).all()), float(off.max())
        off = (mass[b].double() - rm[b]).abs()
        bound = rm[b] * (2 * logit + 2.0 ** -18) + nq * (hq // h) * 2.0 ** -126
        worst = float((off / bound).max())
        assert worst <= 1, f"row {b}: mass off by {worst} bounds"
    return out, lse, mass


CASES = [
    # B, hq, h, d, nq, nk, q_len, kv_len, sink, window
    (1, 2, 2, 64, 1, 1, None, None, 0, 0),
    (1, 8, 2, 64, 1, 130, None, None, 0, 0),
    (2, 16, 2, 128, 1, 1000, None, [1000, 3], 4, 300),
    (3, 4, 4, 128, 7, 129, [7, 0, 3], [129, 0, 100], 0, 0),
    (2, 8, 8, 64, 255, 257, [255, 200], [257, 200], 0, 0),
    (1, 4, 1, 128, 127, 127, None, None, 0, 0),
    (1, 8, 1, 64, 128, 128, None, None, 0, 1),
    (1, 8, 1, 128, 129, 129, None, None, 1, 2),
    (2, 2, 1, 64, 300, 700, [300, 299], [700, 299], 128, 129),
    (1, 4, 4, 128, 513, 513, None, None, 127, 127),
    (1, 1, 1, 64, 600, 600, None, None, 129, 128),
    (1, 4, 2, 128, 64, 1500, None, None, 200, 64),
    (2, 8, 2, 64, 400, 400, [400, 1], [400, 1], 5, 399),
    (2, 8, 2, 128, 400, 400, [0, 0], [0, 400], 5, 100),
    (1, 8, 4, 128, 50, 2000, None, None, 0, 0),
    (1, 16, 2, 128, 1000, 1000, None, None, 4, 260),
    (7, 32, 8, 64, 70, 190, [70, 1, 0, 64, 33, 70, 2], [190, 1, 9, 64, 190, 70, 129], 3, 65),
    (40, 8, 4, 128, 2, 150, None, None, 0, 0),
    (1, 32, 8, 128, 1100, 1100, None, None, 0, 0),
]


@pytest.mark.parametrize("case", CASES, ids=[str(c) for c in CASES])
def test_against_definition(F, case):
    B, hq, h, d, nq, nk, q_len, kv_len, sink, window = case
    q = _draw((B, nq, hq, d), 1, 1.5)
    k, v = _draw((B, nk, h, d), 2, 1.5), _draw((B, nk, h, d), 3)
    _check(F, _cfg(F, B, hq, h, d), q, k, v, q_len, kv_len, sink, window)


def test_strides_and_other_orders(F):
    """Slices of a fused projection, head-major prompts, a batch-last order, broadcast keys."""
    B, hq, h, d, n = 2, 8, 2, 64, 200
    cfg = _cfg(F, B, hq, h, d)
    fused = _draw((B, n, hq + 2 * h, d), 5)
    q, k, v = fused[:, :, :hq], fused[:, :, hq:hq + h], fused[:, :, hq + h:]
    plain = _check(F, cfg, q, k, v, sink=3, window=77)
    for order in ((0, 2, 1, 3), (1, 0, 2, 3), (2, 1, 0, 3)):
        q2, k2, v2 = (x.permute(order).contiguous().permute(np.argsort(order).tolist())
                      for x in (q, k, v))
        wide = torch.zeros((B, hq, n, 2 * d), dtype=torch.float16, device="cuda")
        out = wide[..., :d].transpose(1, 2)
        lse = torch.zeros((B, n, hq), device="cuda")
        F.fade_prompt_attention(cfg, q2, k2, v2, out, lse, n_sink=3, window=77)
        assert torch.equal(out, plain[0]) and torch.equal(lse, plain[1])
        assert bool((wide[..., d:] == 0).all())
    one = k[:1, :, :1]
    ex = one.expand(B, n, h, d)
    assert ex.stride(0) == 0 and ex.stride(2) == 0
    _check(F, cfg, q, ex, v, sink=3, window=77)
    _check(F, cfg, q[:1].expand(B, n, hq, d), k, ex)


def test_sharp_and_flat_logits(F):
    """Logits of thousands (a row is one token) and of zero (every token the same)."""
    B, hq, h, d, n = 1, 4, 2, 128, 300
    cfg = _cfg(F, B, hq, h, d)
    q, k, v = (_draw((B, n, x, d), 10 + x, 20.0) for x in (hq, h, h))
    _check(F, cfg, q, k, _draw((B, n, h, d), 3))
    _check(F, cfg, torch.zeros_like(q), k, v)
    # growing logits: the reference moves with every tile
    k2 = torch.ones_like(k) * torch.linspace(0, 30, n, device="cuda").half()[None, :, None, None]
    _check(F, cfg, torch.ones_like(q), k2, _draw((B, n, h, d), 3))
    _check(F, cfg, torch.ones_like(q), k2.flip(1), _draw((B, n, h, d), 3), sink=2, window=100)


@pytest.mark.parametrize("d,G,window,sink", [(64, 4, 0, 0), (128, 1, 100, 3), (128, 8, 200, 130),
                                             (64, 2, 64, 1)])
def test_what_is_not_seen_does_not_reach_the_output(F, d, G, window, sink):
    """Infinities and NaN past the rows' lengths, in later tokens and outside the window."""
    B, h, n = 2, 2, 700
    hq = G * h
    cfg = _cfg(F, B, hq, h, d)
    q, k, v = _draw((B, n, hq, d), 1), _draw((B, n, h, d), 2), _draw((B, n, h, d), 3)
    lens = np.array([n - 45, 301], np.int32)
    clean = _check(F, cfg, q, k, v, lens, lens, sink, window)
    q2, k2, v2 = q.clone(), k.clone(), v.clone()
    for b, a in enumerate(lens):
        q2[b, a:], k2[b, a:], v2[b, a:] = math.nan, math.nan, math.inf
    outs = [torch.full_like(clean[0], 7.0), torch.full_like(clean[1], 7.0), torch.empty_like(clean[2])]
    see = dict(q_len=lens, kv_len=lens, n_sink=sink, window=window)
    F.fade_prompt_attention(cfg, q2, k2, v2, outs[0], outs[1], **see)
    F.fade_prompt_mass(cfg, q2, k2, outs[1], outs[2], **see)
    for x, y in zip(outs, clean):
        assert torch.equal(x, y)
    # tokens of the rows: who does not see them keeps his bits, who sees them gets what they hold
    bad = {5: math.nan, 129: math.inf, 250: -math.inf, 500: math.nan}
    for j, x in bad.items():
        v2[:, j, :, 3] = x
        v2[:, j, 1, d - 1] = x
    out = torch.full_like(clean[0], 7.0)
    F.fade_prompt_attention(cfg, q2, k2, v2, out, None, **see)
    for b, a in enumerate(lens.tolist()):
        see_row = _sees(a, a, sink, window)
        want = clean[0][b, :a].clone()
        for i in range(a):
            hit = [x for j, x in bad.items() if j < a and bool(see_row[i, j])]
            if hit:
                y = math.nan if any(math.isnan(x) for x in hit) or len(set(hit)) > 1 else hit[0]
                want[i, :, 3] = y
                want[i, G:, d - 1] = y
        assert torch.equal(torch.nan_to_num(out[b, :a], 1e4, 2e4, -2e4),
                           torch.nan_to_num(want, 1e4, 2e4, -2e4))
    # keys: a logit of NaN or +inf makes the rows that see it NaN, and no other
    k2[0, 129, :, 0] = math.nan
    out = torch.full_like(clean[0], 7.0)
    F.fade_prompt_attention(cfg, q2, k2, v, out, None, **see)
    a = int(lens[0])
    hit = _sees(a, a, sink, window)[:, 129]
    assert bool(out[0, :a][hit].isnan().all())
    assert torch.equal(out[0, :a][~hit], clean[0][0, :a][~hit])
    assert torch.equal(out[1], clean[0][1])


def test_chunks_add_up_to_the_prompt(F):
    """A prompt in chunks: the same attention, and masses that accumulate to the prompt's."""
    B, hq, h, d, n = 2, 8, 2, 128, 900
    cfg = _cfg(F, B, hq, h, d)
    q, k, v = _draw((B, n, hq, d), 1), _draw((B, n, h, d), 2), _draw((B, n, h, d), 3)
    lens = np.array([900, 611], np.int32)
    out, lse, mass = _check(F, cfg, q, k, v, lens, lens, 4, 333)
    acc = torch.zeros_like(mass)
    for c0 in range(0, n, 256):
        c1 = min(n, c0 + 256)
        kl = np.minimum(lens, c1).astype(np.int32)
        ql = np.maximum(kl - c0, 0).astype(np.int32)
        o, l = torch.zeros_like(out[:, c0:c1]), torch.zeros((B, c1 - c0, hq), device="cuda")
        see = dict(q_len=ql, kv_len=kl, n_sink=4, window=333)
        F.fade_prompt_attention(cfg, q[:, c0:c1], k, v, o, l, **see)
        F.fade_prompt_mass(cfg, q[:, c0:c1], k, l, acc, accumulate=True, **see)
        for b in range(B):
            a = int(ql[b])
            # the same P up to their references: two roundings of each
            off = (o[b, :a].float() - out[b, c0:c0 + a].float()).abs()
            assert bool((off <= 2.0 ** -9 * 4).all())
            assert bool(((l[b, :a] - lse[b, c0:c0 + a]).abs() <= 2.0 ** -15).all())
    assert bool(((acc - mass).abs() <= 2.0 ** -14 * mass).all())


def test_mass_is_what_prefill_mass_computes(F):
    B, hq, h, d, n = 2, 8, 2, 64, 333
    cfg = _cfg(F, B, hq, h, d)
    q, k, v = _draw((B, hq, n, d), 1), _draw((B, h, n, d), 2), _draw((B, h, n, d), 3)
    lens = np.array([333, 100], np.int32)
    want = torch.empty((B, h, n), device="cuda")
    F.fade_prefill_mass(cfg, q, k, n, lens, want)
    mass = _check(F, cfg, q.transpose(1, 2), k.transpose(1, 2), v.transpose(1, 2), lens, lens)[2]
    assert bool(((mass - want).abs() <= 2.0 ** -14 * want).all())


def test_same_bits_streams_and_graphs(F):
    """The same bits on every run, on another stream, and in two graphs that are replayed at once."""
    B, hq, h, d, n = 1, 8, 2, 128, 500
    cfg = _cfg(F, B, hq, h, d)
    q, k, v = _draw((B, n, hq, d), 1), _draw((B, n, h, d), 2), _draw((B, n, h, d), 3)
    first = _check(F, cfg, q, k, v, sink=4, window=200)

    def call(ws):
        out, lse = torch.zeros_like(q), torch.zeros((B, n, hq), device="cuda")
        mass = torch.zeros((B, h, n), device="cuda")
        see = dict(n_sink=4, window=200, ws=ws)
        F.fade_prompt_attention(cfg, q, k, v, out, lse, **see)
        F.fade_prompt_mass(cfg, q, k, lse, mass, **see)
        return out, lse, mass

    ws = [torch.empty(F.fade_prompt_ws_bytes(cfg, n, n), dtype=torch.uint8, device="cuda")
          for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = call(ws[0])
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for w in ws:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = call(w)
        graphs.append((g, outs))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for (g, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for outs in (other, graphs[0][1], graphs[1][1]):
        for x, y in zip(outs, first):
            assert torch.equal(x, y)


def test_workspace_made_for_another_stream(F, monkeypatch):
    """A workspace that a call makes for itself is not given to the current stream while the call's own
    stream has yet to use it."""
    cfg, n = _cfg(F, 1, 8, 2, 64), 700
    q, k, v = _draw((1, n, 8, 64), 1), _draw((1, n, 2, 64), 2), _draw((1, n, 2, 64), 3)
    want, lse, mass = _check(F, cfg, q, k, v)[:3]
    out, lse2, mass2 = torch.zeros_like(q), torch.zeros_like(lse), torch.zeros_like(mass)
    made, empty = [], torch.empty

    def spy(*a, **kw):
        made.append(empty(*a, **kw))
        return made[-1]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    monkeypatch.setattr(torch, "empty", spy)
    ptrs = []
    for call in (lambda: F.fade_prompt_attention(cfg, q, k, v, out, lse2, stream=side),
                 lambda: F.fade_prompt_mass(cfg, q, k, lse2, mass2, stream=side)):
        call()
        ptrs.append(made[-1].data_ptr())
        made.clear()
    monkeypatch.undo()
    ours = [torch.empty(F.fade_prompt_ws_bytes(cfg, n, n), dtype=torch.uint8, device="cuda")
            for _ in range(4)]
    assert not set(ptrs) & {x.data_ptr() for x in ours}
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse2, lse) and torch.equal(mass2, mass)


def test_offsets_past_32_bits(F):
    """Tokens 2^25 elements apart: the last ones lie past 2^32 elements."""
    B, hq, h, d, n = 1, 2, 1, 64, 140
    far = 1 << 25
    flat = torch.empty(far * n, dtype=torch.float16, device="cuda")
    view = lambda at: flat[at:].as_strided((B, n, h, d), (far, far, d, 1))
    k, v = view(0), view(64)
    k.copy_(_draw((B, n, h, d), 2))
    v.copy_(_draw((B, n, h, d), 3))
    out = flat[128:].as_strided((B, n, hq, d), (far, far, d, 1))
    q = _draw((B, n, hq, d), 1)
    cfg = _cfg(F, B, hq, h, d)
    want = _check(F, cfg, q, k, v)[0]
    F.fade_prompt_attention(cfg, q, k, v, out, None)
    assert torch.equal(out, want)
