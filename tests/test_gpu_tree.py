"""Drafted-token operators on the GPU against plain 64-bit implementations.

Tolerances count roundings. u = 2^-11 is half a step of fp16 relative to the value, 2^-24 of fp32.
Attention: a middle key is fp16 plus the remainder of its rounding (at most u |k|), which meets the
query rounded to E5M2 (off by |q| / 8, or half a subnormal step, 2^-17), so a logit moves by at most
delta = u * scale * sum_c |k_c| (|q_c| / 8 + 2^-17); the softmax then moves every probability by a
factor within e^(+-2 delta); probabilities and dequantised values round to fp16 once each (u each),
the output once (u |out|); a probability's rounding is off by half a subnormal step, 2^-25, at
least, where the largest one is held as 2^6 or more: 2^-31 of the largest, sum |v| times over the
sum of e; fp32 sums over d channels and N tokens add (N + d) 2^-24, the fast exponential and
logarithm 2^-20; the scaled logit's own fp32 rounding 2^-23 of the largest.
Scores: the codes enter the products exactly; sums over d channels, the group's scale, the offset
and the exponential round in fp32.
"""

import numpy as np
import pytest
import torch

from oracle import pq, quant

pytestmark = pytest.mark.gpu

U = 2.0 ** -11


@pytest.fixture(scope="module")
def F():
    from tiered_mixed_precision_gb300 import build

    build.build()
    from tiered_mixed_precision_gb300 import fade as F

    return F


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def random_parents(rng, B, T, kind="tree"):
    if kind == "chain":
        return np.tile(np.arange(T, dtype=np.int32) - 1, (B, 1))
    if kind == "flat":
        return np.full((B, T), -1, np.int32)
    p = np.full((B, T), -1, np.int32)
    for i in range(1, T):
        p[:, i] = rng.integers(-1, i, B)
    return p


def plain_layout(parents, n):
    """Ancestor sets as a bool [T][T] and depths, by walking up the parents."""
    T = len(parents)
    see, depth = np.zeros((T, T), bool), np.zeros(T, int)
    for i in range(n):
        j = i
        while True:
            see[i, j] = True
            p = parents[j]
            if not 0 <= p < j:
                break
            depth[i] += 1
            j = p
    return see, depth


def mask_words(see):
    """bool [B][T][T] -> i64 [B][T]"""
    w = (see.astype(np.uint64) << np.arange(see.shape[-1], dtype=np.uint64)).sum(-1, dtype=np.uint64)
    return w.view(np.int64)


# --------------------------------------------------------------------------- layout
@pytest.mark.parametrize("B,T,kind", [(1, 1, "tree"), (3, 2, "chain"), (2, 64, "chain"),
                                      (5, 64, "tree"), (256, 33, "tree"), (2, 17, "flat")])
@pytest.mark.parametrize("ragged", [False, True])
def test_layout(F, B, T, kind, ragged):
    rng = np.random.default_rng(B * 100 + T)
    par = random_parents(rng, B, T, kind)
    if T > 4:   # what is no lower index is a root
        par[0, 2], par[0, 3], par[B - 1, 4] = 2, 60000, -7
    n = rng.integers(0, T + 1, B).astype(np.int32) if ragged else None
    if ragged:
        n[0] = T + 5    # clamped
    base = rng.integers(0, 1 << 20, B).astype(np.int32)
    cfg = F.Config(batch=B, num_q_heads=4, num_kv_heads=1, head_dim=64, mid_capacity=16)
    mask = torch.full((B, T), -1, dtype=torch.int64, device="cuda")
    pos = torch.full((B, T), -1, dtype=torch.int32, device="cuda")
    F.fade_tree_layout(cfg, dev(par), None if n is None else dev(n), dev(base), mask, pos)
    for b in range(B):
        nb = T if n is None else min(int(n[b]), T)
        see, depth = plain_layout(par[b], nb)
        assert np.array_equal(mask[b].cpu().numpy(), mask_words(see)), b
        assert np.array_equal(pos[b].cpu().numpy(), base[b] + depth), b


# --------------------------------------------------------------------------- norm + rotation
def norm_reference(x, w, eps, table, pos, r):
    """x [n][t][heads][d] fp16, table [max_pos][d/4][4] -> (fp64 result, error bound)."""
    x = x.astype(np.float64)
    d = x.shape[-1]
    y = x if w is None else (x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
                             * w.astype(np.float64))
    a, b = y[..., :r // 2], y[..., r // 2:r]
    rows = table[pos][..., :r // 4, :].astype(np.float64)
    c = rows[..., 0:2].reshape(*pos.shape, 1, r // 2)
    s = rows[..., 2:4].reshape(*pos.shape, 1, r // 2)
    out = np.concatenate([a * c - b * s, b * c + a * s, y[..., r:]], -1)
    mag = np.abs(y)
    pair = np.abs(a) + np.abs(b)
    mag = np.concatenate([pair, pair, mag[..., r:]], -1)
    # one rounding to fp16 (half a subnormal step at least) after at most d/8 + 16 fp32 roundings
    return out, U * np.abs(out) + 2.0 ** -25 + (d / 8 + 16) * 2.0 ** -24 * mag * (1 + U)


@pytest.mark.parametrize("d,heads,rows,tokens,rotary,weights,layout", [
    (128, (16, 2), 1, 1, 0, "both", "fused"),
    (64, (8, 8), 2, 3, 0, "both", "tokens"),
    (128, (32, 8), 3, 37, 0, "both", "heads"),
    (128, (8, 1), 2, 513, 96, "both", "fused"),
    (64, (4, 2), 5, 7, 4, "q", "tokens"),
    (64, (1, 1), 1, 5000, 44, "k", "heads"),
    (128, (4, 4), 2, 2, 124, "none", "tokens"),
    (128, (32, 8), 64, 16, 0, "both", "in place"),
])
def test_norm(F, d, heads, rows, tokens, rotary, weights, layout):
    rng = np.random.default_rng(d + tokens)
    hq, h = heads
    maxpos = 5003
    cfg = F.Config(batch=1, num_q_heads=hq, num_kv_heads=h, head_dim=d, mid_capacity=16,
                   rope_rotary_dim=rotary)
    table = torch.zeros(maxpos * d, device="cuda")
    F.fade_rope_table_init(cfg, table, maxpos)
    x = rng.standard_normal((rows, tokens, hq + 2 * h, d)).astype(np.float16)
    x[0, 0, 0] = 0                           # a vector of zeros
    x[-1, -1, hq] = 6e4                      # squares past fp16
    x[0, -1, hq - 1] *= np.float16(2e-6)     # subnormal channels
    gx = dev(x)
    if layout == "heads":
        q = gx[:, :, :hq].transpose(1, 2).contiguous().transpose(1, 2)
        k = gx[:, :, hq:hq + h].transpose(1, 2).contiguous().transpose(1, 2)
    elif layout == "tokens":
        q, k = gx[:, :, :hq].contiguous(), gx[:, :, hq:hq + h].contiguous()
    else:
        q, k = gx[:, :, :hq], gx[:, :, hq:hq + h]
    w = [(1 + 0.3 * rng.standard_normal(d)).astype(np.float16) for _ in range(2)]
    qw = w[0] if weights in ("both", "q") else None
    kw = w[1] if weights in ("both", "k") else None
    pos = rng.integers(0, maxpos, (rows, tokens)).astype(np.int32)
    pos[0, 0], pos[-1, -1] = -3, maxpos + 9   # clamped
    if layout == "in place":
        qo, ko = q, k
    else:
        qo = torch.empty((rows, tokens, hq, d), dtype=torch.float16, device="cuda")
        ko = torch.empty((rows, h, tokens, d), dtype=torch.float16, device="cuda").transpose(1, 2)
    opt = lambda a: None if a is None else dev(a)
    F.fade_qk_norm_rope(cfg, table, maxpos, q, k, opt(qw), opt(kw), 1e-6, dev(pos), qo, ko)
    tab = table.cpu().numpy().reshape(maxpos, d // 4, 4)
    cl = np.clip(pos, 0, maxpos - 1)
    for got, src, ww in ((qo, x[:, :, :hq], qw), (ko, x[:, :, hq:hq + h], kw)):
        ref, tol = norm_reference(src, ww, 1e-6, tab, cl, rotary or d)
        err = np.abs(got.double().cpu().numpy() - ref)
        fits = np.abs(ref) + tol < 65504
        assert (err[fits] <= tol[fits]).all(), float((err - tol)[fits].max())
    if layout in ("fused", "in place"):   # the projection's v is not touched
        assert torch.equal(gx[:, :, hq + h:].cpu(), torch.from_numpy(x[:, :, hq + h:]))


def test_norm_without_weights_is_rope_apply(F):
    """No weights: bit for bit the rotation fade_rope_apply makes, and a copy without RoPE."""
    for kind in ("llama3", "none"):
        cfg = F.Config(batch=3, num_q_heads=8, num_kv_heads=2, head_dim=128, mid_capacity=16,
                       rope_kind=kind, rope_factor=8.0)
        table = torch.zeros(400 * 128, device="cuda")
        if kind != "none":
            F.fade_rope_table_init(cfg, table, 400)
        q = torch.randn((3, 1, 8, 128), device="cuda").half()
        pos = torch.tensor([[0], [399], [77]], dtype=torch.int32, device="cuda")
        got, want = torch.empty_like(q), torch.empty_like(q)
        F.fade_qk_norm_rope(cfg, table, 400, q, None, None, None, 1.0, pos, got, None)
        F.fade_rope_apply(cfg, table, 400, q, want, 3, 8, pos, 0)
        assert torch.equal(got, want)


# --------------------------------------------------------------------------- attention
class Cache:
    """One layer with random contents in cache order, and its tiers on the host."""

    def __init__(self, F, rng, B, hq, h, d, lens, S=4, W=64, rec=None, kb=4, vb=2, codec="int",
                 policy="none", extra=70, scale=1.0, decay=0.9, shared=False, budget=None):
        self.F = F
        mid = [max(0, n - S - (W if rec is None else rec)) for n in lens]
        evicts = policy != "none"
        budget = max(mid) if budget is None else budget
        self.cfg = F.Config(batch=B, num_q_heads=hq, num_kv_heads=h, head_dim=d, n_sink=S,
                            recent_window=W, int4_budget=budget if evicts else -1,
                            middle_k_bits=kb, middle_v_bits=vb, mid_capacity=max(mid) + extra,
                            policy=policy, rope_kind="none", v_codec=codec, ema_decay=decay,
                            shared_rows=shared)
        self.L = L = F.TieredLayer(self.cfg, max(1, max(lens)), "cuda")
        self.cb = None
        if codec == "pq":
            self.cb = (scale * rng.standard_normal((d // 4, 256, 4))).astype(np.float16)
            L.set_pq_codebook(dev(self.cb))
        P = max(1, max(lens))
        k = (scale * rng.standard_normal((B, h, P, d))).astype(np.float16)
        k[..., 3] *= 4
        v = (scale * rng.standard_normal((B, h, P, d))).astype(np.float16)
        mass = dev(rng.random((B, h, P)).astype(np.float32)) if policy == "h2o" else None
        F.fade_cache_reset(L)
        F.fade_cache_prefill(L, dev(k), dev(v), P, lens, mass, None, 0)

    def unit(self, b, h):
        """(n_sink, n_mid, n_recent, keys, values, scores) of a unit, cache order, float64."""
        L, c = self.L, self.cfg
        m = L.meta[b, h].cpu().numpy()
        ns, nm, nr, head, cur = (int(x) for x in m[:5])
        ring = [(head + i) % c.recent_window for i in range(nr)]
        g = lambda t: t[b, h].cpu().numpy()
        kq = quant.unpack(g(L.mid_k_codes[cur])[:nm], c.middle_k_bits)
        mk = quant.dequantize(kq, g(L.mid_k_scales[cur])[:nm])
        vc = g(L.mid_v_codes[cur])[:nm]
        if self.cb is not None:
            mv = pq.decode(vc, self.cb).astype(np.float64)
        else:
            mv = quant.dequantize(quant.unpack(vc, c.middle_v_bits), g(L.mid_v_scales[cur])[:nm])
        cat = lambda s, x, r: np.concatenate([s[:ns].astype(np.float64), x,
                                              r[ring].astype(np.float64)])
        return (ns, nm, nr, cat(g(L.sink_k), mk, g(L.recent_k)),
                cat(g(L.sink_v), mv, g(L.recent_v)),
                np.concatenate([g(L.sink_scores)[:ns], g(L.mid_scores[cur])[:nm],
                                g(L.recent_scores)[ring]]))

    def draft(self, rng, T, scale=1.0, fused=True):
        c = self.cfg
        B, hq, h, d = c.batch, c.num_q_heads, c.num_kv_heads, c.head_dim
        self.q = (scale * rng.standard_normal((B, T, hq, d))).astype(np.float16)
        self.tk = rng.standard_normal((B, T, h, d)).astype(np.float16)
        self.tv = rng.standard_normal((B, T, h, d)).astype(np.float16)
        self.dq = dev(self.q)
        self.out = torch.full(self.q.shape, 7.0, dtype=torch.float16, device="cuda")
        self.lse = torch.full(self.q.shape[:3], 7.0, device="cuda")
        self.ws = torch.full((self.F.fade_tree_ws_bytes(c, T),), 0xff, dtype=torch.uint8,
                             device="cuda")   # NaN patterns: nothing is read before it is written
        self.fused = fused
        self.load_tree()

    def load_tree(self):
        if self.fused:   # slices of a projection, token-major, and a head-major tensor
            x = torch.zeros((*self.tk.shape[:2], 3 * self.tk.shape[2], self.tk.shape[3]),
                            dtype=torch.float16, device="cuda")
            self.dk = x[:, :, self.tk.shape[2]:2 * self.tk.shape[2]]
            self.dk.copy_(dev(self.tk))
            self.dv = dev(self.tv.transpose(0, 2, 1, 3)).transpose(1, 2)
        else:
            self.dk, self.dv = dev(self.tk), dev(self.tv)

    def attend(self, see, n_nodes=None):
        self.F.fade_tree_attention(self.L, self.dq, self.dk, self.dv, dev(mask_words(see)),
                                   None if n_nodes is None else dev(n_nodes), self.out, self.lse,
                                   self.ws)
        return self.out.double().cpu().numpy(), self.lse.double().cpu().numpy()

    def check(self, see, n_nodes=None, rows=None):
        """Every node of every row, or of the rows given."""
        out, lse = self.attend(see, n_nodes)
        c = self.cfg
        G = c.num_q_heads // c.num_kv_heads
        for b in range(c.batch) if rows is None else rows:
            n = see.shape[1] if n_nodes is None else int(n_nodes[b])
            assert (out[b, n:] == 7).all() and (lse[b, n:] == 7).all()
            for h in range(c.num_kv_heads):
                _, _, _, K, V, _ = self.unit(b, h)
                for i in range(n):
                    js = np.nonzero(see[b, i, :n])[0]
                    k = np.concatenate([K, self.tk[b, js, h].astype(np.float64)])
                    v = np.concatenate([V, self.tv[b, js, h].astype(np.float64)])
                    for g in range(G):
                        o, l = out[b, i, h * G + g], lse[b, i, h * G + g]
                        compare(o, l, self.q[b, i, h * G + g].astype(np.float64), k, v,
                                (b, i, h, g))
        self.F.fade_check_status(self.L)


def compare(o, l, q, k, v, where):
    if not len(k):
        assert (o == 0).all() and l == -np.inf, where
        return
    d = len(q)
    scale = 1 / np.sqrt(d)
    s = k @ q * scale
    m = s.max()
    e = np.exp(s - m)
    p = e / e.sum()
    ref, ref_l = p @ v, m + np.log(e.sum())
    delta = U * scale * (np.abs(k) @ (np.abs(q) / 8 + 2.0 ** -17)).max() \
        + 2.0 ** -23 * np.abs(s).max()
    sums = (len(k) + d) * 2.0 ** -24 + 2.0 ** -20
    tol = (np.expm1(2 * delta) + 2 * U + sums) * (p @ np.abs(v)) * (1 + U) + U * np.abs(ref) \
        + 2.0 ** -25 + 2.0 ** -31 / e.sum() * np.abs(v).sum(0)
    assert (np.abs(o - ref) <= tol).all(), (where, float((np.abs(o - ref) / tol).max()))
    assert abs(l - ref_l) <= delta + sums + 2.0 ** -22 * abs(ref_l), (where, l, ref_l)


CASES = [
    # B, hq, h, d, lens, T, kind, options
    (1, 8, 2, 64, [511], 4, "chain", {}),
    (2, 16, 2, 128, [701, 64], 16, "tree", dict(vb=4)),
    (1, 4, 4, 64, [300], 1, "chain", dict(kb=2)),
    (3, 8, 1, 128, [0, 1, 5], 9, "tree", {}),                     # empty and sink-only rows
    (2, 4, 1, 64, [130, 200], 64, "tree", dict(codec="pq")),
    (1, 8, 1, 128, [900], 64, "tree", dict(codec="pq", kb=2)),     # 512 query rows
    (1, 16, 8, 128, [196], 33, "tree", dict(kb=2, vb=4)),
    (2, 4, 2, 64, [193, 333], 25, "flat", dict(vb=4)),
    (1, 2, 1, 128, [2500], 64, "chain", dict(kb=2, vb=2)),
    (2, 2, 2, 128, [70, 199], 7, "tree", dict(S=0, W=1)),
    (1, 4, 1, 64, [400], 12, "tree", dict(S=130, W=200)),          # more FP16 tokens than a tile
    (4, 32, 8, 128, [1030, 517, 1028, 69], 16, "tree", {}),
]


@pytest.mark.parametrize("B,hq,h,d,lens,T,kind,opt", CASES)
@pytest.mark.parametrize("ragged", [False, True])
def test_attention(F, B, hq, h, d, lens, T, kind, opt, ragged):
    rng = np.random.default_rng(sum(lens) + T)
    c = Cache(F, rng, B, hq, h, d, lens, **opt)
    c.draft(rng, T, fused=ragged)
    n = rng.integers(0, T + 1, B).astype(np.int32) if ragged else np.full(B, T, np.int32)
    n[B - 1] = T
    par = random_parents(rng, B, T, kind)
    see = np.stack([plain_layout(par[b], T)[0] for b in range(B)])
    if ragged:
        see[:, 0, :] = False     # a node that sees no node, itself included
        see[:, :, T - 1] = True  # bits past a row's nodes (where it has fewer) are ignored
        for b in range(B):       # what the padding holds does not matter
            c.tk[b, n[b]:] = np.nan
            c.tv[b, n[b]:] = np.inf
            c.q[b, n[b]:] = np.nan
        c.dq = dev(c.q)
        c.load_tree()
    c.check(see, n if ragged else None)


@pytest.mark.parametrize("B,hq,h,d,T,lens,opt", [
    (40, 8, 8, 128, 16, (60, 400), {}),                        # a few blocks of query rows a CTA
    (256, 8, 4, 64, 5, (0, 75), dict(kb=2)),                   # many one-tile blocks a CTA
    (12, 64, 8, 64, 64, (100, 300), dict(codec="pq")),         # four blocks of rows a unit
    (64, 16, 8, 128, 13, (64, 330), dict(codec="pq")),
])
def test_many_short_blocks(F, B, hq, h, d, T, lens, opt):
    """CTAs that take many blocks of query rows one after another, ragged rows among them some
    without nodes."""
    rng = np.random.default_rng(B)
    held = rng.integers(lens[0], lens[1] + 1, B).tolist()
    c = Cache(F, rng, B, hq, h, d, held, **opt)
    c.draft(rng, T)
    n = rng.integers(0, T + 1, B).astype(np.int32)
    n[0], n[B - 1] = 0, T
    see = np.stack([plain_layout(p, T)[0] for p in random_parents(rng, B, T)])
    c.check(see, n, sorted({0, 1, B // 3, B // 2, B - 2, B - 1}))
    first = c.out.clone(), c.lse.clone()
    for _ in range(3):
        c.attend(see, n)
        assert torch.equal(c.out, first[0]) and torch.equal(c.lse, first[1])


def test_more_blocks_than_one_cta_each_can_list(F):
    """24576 blocks of query rows: the grid grows past one CTA a multiprocessor."""
    rng = np.random.default_rng(8)
    B, hq, h, d, T = 256, 256, 32, 64, 33
    c = Cache(F, rng, B, hq, h, d, [9] * B, W=8)
    c.draft(rng, 1)
    g = torch.Generator("cuda").manual_seed(3)
    q, k, v = (torch.randn(s, generator=g, device="cuda", dtype=torch.float16)
               for s in ((B, T, hq, d), (B, T, h, d), (B, T, h, d)))
    out, lse = torch.full_like(q, 7.0), torch.full((B, T, hq), 7.0, device="cuda")
    ws = torch.empty(F.fade_tree_ws_bytes(c.cfg, T), dtype=torch.uint8, device="cuda")
    see = plain_layout(random_parents(rng, 1, T)[0], T)[0]
    F.fade_tree_attention(c.L, q, k, v, dev(np.tile(mask_words(see[None]), (B, 1))), None, out,
                          lse, ws)
    F.fade_check_status(c.L)
    host = lambda t: t.double().cpu().numpy()
    for b in [0, 255, *rng.integers(0, B, 10)]:
        for u in rng.integers(0, h, 2):
            K, V = c.unit(b, u)[3:5]
            tk, tv = host(k[b, :, u]), host(v[b, :, u])
            for i in {0, 32, int(rng.integers(T))}:
                a = u * 8 + int(rng.integers(8))
                js = np.nonzero(see[i])[0]
                compare(host(out[b, i, a]), float(lse[b, i, a]), host(q[b, i, a]),
                        np.concatenate([K, tk[js]]), np.concatenate([V, tv[js]]), (b, u, i, a))


@pytest.mark.parametrize("hq,h,T,long,pattern", [
    (32, 8, 16, 16384, "L" * 32 + "s" * 32),                 # the short rows behind the long ones
    (16, 2, 64, 131000, ("L" + "s" * 40) * 2 + "L"),         # 512 query rows a unit, long between short
    (8, 8, 5, 30000, "s" * 50 + "L" + "s" * 77 + "LL"),
])
def test_short_rows_beside_long_ones(F, hq, h, T, long, pattern):
    """CTAs take equal tiles, so beside long rows some take hundreds of one-tile blocks: every block
    of the short rows is written, and by the 64-bit form."""
    rng = np.random.default_rng(len(pattern))
    B, d = len(pattern), 64
    c = Cache(F, rng, B, hq, h, d, [60] * B, extra=long)
    rows = [b for b in range(B) if pattern[b] == "L"]
    fill_middle(c, rows, long)
    c.draft(rng, T)
    n = rng.integers(max(1, T // 2), T + 1, B).astype(np.int32)
    see = np.stack([plain_layout(p, T)[0] for p in random_parents(rng, B, T)])
    out, lse = c.attend(see, n)
    for b in range(B):   # every block is written
        assert not (out[b, :n[b]] == 7).all(-1).any() and not (lse[b, :n[b]] == 7).any(), b
    some = [b for b in range(B) if pattern[b] == "s"]
    c.check(see, n, some if T * hq * len(some) <= 1 << 14 else some[::6])
    first = c.out.clone(), c.lse.clone()
    # the long rows, against the same rows by themselves
    few = Cache(F, rng, len(rows), hq, h, d, [60] * len(rows), extra=long)
    for name in ("sink_k", "sink_v", "recent_k", "recent_v", "meta"):
        getattr(few.L, name).copy_(getattr(c.L, name)[rows])
    cur = int(c.L.meta[0, 0, 4])
    for name in ("mid_k_codes", "mid_v_codes", "mid_k_scales", "mid_v_scales"):
        getattr(few.L, name)[cur].copy_(getattr(c.L, name)[cur][rows])
    few.draft(rng, T)
    few.dq, few.dk, few.dv = c.dq[rows], c.dk[rows].contiguous(), c.dv[rows].contiguous()
    want, want_lse = few.attend(see[rows], n[rows])
    for i, b in enumerate(rows):
        # other cuts of the tiles, so other references: every probability rounds anew (U, and |v| of
        # the middle tokens is below 1), as does the output; sums of 32 terms a thread and tile, of 1024
        # tiles, of 152 partials and their exponentials round in fp32
        w, wl = want[i, :n[b]], want_lse[i, :n[b]]
        assert np.abs(out[b, :n[b]] - w).max() <= 3 * U * (1 + np.abs(w).max())
        assert np.abs(lse[b, :n[b]] - wl).max() <= 2 * (1300 * 2.0 ** -24 + 2.0 ** -20)
    c.attend(see, n)
    assert torch.equal(c.out, first[0]) and torch.equal(c.lse, first[1])
    c.out.fill_(7), c.lse.fill_(7)
    one = np.zeros(B, np.int32)
    one[rows[0]] = 1
    c.check(see, one, rows[:1])


def fill_middle(c, rows, n_mid):
    """Random codes and scales in the middle tiers of rows, n_mid tokens each."""
    L, cfg = c.L, c.cfg
    g = torch.Generator("cuda").manual_seed(n_mid)
    cur = int(L.meta[0, 0, 4])
    for b in rows:
        for codes, scales, bits in ((L.mid_k_codes, L.mid_k_scales, cfg.middle_k_bits),
                                    (L.mid_v_codes, L.mid_v_scales, cfg.middle_v_bits)):
            x, q = codes[cur][b, :, :n_mid], 2 ** (bits - 1) - 1
            w = torch.zeros(x.shape, dtype=torch.int32, device="cuda")
            for i in range(8 // bits):
                code = torch.randint(-q, q + 1, x.shape, generator=g, device="cuda", dtype=torch.int32)
                w |= (code & ((1 << bits) - 1)) << (bits * i)
            x.copy_(w)
            s = scales[cur][b, :, :n_mid]
            s.copy_(torch.rand(s.shape, generator=g, device="cuda") / q)
        L.meta[b, :, c.F.META["n_mid"]] = n_mid
        L.h_n_mid[b] = n_mid


def test_offsets_past_32_bits(F):
    """A capacity whose codes lie past 4 GiB: attention and commit of the last rows."""
    rng = np.random.default_rng(32)
    B, hq, h, d, T = 64, 8, 8, 128, 6
    c = Cache(F, rng, B, hq, h, d, [300] * B, extra=131072 - 232, policy="h2o", budget=131071)
    assert c.L.mid_k_codes[0].numel() >= 1 << 32
    c.draft(rng, T)
    par = np.tile(np.arange(T, dtype=np.int32) - 1, (B, 1))
    see = np.stack([plain_layout(p, T)[0] for p in par])
    c.check(see, None, [0, B - 1])
    before = c.unit(B - 1, h - 1)
    lse = c.lse.double().cpu().numpy()
    path = np.tile(np.arange(T, dtype=np.int32), (B, 1))
    F.fade_tree_commit(c.L, c.dq, c.lse, c.dk, c.dv, dev(path), [T] * B, c.ws)
    F.fade_check_status(c.L)
    now = c.unit(B - 1, h - 1)
    assert now[:3] == (4, 238, 64)
    want, tol = scores_reference(c, B - 1, h - 1, 1, before[3], before[5], path[B - 1], lse, "h2o")
    assert (np.abs(now[5] - want) <= tol).all()
    assert np.array_equal(now[3][:236], before[3][:236])   # what was in the tiers stays


def test_nodes_keys_and_values_of_any_stride(F):
    """Expanded (stride 0), reversed-layout and padded keys and values: the bits of contiguous
    ones."""
    rng = np.random.default_rng(6)
    B, hq, h, d, T = 3, 8, 4, 64, 9
    c = Cache(F, rng, B, hq, h, d, [200, 90, 3], policy="h2o")
    c.draft(rng, T, fused=False)
    see = np.stack([plain_layout(p, T)[0] for p in random_parents(rng, B, T)])
    for k, v in ((c.dk[:1].expand(B, T, h, d), c.dv[:, :1].expand(B, T, h, d)),
                 (c.dk[:, :, :1].expand(B, T, h, d), c.dv.permute(2, 1, 0, 3).contiguous()
                  .permute(2, 1, 0, 3)),
                 (torch.nn.functional.pad(c.dk, (0, 8))[..., :d],
                  torch.nn.functional.pad(c.dv, (16, 8))[..., 16:16 + d])):
        c.dk, c.dv = k.contiguous(), v.contiguous()
        c.attend(see)
        want = c.out.clone(), c.lse.clone()
        c.dk, c.dv = k, v
        c.attend(see)
        assert torch.equal(c.out, want[0]) and torch.equal(c.lse, want[1])
        c.dk, c.dv = dev(c.tk), dev(c.tv)


def test_attention_of_an_empty_cache_with_nodes_that_see_nothing(F):
    rng = np.random.default_rng(5)
    c = Cache(F, rng, 2, 8, 2, 64, [0, 0])
    c.draft(rng, 6)
    see = np.stack([plain_layout(np.arange(6) - 1, 6)[0]] * 2)
    see[0, 2] = see[1, 5] = False
    c.check(see)


@pytest.mark.parametrize("d,codec", [(64, "int"), (128, "int"), (128, "pq")])
def test_what_a_node_does_not_see_does_not_reach_it(F, d, codec):
    """Infinities and NaN in the keys and values of other branches leave a node's bits alone; a
    node that sees them is not finite."""
    rng = np.random.default_rng(d)
    c = Cache(F, rng, 1, 8, 2, d, [300], codec=codec)
    T = 12
    c.draft(rng, T)
    par = np.array([-1, 0, 1, 2, 3, -1, 5, 6, 7, 8, 9, 10])   # two branches
    see = plain_layout(par, T)[0][None]
    c.check(see)
    clean = c.out.clone(), c.lse.clone()
    c.tv[0, 6, :, 5], c.tv[0, 7, :, 9], c.tk[0, 8] = np.inf, np.nan, np.nan
    c.load_tree()
    c.attend(see)
    assert torch.equal(c.out[:, :6], clean[0][:, :6]) and torch.equal(c.lse[:, :6], clean[1][:, :6])
    o = c.out.float().cpu().numpy()
    for node in (6, 7):
        assert not np.isfinite(o[0, node, :, 5]).any()
    assert np.isfinite(o[0, 6, :, 9]).all() and np.isnan(o[0, 7, :, 9]).all()
    assert np.isnan(o[0, 8:]).all()


@pytest.mark.parametrize("lens", [[300], [6000], [0]])
def test_a_query_that_is_not_a_number_gives_none(F, lens):
    """NaN in a query row: NaN and a NaN lse in that row, not the zeros of a row that sees nothing; the
    other rows' bits stay. NaN in a cached key: in every row."""
    rng = np.random.default_rng(17)
    c = Cache(F, rng, 1, 8, 2, 64, lens)
    T = 6
    c.draft(rng, T)
    see = np.tril(np.ones((1, T, T), bool))
    c.check(see)
    clean, clean_lse = c.out.clone(), c.lse.clone()
    c.dq[0, 2, 5, 9], c.dq[0, 4, 1] = float("nan"), float("nan")
    c.attend(see)
    assert torch.isnan(c.out[0, 2, 5]).all() and torch.isnan(c.lse[0, 2, 5])
    assert torch.isnan(c.out[0, 4, 1]).all() and torch.isnan(c.lse[0, 4, 1])
    rest = torch.ones(1, T, 8, dtype=torch.bool, device="cuda")
    rest[0, 2, 5] = rest[0, 4, 1] = False
    assert torch.equal(c.out[rest], clean[rest]) and torch.equal(c.lse[rest], clean_lse[rest])
    c.dq = dev(c.q)
    if lens[0]:
        c.L.sink_k[0, 1, 0, 3] = float("nan")
        c.attend(see)
        assert torch.equal(c.out[:, :, :4], clean[:, :, :4])
        assert torch.isnan(c.out[:, :, 4:]).all() and torch.isnan(c.lse[:, :, 4:]).all()


def test_large_logits_and_extreme_scales(F):
    """Logits hundreds apart (the running maximum moves by whole exponents), keys near fp16's
    largest value and values among its smallest."""
    rng = np.random.default_rng(11)
    c = Cache(F, rng, 1, 4, 1, 64, [600])
    c.draft(rng, 8, scale=8.0)
    see = np.tril(np.ones((1, 8, 8), bool))
    c.check(see)
    c = Cache(F, rng, 1, 4, 1, 128, [400], scale=1.0)
    L = c.L
    cur = int(L.meta[0, 0, 4])
    L.mid_k_scales[cur][:, :, 7] = 9360.0
    L.mid_k_codes[cur][:, :, 7] = 0x77
    L.mid_v_scales[cur][:, :, 9] = 65504.0
    L.mid_v_scales[cur][:, :, 11:200] = 2.0 ** -24
    c.draft(rng, 8, scale=2.0 ** -12)
    c.check(see)


def key_error(K, s):
    """How far a middle INT4 key of scale s may be from code * scale: nothing from 2^-5 on (fp16 and an
    E5M2 remainder hold its 14 bits), else what lies under E5M2's last bit, 2^-16 of a halved key and
    never more than the remainder itself, and half of fp16's last bit for a halved key, 2^-25."""
    return np.zeros_like(K) if s >= 2.0 ** -5 else np.minimum(U * np.abs(K), 2.0 ** -15) + 2.0 ** -24


@pytest.mark.parametrize("d,kb", [(64, 4), (128, 4), (64, 2)])
@pytest.mark.parametrize("exp", [-20, -14, -13, -10, -7, -5, -2, 4, 13])
def test_keys_of_every_scale(F, d, kb, exp):
    """Middle keys whose fp16 roundings all fall to the same side, queries that make logits of about 40 of
    them. From scales of 2^-5 on the log-sum moves by 2^-14 of a logit's terms at most (a rounding to
    fp16 alone would move it six times as far); below, by the keys' error as well."""
    rng = np.random.default_rng(exp + 100)
    c = Cache(F, rng, 1, 4, 1, d, [300], kb=kb)
    L, T = c.L, 5
    cur = int(L.meta[0, 0, 4])
    # 5 x 1026 units: half an ulp of fp16 past an even number; subnormal scales are whole 2^-24
    s = 1026 * 2.0 ** (exp - 10) if exp >= -14 else 33 * 2.0 ** -24
    code = 5 if kb == 4 else 1
    L.mid_k_codes[cur].fill_(0x55)        # INT4 5, INT2 1
    L.mid_k_scales[cur].fill_(s)
    if kb == 4:   # a few keys of other codes
        L.mid_k_codes[cur][:, :, ::7] = torch.tensor(0x33, dtype=torch.uint8, device="cuda")
    L.sink_k.zero_(), L.recent_k.zero_()
    c.draft(rng, T)
    q = 40 / (code * s * np.sqrt(d)) * rng.uniform(0.75, 1.25, c.q.shape)
    c.q = np.minimum(q, 60000).astype(np.float16)
    c.tk[:] = 0
    c.dq = dev(c.q)
    c.load_tree()
    see = np.tril(np.ones((1, T, T), bool))
    _, lse = c.attend(see)
    _, _, _, K, V, _ = c.unit(0, 0)
    for i in range(T):
        for g in range(4):
            qq = c.q[0, i, g].astype(np.float64)
            z = np.concatenate([K, np.zeros((i + 1, d))]) @ qq / np.sqrt(d)
            want = z.max() + np.log(np.exp(z - z.max()).sum())
            terms = (np.abs(K) @ qq).max() / np.sqrt(d)
            # the remainder against E5M2 queries (1/8, a subnormal's half step 2^-17), the keys' own
            # error; fp32: products, the logarithm, the sum
            off = U * np.abs(K) @ (qq / 8 + 2.0 ** -17)
            off = off + (key_error(K, s) @ qq if kb == 4 else 2.0 ** -24 * qq.sum() * (s < 2.0 ** -13))
            tol = off.max() / np.sqrt(d) + 2.0 ** -22 * terms + (len(z) + d) * 2.0 ** -24 + 2.0 ** -20
            assert abs(lse[0, i, g] - want) <= tol, (i, g, lse[0, i, g], want, tol)
    if s >= 2.0 ** -5:
        c.check(see)


def test_attention_runs_the_same_twice_and_beside_another_stream(F):
    rng = np.random.default_rng(3)
    c = Cache(F, rng, 2, 8, 2, 128, [1500, 700])
    c.draft(rng, 16)
    see = np.stack([plain_layout(p, 16)[0] for p in random_parents(rng, 2, 16)])
    c.check(see)
    first = c.out.clone(), c.lse.clone()
    mask, out2 = dev(mask_words(see)), torch.empty_like(c.out)
    lse2, ws2 = torch.empty_like(c.lse), torch.empty_like(c.ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(20):   # two calls at once, each with its own workspace
        F.fade_tree_attention(c.L, c.dq, c.dk, c.dv, mask, None, c.out, c.lse, c.ws)
        with torch.cuda.stream(side):
            F.fade_tree_attention(c.L, c.dq, c.dk, c.dv, mask, None, out2, lse2, ws2)
    torch.cuda.synchronize()
    assert torch.equal(c.out, first[0]) and torch.equal(c.lse, first[1])
    assert torch.equal(out2, first[0]) and torch.equal(lse2, first[1])


def test_rows_without_nodes_leave_everything_as_it_was(F):
    rng = np.random.default_rng(21)
    c = Cache(F, rng, 3, 8, 2, 64, [500, 0, 90])
    c.draft(rng, 5)
    see = np.tile(np.tril(np.ones((5, 5), bool)), (3, 1, 1))
    for n in ([0, 0, 0], [5, 0, 2], [0, 5, 0]):
        c.out.fill_(7), c.lse.fill_(7)
        c.check(see, np.array(n, np.int32))


def test_two_captured_calls_replayed_in_any_order(F):
    """Two layers' calls captured into graphs of their own, each with its workspace, replayed at
    once and in either order: the bits of eager calls."""
    rng = np.random.default_rng(22)
    calls, see = [], np.tril(np.ones((2, 9, 9), bool))
    for lens in ([700, 90], [33, 2000]):
        c = Cache(F, rng, 2, 8, 2, 128, lens)
        c.draft(rng, 9)
        c.check(see)
        calls.append((c, c.out.clone(), c.lse.clone(), torch.cuda.CUDAGraph()))
    mask = dev(mask_words(see))
    for c, _, _, g in calls:
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            F.fade_tree_attention(c.L, c.dq, c.dk, c.dv, mask, None, c.out, c.lse, c.ws)
    side = torch.cuda.Stream()
    for order in ((0, 1), (1, 0), (0, 1)):
        for c, *_ in calls:
            c.out.fill_(7), c.lse.fill_(7), c.ws.fill_(255)
        side.wait_stream(torch.cuda.current_stream())
        calls[order[0]][3].replay()
        with torch.cuda.stream(side):
            calls[order[1]][3].replay()
        torch.cuda.synchronize()
        for c, out, lse, _ in calls:
            assert torch.equal(c.out, out) and torch.equal(c.lse, lse)


# --------------------------------------------------------------------------- commit
def state(c):
    """Every unit's held bytes in cache order (codes as they are)."""
    L, res = c.L, []
    for b in range(c.cfg.batch):
        for h in range(c.cfg.num_kv_heads):
            m = L.meta[b, h].cpu().numpy()
            ns, nm, nr, head, cur = (int(x) for x in m[:5])
            ring = [(head + i) % c.cfg.recent_window for i in range(nr)]
            g = lambda t: t[b, h].cpu().numpy()
            res.append([np.array([ns, nm, nr]), g(L.sink_k)[:ns], g(L.sink_v)[:ns],
                        g(L.mid_k_codes[cur])[:nm], g(L.mid_k_scales[cur])[:nm],
                        g(L.mid_v_codes[cur])[:nm], g(L.mid_v_scales[cur])[:nm],
                        g(L.recent_k)[ring], g(L.recent_v)[ring]])
    return res


COMMITS = [
    # B, hq, h, d, lens, W, S, T, n_path, options
    (2, 8, 2, 64, [200, 150], 64, 4, 16, [5, 3], {}),
    (3, 4, 1, 128, [90, 0, 2], 16, 4, 9, [9, 9, 0], dict(vb=4)),        # sinks still filling
    (2, 4, 4, 64, [30, 7], 3, 2, 20, [20, 1], dict(kb=2)),              # path longer than the ring
    (1, 8, 1, 128, [300], 1, 0, 64, [64], dict(codec="pq")),
    (2, 2, 1, 64, [10, 66], 64, 4, 7, [7, 7], dict(kb=2, vb=4)),        # ring with free slots
]


@pytest.mark.parametrize("policy", ["position", "h2o", "ema"])
@pytest.mark.parametrize("B,hq,h,d,lens,W,S,T,n_path,opt", COMMITS)
def test_commit(F, B, hq, h, d, lens, W, S, T, n_path, opt, policy):
    """The tiers are bit for bit what demotions and appends one token at a time make of the same
    tokens; the scores follow the accumulation in 64 bits."""
    caches = [Cache(F, np.random.default_rng(sum(lens) + T), B, hq, h, d, lens, W=W, S=S,
                    policy=policy, **opt) for _ in range(2)]
    c, step = caches
    rng = np.random.default_rng(1)
    c.draft(rng, T)
    path = np.zeros((B, T), np.int32)
    par = np.full((B, T), -1, np.int32)
    for b in range(B):   # increasing nodes, each the parent of the next
        path[b, :n_path[b]] = np.sort(rng.choice(T, n_path[b], replace=False))
        for i in range(1, n_path[b]):
            par[b, path[b, i]] = path[b, i - 1]
    see = np.stack([plain_layout(par[b], T)[0] for b in range(B)])
    _, lse = c.attend(see)
    before = [[c.unit(b, x) for x in range(h)] for b in range(B)]
    F.fade_tree_commit(c.L, c.dq, c.lse, c.dk, c.dv, dev(path), n_path, c.ws)
    F.fade_check_status(c.L)
    # one token at a time, row by row: caches of one row each
    for b in range(B):
        one = Cache(F, np.random.default_rng(sum(lens) + T), B, hq, h, d, lens, W=W, S=S,
                    policy=policy, **opt)
        for i in range(n_path[b]):
            F.fade_cache_demote(one.L)
            kk, vv = (dev(np.repeat(x[b, path[b, i]][None], B, 0)) for x in (c.tk, c.tv))
            F.fade_cache_append(one.L, kk, vv)
        for x in range(h):
            for got, want in zip(state(c)[b * h + x], state(one)[b * h + x]):
                assert np.array_equal(got.view(np.uint8), want.view(np.uint8)), (b, x)
        counts = F.fade_tier_counts(c.L)[b]
        assert np.array_equal(counts, state(one)[b * h][0])
    G = hq // h
    for b in range(B):
        for x in range(h):
            ns, nm, nr, K, _, old = before[b][x]
            got = c.unit(b, x)[5]
            a = n_path[b]
            if policy == "position" or a == 0:
                want, tol = np.concatenate([old, np.zeros(a)]), 0.0
            else:
                want, tol = scores_reference(c, b, x, G, K, old, path[b, :a], lse, policy)
            # held order: sinks, middle, recent; new tokens come last in every case
            assert got.shape == want.shape
            assert (np.abs(got - want) <= tol).all(), (b, x, float(np.abs(got - want).max()))


def scores_reference(c, b, h, G, K, old, path, lse, policy):
    """Scores in path order, and a bound: every probability moves by its logit's roundings (fp32
    sums) and lse's; each update rounds to fp32 three times."""
    d = K.shape[1]
    k = np.concatenate([K, c.tk[b, path, h].astype(np.float64)])
    s = np.concatenate([old, np.zeros(len(path))])
    tol = np.zeros_like(s)
    delta_max = 0.0
    for i, node in enumerate(path):
        live = len(old) + i + 1
        q = c.q[b, node, h * G:(h + 1) * G].astype(np.float64)
        z = q @ k[:live].T / np.sqrt(d)
        p = np.exp(z - lse[b, node, h * G:(h + 1) * G][:, None])
        delta = (d + 4) * 2.0 ** -24 / np.sqrt(d) * (np.abs(q) @ np.abs(k[:live]).T)
        err = (p * (np.expm1(delta) + 2.0 ** -19 + 2.0 ** -23 * np.abs(z))).sum(0)
        if policy == "h2o":
            s[:live] += p.sum(0)
            tol[:live] += err
        else:
            dl, g = c.cfg.ema_decay, 1 - c.cfg.ema_decay
            dl, g = float(np.float32(dl)), float(np.float32(1) - np.float32(dl))
            s[:live] = dl * s[:live] + g * p.sum(0)
            tol[:live] = dl * tol[:live] + g * err
        tol[:live] += 4 * 2.0 ** -24 * np.abs(s[:live])
        delta_max = max(delta_max, delta.max())
    return s, tol + 2.0 ** -30


@pytest.mark.parametrize("policy", ["h2o", "ema"])
@pytest.mark.parametrize("B,hq,h,d,hi,kb", [(70, 8, 2, 64, 300, 4), (200, 4, 4, 128, 90, 2),
                                            (5, 16, 2, 128, 4000, 4)])
def test_scores_of_ragged_rows(F, B, hq, h, d, hi, kb, policy):
    """Rows of different lengths and paths (some empty): scores by the 64-bit accumulation, and
    the same bits from a second cache."""
    T = 12
    make = lambda: Cache(F, np.random.default_rng(B), B, hq, h, d,
                         np.random.default_rng(B + 1).integers(0, hi, B).tolist(), W=16,
                         policy=policy, kb=kb)
    c, twin = make(), make()
    rng = np.random.default_rng(4)
    c.draft(rng, T)
    see = np.tile(np.tril(np.ones((T, T), bool)), (B, 1, 1))
    _, lse = c.attend(see)
    path = np.tile(np.arange(T, dtype=np.int32), (B, 1))
    n_path = rng.integers(0, T + 1, B)
    n_path[B // 2] = 0
    some = sorted({0, 1, B // 2, B - 1, *rng.integers(0, B, 4)})
    before = {b: [c.unit(b, u) for u in range(h)] for b in some}
    for x in (c, twin):
        F.fade_tree_commit(x.L, c.dq, c.lse, c.dk, c.dv, dev(path), n_path, c.ws)
        F.fade_check_status(x.L)
    for b in some:
        for u in range(h):
            got, old = c.unit(b, u)[5], before[b][u]
            if n_path[b] == 0:
                assert np.array_equal(got, old[5])
                continue
            want, tol = scores_reference(c, b, u, hq // h, old[3], old[5], path[b, :n_path[b]],
                                         lse, policy)
            assert (np.abs(got - want) <= tol).all(), (b, u)
            assert np.array_equal(got, twin.unit(b, u)[5])


def test_commit_of_a_bad_path_is_recorded(F):
    rng = np.random.default_rng(2)
    c = Cache(F, rng, 1, 4, 1, 64, [100], policy="position")
    c.draft(rng, 4)
    path = dev(np.array([[1, 77, -2, 3]], np.int32))
    F.fade_tree_commit(c.L, c.dq, None, c.dk, c.dv, path, [3])
    with pytest.raises(F.FadeError) as e:
        F.fade_check_status(c.L)
    assert e.value.status == 6
    # counts and contents stay consistent: the bad nodes read as node 0
    assert F.fade_tier_counts(c.L)[0].tolist() == [4, 35, 64]
    ring = c.unit(0, 0)[3][-3:]
    assert np.array_equal(ring[1], c.tk[0, 0, 0].astype(np.float64))


@pytest.mark.parametrize("policy", ["h2o", "ema"])
def test_a_key_of_minus_infinity_gets_no_mass(F, policy):
    """A cached key whose logits are -inf: probability 0, whatever the number of query rows."""
    rng = np.random.default_rng(15)
    c = Cache(F, rng, 1, 4, 2, 64, [150], policy=policy)
    T, a = 5, 3
    c.draft(rng, T)
    c.q[..., 3] = np.abs(c.q[..., 3]) + np.float16(0.25)
    c.dq = dev(c.q)
    c.L.sink_k[0, :, 2, 3] = -float("inf")
    see = np.tril(np.ones((1, T, T), bool))
    _, lse = c.attend(see)
    before = [c.unit(0, u) for u in range(2)]
    path = np.arange(T, dtype=np.int32)[None]
    F.fade_tree_commit(c.L, c.dq, c.lse, c.dk, c.dv, dev(path), [a], c.ws)
    F.fade_check_status(c.L)
    for u in range(2):
        _, _, _, K, _, old = before[u]
        got = c.unit(0, u)[5]
        keep = 1.0 if policy == "h2o" else np.float64(np.float32(0.9)) ** a
        assert abs(got[2] - keep * old[2]) <= 4 * 2.0 ** -24 * old[2]
        K[2] = 0.0   # the rest as in any commit
        want, tol = scores_reference(c, 0, u, 2, K, old, path[0, :a], lse, policy)
        rest = np.arange(len(want)) != 2
        assert (np.abs(got - want) <= tol)[rest].all()


@pytest.mark.parametrize("policy", ["h2o", "ema"])
def test_a_replayed_commit_past_the_capacity_leaves_the_row(F, policy):
    """A captured commit replayed until one row's middle tier is full: from then on the row keeps all it
    holds, its scores among it, the refusal is recorded, and the other row goes on."""
    rng = np.random.default_rng(14)
    c = Cache(F, rng, 2, 8, 2, 64, [200, 150], policy=policy, extra=60)
    T, n_path = 4, [3, 3]
    c.draft(rng, T)
    see = np.tile(np.tril(np.ones((T, T), bool)), (2, 1, 1))
    c.attend(see)
    path = torch.arange(T, dtype=torch.int32, device="cuda").repeat(2, 1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        F.fade_tree_commit(c.L, c.dq, c.lse, c.dk, c.dv, path, n_path, c.ws)
    slots = c.L.mid_k_codes[0].shape[2]
    fits = (slots - 132) // 3
    for _ in range(fits):
        g.replay()
    F.fade_check_status(c.L)
    assert c.unit(0, 0)[1] == 132 + 3 * fits
    held = lambda b: [x for h in range(2) for x in (*state(c)[b * 2 + h], c.unit(b, h)[5])]
    before, other = held(0), c.unit(1, 0)
    g.replay()
    for got, want in zip(held(0), before):
        assert np.array_equal(got.view(np.uint8), want.view(np.uint8))
    assert c.unit(1, 0)[1] == other[1] + 3
    assert not np.array_equal(c.unit(1, 0)[5][:other[1]], other[5][:other[1]])
    with pytest.raises(F.FadeError) as e:
        F.fade_check_status(c.L)
    assert e.value.status == 6


# --------------------------------------------------------------------------- together
@pytest.mark.parametrize("policy,codec,norm", [("none", "int", True), ("position", "int", False),
                                               ("h2o", "int", True), ("ema", "pq", False)])
def test_draft_steps_together(F, policy, codec, norm):
    """Draft, attend, commit, evict, draft again, then a plain step, through FadeCache; every
    attention against the 64-bit form of the state it read, every commit's counts and scores."""
    from tiered_mixed_precision_gb300.model import FadeCache

    rng = np.random.default_rng(7)
    B, hq, h, d, T, P, layers = 2, 8, 2, 64, 11, 150, 2
    cfg = F.Config(batch=B, num_q_heads=hq, num_kv_heads=h, head_dim=d, n_sink=4,
                   recent_window=16, int4_budget=90 if policy != "none" else -1,
                   mid_capacity=400, policy=policy, v_codec=codec)
    fc = FadeCache(cfg, layers, P, 800)
    cb = None
    if codec == "pq":
        cb = rng.standard_normal((d // 4, 256, 4)).astype(np.float16)
        fc.set_pq_codebook(dev(cb))
    if norm:
        fc.set_qk_norm(*(dev((1 + 0.2 * rng.standard_normal(d)).astype(np.float16))
                         for _ in range(2)))
    draw = lambda *s: dev(rng.standard_normal(s).astype(np.float16))
    for layer in range(layers):
        fc.prefill(layer, draw(B, h, P, d), draw(B, h, P, d), q_raw=draw(B, hq, P, d))
    view = Cache.__new__(Cache)
    view.F, view.cfg, view.cb, view.fused = F, cfg, cb, False
    for step in range(4):
        par = random_parents(rng, B, T)
        n = rng.integers(T // 2, T + 1, B).astype(np.int32)
        want_pos = fc.next_positions()
        tree = fc.tree_begin(dev(par), dev(n))
        see = np.stack([plain_layout(par[b], n[b])[0] for b in range(B)])
        assert np.array_equal(tree.mask.cpu().numpy(), mask_words(see))
        for b in range(B):
            assert np.array_equal(tree.pos[b].cpu().numpy(),
                                  want_pos[b] + plain_layout(par[b], n[b])[1])
            held = fc.layers[0].h_n_sink[b] + fc.layers[0].h_n_mid[b] + fc.layers[0].h_n_recent[b]
            assert held == want_pos[b]
        before = []
        for layer in range(layers):
            x = draw(B, T, hq + 2 * h, d)
            out = torch.full((B, T, hq, d), 7.0, dtype=torch.float16, device="cuda")
            fc.tree_attend(layer, tree, x[:, :, :hq], x[:, :, hq:hq + h], x[:, :, hq + h:], out)
            view.L = fc.layers[layer]
            view.q, view.tk = (t[layer].cpu().numpy() for t in (tree.q_rot, tree.k_rot))
            view.tv = x[:, :, hq + h:].cpu().numpy()
            got, lse = out.double().cpu().numpy(), tree.lse[layer].double().cpu().numpy()
            units = [[view.unit(b, u) for u in range(h)] for b in range(B)]
            before.append((units, view.q, view.tk, lse))
            for b in range(B):
                assert (got[b, n[b]:] == 7).all()
                for i in range(n[b]):
                    js = np.nonzero(see[b, i])[0]
                    for a in range(hq):
                        u = a // (hq // h)
                        compare(got[b, i, a], lse[b, i, a], view.q[b, i, a].astype(np.float64),
                                np.concatenate([units[b][u][3], view.tk[b, js, u]]),
                                np.concatenate([units[b][u][4], view.tv[b, js, u]]), (step, b, i))
        path, lens = np.zeros((B, T), np.int32), []
        for b in range(B):
            leaf = int(n[b]) - 1
            nodes = np.nonzero(see[b, leaf])[0]
            nodes = nodes[:rng.integers(0, len(nodes) + 1)]
            path[b, :len(nodes)] = nodes
            lens.append(len(nodes))
        fc.tree_commit(tree, dev(path), lens)
        for layer in range(layers):
            units, view.q, view.tk, lse = before[layer]
            view.L = fc.layers[layer]
            F.fade_check_status(view.L)
            for b in range(B):
                for u in range(h):
                    now = view.unit(b, u)
                    assert sum(now[:3]) == sum(units[b][u][:3]) + lens[b]
                    if policy in ("h2o", "ema") and lens[b]:
                        want, tol = scores_reference(view, b, u, hq // h, units[b][u][3],
                                                     units[b][u][5], path[b, :lens[b]], lse,
                                                     policy)
                        assert (np.abs(now[5] - want) <= tol).all()
    # a plain step goes on from there
    q, k, v = draw(layers, B, hq, d), draw(layers, B, h, d), draw(layers, B, h, d)
    out = torch.empty_like(q)
    fc.step_all(q, k, v, out)
    for layer in range(layers):
        F.fade_check_status(fc.layers[layer])
        assert torch.isfinite(out[layer]).all()


def test_a_captured_tree_step_follows_the_cache(F):
    """norm and attention captured once and replayed while the cache grows: the bits of an eager
    call on the same state."""
    rng = np.random.default_rng(9)
    c = Cache(F, rng, 2, 8, 2, 128, [900, 300], extra=700)
    T = 6
    c.draft(rng, T)
    see = np.stack([plain_layout(p, T)[0] for p in random_parents(rng, 2, T)])
    mask, path = dev(mask_words(see)), torch.arange(T, dtype=torch.int32, device="cuda").repeat(2, 1)
    c.check(see)
    ws2, out2, lse2 = torch.empty_like(c.ws), torch.empty_like(c.out), torch.empty_like(c.lse)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        F.fade_tree_attention(c.L, c.dq, c.dk, c.dv, mask, None, out2, lse2, ws2)
    for n_path in ([6, 1], [6, 6], [0, 3]):
        for _ in range(40):
            F.fade_tree_commit(c.L, c.dq, None, c.dk, c.dv, path, n_path)
        c.attend(see)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out2, c.out) and torch.equal(lse2, c.lse)
    c.check(see)


def test_the_codes_that_a_commit_records_are_named(F):
    c = Cache(F, np.random.default_rng(0), 1, 4, 1, 64, [20])
    for code, name in ((20, "path node"), (21, "middle slot or ring head")):
        c.L.status[0] = code
        with pytest.raises(F.FadeError) as e:
            F.fade_check_status(c.L)
        assert e.value.status == 6 and f"{code} tree commit's {name}" in str(e.value)


def test_tree_buffers_do_not_pile_up(F):
    """Trees of every size, each attended to: at most two sizes' buffers are held. Trees of two sizes can
    be held at once, each with buffers of its own."""
    rng = np.random.default_rng(25)
    c, _, _, _ = twins(F, rng, "none", -1)
    B, hq, h, d = 2, 8, 2, 64

    def attend(T):
        par = torch.arange(T, dtype=torch.int32, device="cuda").sub(1).repeat(B, 1)
        tree = c.tree_begin(par)
        x = torch.randn((B, T, hq + 2 * h, d), device="cuda").half()
        out = torch.empty((B, T, hq, d), dtype=torch.float16, device="cuda")
        for layer in range(2):
            c.tree_attend(layer, tree, x[:, :, :hq], x[:, :, hq:hq + h], x[:, :, hq + h:], out)
        return tree

    size = lambda t: sum(x.untyped_storage().nbytes()
                         for x in (t.mask, t.pos, t.q_rot, t.k_rot, t.lse, t.ws))
    attend(64)
    torch.cuda.synchronize()
    start = torch.cuda.memory_allocated()
    largest = size(c.tree_begin(torch.zeros((B, 64), dtype=torch.int32, device="cuda")))
    for T in range(1, 64):
        attend(T)
    assert torch.cuda.memory_allocated() <= start + largest
    small, wide = attend(9), attend(30)
    assert small.q_rot.data_ptr() != wide.q_rot.data_ptr()
    lse = small.lse.clone()
    again = attend(30)
    assert again.q_rot.data_ptr() == wide.q_rot.data_ptr()   # as many nodes: the same buffers
    path = torch.arange(9, dtype=torch.int32, device="cuda").repeat(B, 1)
    before = F.fade_tier_counts(c.layers[0]).sum(1)
    c.tree_commit(small, path, [9, 4])
    assert torch.equal(small.lse, lse)
    assert (F.fade_tier_counts(c.layers[0]).sum(1) - before).tolist() == [9, 4]


def test_tree_buffers_of_captured_and_side_stream_calls_outlive_their_tree(F):
    """A captured tree_attend whose tree is dropped: the next tree of as many nodes has its buffers, and a
    replay writes there. Calls on another stream: the buffers are not given away while they run."""
    rng = np.random.default_rng(26)
    c, _, _, _ = twins(F, rng, "none", -1)
    B, hq, h, d, T = 2, 8, 2, 64, 12
    par = torch.arange(T, dtype=torch.int32, device="cuda").sub(1).repeat(B, 1)
    x = torch.randn((B, T, hq + 2 * h, d), device="cuda").half()
    out, want = (torch.empty((B, T, hq, d), dtype=torch.float16, device="cuda") for _ in range(2))
    run = lambda tree, o: c.tree_attend(0, tree, x[:, :, :hq], x[:, :, hq:hq + h],
                                        x[:, :, hq + h:], o)
    tree = c.tree_begin(par)
    run(tree, want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(tree, out)
    at = tree.q_rot.data_ptr()
    del tree
    for n in (3, 40, 7):   # other sizes, and memory of other uses
        c.tree_begin(par[:, :n].contiguous() if n < T else torch.full((B, n), -1, dtype=torch.int32,
                                                                      device="cuda"))
        torch.full((1 << 20,), 0xff, dtype=torch.uint8, device="cuda")
    tree = c.tree_begin(par)
    assert tree.q_rot.data_ptr() == at
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    side = torch.cuda.Stream()
    for _ in range(4):
        tree = c.tree_begin(par[:, :9].contiguous())
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(20000000)
            c.tree_attend(0, tree, x[:, :9, :hq], x[:, :9, hq:hq + h], x[:, :9, hq + h:],
                          out.view(-1)[:B * 9 * hq * d].view(B, 9, hq, d))
        got = tree.q_rot.untyped_storage().data_ptr()
        del tree
        c.tree_begin(par[:, :5].contiguous())   # the nine nodes' buffers are let go
        other = torch.empty(2 * B * 9 * hq * d, dtype=torch.float16, device="cuda")
        assert other.data_ptr() != got
        side.synchronize()


# --------------------------------------------------------------------------- norms that change
def twins(F, rng, policy, budget, layers=2):
    """Two caches of the same contents and a function that draws a step's q, k and v."""
    from tiered_mixed_precision_gb300.model import FadeCache

    B, hq, h, d, P = 2, 8, 2, 64, 200
    cfg = F.Config(batch=B, num_q_heads=hq, num_kv_heads=h, head_dim=d, n_sink=4, recent_window=16,
                   int4_budget=budget, mid_capacity=400, policy=policy)
    draw = lambda *s: dev(rng.standard_normal(s).astype(np.float16))
    prompt = [(draw(B, h, P, d), draw(B, h, P, d)) for _ in range(layers)]
    caches = []
    for _ in range(2):
        caches.append(FadeCache(cfg, layers, P, 800))
        for layer, (k, v) in enumerate(prompt):
            caches[-1].prefill(layer, k.clone(), v.clone())
    step = lambda n=1: (draw(n, layers, B, hq, d), draw(n, layers, B, h, d), draw(n, layers, B, h, d))
    weights = lambda: [dev((1 + 0.5 * rng.standard_normal(d)).astype(np.float16)) for _ in range(2)]
    return (*caches, step, weights)


def test_growing_steps_follow_a_changed_norm(F):
    """growing_step after set_qk_norm sets, changes (weights, eps) or clears the norm: the bits of an
    eager step."""
    rng = np.random.default_rng(19)
    grow, eager, step, weights = twins(F, rng, "none", -1)
    bufs = [t[0].clone() for t in step()]
    out, want = torch.empty_like(bufs[0]), torch.empty_like(bufs[0])
    w = weights()
    for norm in (None, (*w, 1e-6), (*weights(), 1e-6), (*w, 0.5), (w[0], None, 1e-6), (None, None, 1.0)):
        for c in (grow, eager):
            if norm:
                c.set_qk_norm(*norm)
        for _ in range(2):
            x = [t[0] for t in step()]
            for b, t in zip(bufs, x):
                b.copy_(t)
            grow.growing_step(*bufs, out)
            eager.step_all(*x, want)
            assert torch.equal(out, want), norm
    assert grow.growing_captures <= 8   # one a norm, and for rows that reach a new tile


def test_host_fed_steps_follow_a_changed_norm(F):
    rng = np.random.default_rng(20)
    fed, eager, step, weights = twins(F, rng, "position", 90)
    want = torch.empty_like(step()[0][0])
    for _ in range(3):   # to the steady state
        x = [t[0] for t in step()]
        for c in (fed, eager):
            c.step_all(*x, want)
    for norm in (None, (*weights(), 1e-6), (*weights(), 1e-5), (None, None, 1.0)):
        for c in (fed, eager):
            if norm:
                c.set_qk_norm(*norm)
        x = step(3)
        host = [t.cpu().pin_memory() for t in x]
        out = torch.zeros(x[0].shape, dtype=torch.float16).pin_memory()
        fed.run_from_host(*host, out)
        torch.cuda.current_stream().synchronize()
        for s in range(3):
            eager.step_all(x[0][s], x[1][s], x[2][s], want)
            assert torch.equal(out[s], want.cpu()), norm


def test_host_fed_steps_after_a_drafted_tree(F):
    """A committed path leaves evictions to the next step: the captured steady-state steps are refused
    until a step has made them, and then go on with the bits of eager ones."""
    rng = np.random.default_rng(27)
    fed, eager, step, _ = twins(F, rng, "position", 90)
    B, hq, h, d, T = 2, 8, 2, 64, 6
    want = torch.empty_like(step()[0][0])

    def both(x):
        for c in (fed, eager):
            c.step_all(*(t[0] for t in x), want)

    def host_fed():
        x = step(2)
        out = torch.zeros(x[0].shape, dtype=torch.float16).pin_memory()
        fed.run_from_host(*(t.cpu().pin_memory() for t in x), out)
        torch.cuda.current_stream().synchronize()
        for s in range(2):
            eager.step_all(x[0][s], x[1][s], x[2][s], want)
            assert torch.equal(out[s], want.cpu())

    for _ in range(3):   # to the steady state
        both(step())
    host_fed()
    par = torch.arange(T, dtype=torch.int32, device="cuda").sub(1).repeat(B, 1)
    x = torch.randn((B, T, hq + 2 * h, d), device="cuda").half()
    out = torch.empty((B, T, hq, d), dtype=torch.float16, device="cuda")
    for c in (fed, eager):
        tree = c.tree_begin(par)
        for layer in range(2):
            c.tree_attend(layer, tree, x[:, :, :hq], x[:, :, hq:hq + h], x[:, :, hq + h:], out)
        c.tree_commit(tree, par + 1, [4, 1])
    q, k, v = (t.cpu().pin_memory() for t in step(1))
    before = [[a.copy() for a in m] for m in fed.mirror()]
    with pytest.raises(RuntimeError):
        fed.run_from_host(q, k, v, torch.zeros(q.shape, dtype=torch.float16).pin_memory())
    assert all((a == b).all() for m, n in zip(fed.mirror(), before) for a, b in zip(m, n))
    both(step())
    host_fed()
    for layer in range(2):
        assert (F.fade_tier_counts(fed.layers[layer]) == F.fade_tier_counts(eager.layers[layer])).all()


def test_a_captured_step_keeps_its_norm_weights(F):
    """set_qk_norm after a capture: the graph's weights stay allocated and its replays read them."""
    import gc
    import weakref

    rng = np.random.default_rng(23)
    grow, eager, step, weights = twins(F, rng, "none", -1)
    w = weights()
    kept = [t.clone() for t in w]
    grow.set_qk_norm(*w)
    eager.set_qk_norm(*kept)
    bufs = [t[0].clone() for t in step()]
    out, want = torch.empty_like(bufs[0]), torch.empty_like(bufs[0])
    g = grow.capture_growing_step(*bufs, out)
    refs = [weakref.ref(t) for t in w]
    del w
    grow.set_qk_norm(None, None)
    gc.collect()
    assert all(r() is not None for r in refs)
    junk = [torch.full((64,), float("nan"), dtype=torch.float16, device="cuda") for _ in range(64)]
    grow.replay_growing(g)
    eager.step_all(*bufs, want)
    assert torch.equal(out, want) and len(junk) == 64
