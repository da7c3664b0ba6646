"""What is measured of the drafted-token operators: cases, inputs, plain forms, definitions.

The operators verify a tree of drafted tokens against a tiered cache and keep the accepted path:

* ``layout``: parents -> ancestor bit masks and positions (``fade_tree_layout``);
* ``norm``: per-head RMS norm of queries and keys with the rotation to their positions in the
  same pass (``fade_qk_norm_rope``);
* ``attention``: every node attends to all tiers of the cache and to its ancestors
  (``fade_tree_attention``);
* ``commit``: the accepted path's attention mass is added to the importance scores (H2O, EMA) and
  its tokens are appended, demoting what leaves the recent window (``fade_tree_commit``).

``own`` false computes them with elementary torch operations; ``own`` true calls the framework.
"""

import math

import numpy as np
import torch

own = False

GROUP = 32          # channels per quantisation scale
SINKS, WINDOW = 4, 64
EMA_DECAY = 0.9


# --------------------------------------------------------------------------- cases
def _attn(name, batch, hq, h, d, mid, nodes, kb=4, vb=2, pq=False, tree="tree", lo=None):
    """lo: middle tokens per row uniform in [lo, mid] (ragged); lo None: mid in every row."""
    return {"name": name, "op": "attention", "batch": batch, "hq": hq, "h": h, "d": d,
            "mid": mid, "mid_lo": mid if lo is None else lo, "nodes": nodes, "kb": kb, "vb": vb,
            "pq": pq, "tree": tree}


def _commit(name, batch, hq, h, d, mid, nodes, policy, depth):
    """depth: the longest accepted path (rows accept 1 .. depth tokens)."""
    return {"name": name, "op": "commit", "batch": batch, "hq": hq, "h": h, "d": d, "mid": mid,
            "mid_lo": mid, "nodes": nodes, "kb": 4, "vb": 2, "pq": False, "tree": "tree",
            "policy": policy, "depth": depth}


def _norm(name, batch, tokens, hq, h, d, rotary, maxpos, fused):
    """fused: q and k are slices of one projection's output [rows][tokens][(hq + 2 h) d]."""
    return {"name": name, "op": "norm", "batch": batch, "tokens": tokens, "hq": hq, "h": h,
            "d": d, "rotary": rotary, "maxpos": maxpos, "fused": fused}


def _layout(name, batch, nodes, tree):
    return {"name": name, "op": "layout", "batch": batch, "nodes": nodes, "tree": tree}


def listed():
    return [
        # one request, a small tree: the latency of the step's first launch
        _layout("layout_one_request", 1, 16, "tree"),
        # the largest batch and tree, rows of different sizes
        _layout("layout_full_batch", 256, 64, "tree"),
        # a plain decode token of one request (16 query and 2 KV heads): latency
        _norm("norm_one_token", 1, 1, 16, 2, 128, 0, 8192, True),
        # a drafted tree for 64 requests, out of a fused projection
        _norm("norm_tree_batch", 64, 16, 32, 8, 128, 0, 8192, True),
        # a prompt's keys and queries, partial rotation
        _norm("norm_prompt", 4, 8191, 32, 8, 128, 96, 131072, False),
        # the single-layer workload with a chain of 4 drafted tokens: latency
        _attn("attention_chain_d64", 1, 8, 2, 64, 444, 4, tree="chain"),
        # one request without eviction, INT4 K and V, 8 query heads per KV head
        _attn("attention_safe_one_request", 1, 16, 2, 128, 4096, 16, vb=4),
        # a short cache under eviction, product-quantised V, an odd tree
        _attn("attention_short_pq", 8, 32, 8, 64, 400, 25, pq=True),
        # the throughput workload's cache, a tree of 16 nodes
        _attn("attention_batch64", 64, 32, 8, 128, 4096, 16),
        # long ragged rows without eviction, the widest tree
        _attn("attention_long_ragged", 4, 32, 8, 128, 131001, 64, lo=65473),
        # the accepted paths of the throughput workload (no scores to keep)
        _commit("commit_position", 64, 32, 8, 128, 4096, 16, "position", 6),
        # the accepted paths of a long-context batch whose scores follow the attention
        _commit("commit_ema", 4, 32, 8, 128, 16384, 16, "ema", 6),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["layout", "norm", "attention", "attention", "attention", "commit"])
    tree = rng.choice(["chain", "tree", "tree"])
    if op == "layout":
        c = _layout("", _log(rng, 1, 256), rng.randint(1, 64), tree)
    else:
        d = rng.choice([64, 128])
        h = rng.choice([1, 2, 4, 8])
        hq = h * rng.choice([1, 2, 4, 8])
        if op == "norm":
            tokens = _log(rng, 1, 8192)
            rotary = rng.choice([0, 0, 4 * rng.randint(1, d // 4 - 1)])
            batch = _log(rng, 1, max(1, min(64, 1300000 // (tokens * (hq + h)))))
            c = _norm("", batch, tokens, hq, h, d, rotary, 1 << rng.randint(13, 17),
                      rng.random() < 0.5)
        elif op == "attention":
            mid = _log(rng, 1, 131000)
            batch = _log(rng, 1, max(1, min(64, 12000000 // (mid * hq))))
            pq = rng.random() < 0.25
            c = _attn("", batch, hq, h, d, mid, rng.randint(1, 64), rng.choice([4, 4, 2]),
                      2 if pq else rng.choice([2, 4]), pq, tree,
                      rng.choice([None, max(0, mid // 2)]))
        else:
            mid = _log(rng, 16, 16384)
            batch = _log(rng, 1, max(1, min(64, 262144 // mid)))
            c = _commit("", batch, hq, h, d, mid, rng.randint(8, 64),
                        rng.choice(["position", "h2o", "ema"]), rng.randint(1, 6))
            c["tree"] = tree
    del c["name"]
    return c


def work(case):
    B = case["batch"]
    if case["op"] == "layout":
        n = B * case["nodes"]
        return {"bytes": n * (4 + 8 + 4) + 8 * B, "flops": 0}
    d, hq, h = case["d"], case["hq"], case["h"]
    if case["op"] == "norm":
        n = B * case["tokens"]
        rows = min(n, case["maxpos"])
        r = case["rotary"] or d
        return {"bytes": n * ((hq + h) * d * 4 + 4) + rows * r * 4 + 4 * d,
                "flops": n * (hq + h) * (4 * d + 3 * r)}
    lens, nodes = _row_sizes(case)
    k_row = d * case["kb"] // 8 + 2 * (d // GROUP)
    v_row = d // 4 if case["pq"] else d * case["vb"] // 8 + 2 * (d // GROUP)
    fp16 = SINKS + WINDOW - 1
    if case["op"] == "attention":
        nbytes = flops = 0
        for m, n in zip(lens, nodes):
            nbytes += h * (m * (k_row + v_row) + (fp16 + n) * 4 * d) + n * hq * (4 * d + 4) + 8 * n
            flops += 4 * d * hq * (n * (m + fp16) + n * (n + 1) // 2)
        if case["pq"]:
            nbytes += 512 * d
        return {"bytes": nbytes, "flops": flops}
    paths = _paths(case)
    nbytes = flops = 0
    for m, p in zip(lens, paths):
        a = len(p)
        # the kept and the demoted tokens are read and written once each
        nbytes += h * (8 * d * a + max(0, a - 1) * (4 * d + k_row + v_row) + 32) + 4 * a
        if case["policy"] != "position":
            nbytes += h * (m * k_row + fp16 * 2 * d + (m + fp16) * 8) + a * hq * (2 * d + 4)
            flops += 2 * d * hq * (a * (m + fp16) + a * (a + 1) // 2)
    return {"bytes": nbytes, "flops": flops}


# --------------------------------------------------------------------------- inputs
def _row_sizes(case):
    """Middle tokens and tree nodes of every row (part of the case: the same for every seed)."""
    rng = np.random.default_rng(case["mid"] * 131 + case["nodes"] * 7 + case["batch"])
    B = case["batch"]
    lens = rng.integers(case["mid_lo"], case["mid"] + 1, B)
    lens[0] = case["mid"]
    full = case["nodes"]
    nodes = rng.integers(max(1, (3 * full) // 4), full + 1, B)
    nodes[0] = full
    if case["op"] == "commit":
        nodes[:] = full
    return [int(x) for x in lens], [int(x) for x in nodes]


def _parents(case, seed=None):
    """Parents [B][T]: a chain, or three roots with later nodes hanging from recent ones."""
    B, T = case["batch"], case["nodes"]
    out = np.full((B, T), -1, np.int32)
    if case["tree"] == "chain":
        out[:] = np.arange(T) - 1
        return out
    rng = np.random.default_rng(12345 + T if seed is None else [seed, 17])
    for i in range(1, T):
        out[:, i] = rng.integers(max(-1, i - 6) if i > 2 else -1, i, B)
    return out


def _paths(case):
    """Accepted path of every row: the last nodes' ancestors, cut to 1 .. depth tokens."""
    par = _parents(case)
    rng = np.random.default_rng(777 + case["nodes"])
    out = []
    for b in range(case["batch"]):
        best = []
        for leaf in range(case["nodes"]):
            p, i = [], leaf
            while i >= 0:
                p.append(i)
                i = int(par[b, i])
            if len(p) > len(best):
                best = p
        best = best[::-1]
        out.append(best[:int(rng.integers(1, min(case["depth"], len(best)) + 1))])
    return out


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _quantize(x, bits):
    """Symmetric codes (int8) and fp16 scales of fp16 rows [..., d]."""
    qmax = 2 ** (bits - 1) - 1
    g = x.float().reshape(*x.shape[:-1], -1, GROUP)
    a = g.abs().amax(-1)
    s = (a / qmax).half()
    s = torch.where((a > 0) & (s == 0), torch.full_like(s, 2.0 ** -24), s)
    sf = s.float()[..., None]
    q = torch.where(sf > 0, torch.round(g / torch.where(sf > 0, sf, torch.ones_like(sf))),
                    torch.zeros_like(g))
    return q.clamp_(-qmax, qmax).reshape(x.shape).to(torch.int8), s


def _pack(q, bits):
    per = 8 // bits
    u = (q.to(torch.int32) & ((1 << bits) - 1)).reshape(*q.shape[:-1], -1, per)
    v = sum(u[..., i] << (bits * i) for i in range(per))
    return v.to(torch.uint8)


def _unpack(codes, bits):
    per = 8 // bits
    parts = [(codes >> (bits * i)) & ((1 << bits) - 1) for i in range(per)]
    u = torch.stack(parts, -1).reshape(*codes.shape[:-1], -1).to(torch.int16)
    return torch.where(u >= 1 << (bits - 1), u - (1 << bits), u)


def _normal(shape, g, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).half()


def _cache_inputs(case, seed):
    """One layer's tiers as a program holds them when it drafts: full sinks, a recent window with
    one free slot, middle rows packed; the drafted tokens' rotated q and k, and their v."""
    g = _gen(seed)
    B, H, Hq, d, T = case["batch"], case["h"], case["hq"], case["d"], case["nodes"]
    lens, nodes = _row_sizes(case)
    cap = max(lens) + T + 1
    C = (cap + 63) // 64 * 64
    st = {"lens": lens, "nodes": nodes, "cap": cap, "C": C}
    st["sink_k"], st["sink_v"] = (_normal((B, H, SINKS, d), g) for _ in range(2))
    st["recent_k"], st["recent_v"] = (_normal((B, H, WINDOW, d), g) for _ in range(2))
    kc = torch.zeros((B, H, C, d * case["kb"] // 8), dtype=torch.uint8, device="cuda")
    vc = torch.zeros((B, H, C, d * case["vb"] // 8), dtype=torch.uint8, device="cuda")
    ks = torch.zeros((B, H, C, d // GROUP), dtype=torch.float16, device="cuda")
    vs = torch.zeros_like(ks)
    outlier = torch.ones(d, device="cuda", dtype=torch.float16)
    outlier[int(torch.randint(d, (1,), generator=g, device="cuda"))] = 8.0
    for b in range(B):
        n = lens[b]
        if n == 0:
            continue
        q, s = _quantize(_normal((H, n, d), g) * outlier, case["kb"])
        kc[b, :, :n], ks[b, :, :n] = _pack(q, case["kb"]), s
        if case["pq"]:
            vc[b, :, :n] = torch.randint(256, (H, n, d // 4), generator=g, device="cuda",
                                         dtype=torch.uint8)
        else:
            q, s = _quantize(_normal((H, n, d), g), case["vb"])
            vc[b, :, :n], vs[b, :, :n] = _pack(q, case["vb"]), s
    st["mid_k_codes"], st["mid_v_codes"], st["mid_k_scales"], st["mid_v_scales"] = kc, vc, ks, vs
    if case["pq"]:
        st["codebook"] = _normal((d // 4, 256, 4), g)
    st["head"] = int(torch.randint(WINDOW, (1,), generator=g, device="cuda"))
    st["q"] = _normal((B, T, Hq, d), g)
    # the drafted k and v as a program has them: k rotated, v a slice of a fused projection
    st["tree_k"] = _normal((B, T, H, d), g)
    st["tree_v"] = _normal((B, T, 3 * H, d), g)[:, :, 2 * H:]
    par = _parents(case)
    bits = np.zeros((B, T), np.uint64)
    for b in range(B):
        for i in range(nodes[b]):
            up = bits[b, par[b, i]] if par[b, i] >= 0 else np.uint64(0)
            bits[b, i] = up | (np.uint64(1) << np.uint64(i))
    st["mask"] = torch.from_numpy(bits.view(np.int64)).cuda()
    st["n_nodes"] = torch.tensor(nodes, dtype=torch.int32, device="cuda")
    return st


def _commit_inputs(case, seed):
    """The cache inputs with accepted paths. The tokens that leave the window hold the accepted
    tokens' values, so that a pass repeated from the same counts does the same work."""
    st = _cache_inputs(case, seed)
    g = _gen(seed + 1)
    B, H, T, C = case["batch"], case["h"], case["nodes"], st["C"]
    paths = _paths(case)
    st["paths"] = paths
    st["n_path"] = np.array([len(p) for p in paths], np.int32)
    path = np.zeros((B, T), np.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = p
        for i, node in enumerate(p[1:]):
            slot = (st["head"] + i) % WINDOW
            st["recent_k"][b, :, slot] = st["tree_k"][b, node]
            st["recent_v"][b, :, slot] = st["tree_v"][b, node]
    free = (st["head"] + WINDOW - 1) % WINDOW
    st["recent_k"][:, :, free] = 0
    st["recent_v"][:, :, free] = 0
    st["path"] = torch.from_numpy(path).cuda()
    # no scores to keep under the position policy: they stay zero
    scale = 0.0 if case["policy"] == "position" else 1.0
    rand = lambda *s: torch.rand(s, generator=g, device="cuda") * scale
    st["sink_scores"], st["mid_scores"] = rand(B, H, SINKS), rand(B, H, C)
    st["recent_scores"] = rand(B, H, WINDOW)
    for b in range(B):
        st["mid_scores"][b, :, st["lens"][b]:] = 0
    st["recent_scores"][:, :, free] = 0
    # log-sum-exp of every node's attention (what the attention call left with the program)
    if case["policy"] == "position":
        st["lse"] = torch.zeros((B, T, case["hq"]), device="cuda")
    else:
        st["lse"] = _plain_attention(case, st)[1]
    return st


def _norm_inputs(case, seed):
    g = _gen(seed)
    B, T, Hq, H, d = case["batch"], case["tokens"], case["hq"], case["h"], case["d"]
    if case["fused"]:
        x = _normal((B, T, Hq + 2 * H, d), g, 2.0)
        q, k = x[:, :, :Hq], x[:, :, Hq:Hq + H]
    else:   # head-major, the layout prompts have
        q = _normal((B, Hq, T, d), g, 2.0).transpose(1, 2)
        k = _normal((B, H, T, d), g, 2.0).transpose(1, 2)
    qw = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).half()
    kw = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).half()
    base = torch.randint(0, max(1, case["maxpos"] - T), (B, 1), generator=g, device="cuda")
    pos = (base + torch.arange(T, device="cuda")).clamp_(max=case["maxpos"] - 1).int()
    # the rotation table the framework keeps: [max_pos][d/4] blocks of two cosines, two sines
    r = case["rotary"] or d
    inv = torch.tensor([500000.0 ** (-2.0 * i / r) for i in range(r // 2)],
                       dtype=torch.float64, device="cuda").float()
    ang = (torch.arange(case["maxpos"], device="cuda").float()[:, None] * inv).double()
    table = torch.zeros((case["maxpos"], d // 4, 4), device="cuda")
    table[:, :r // 4, 0:2] = ang.cos().float().reshape(-1, r // 4, 2)
    table[:, :r // 4, 2:4] = ang.sin().float().reshape(-1, r // 4, 2)
    return {"q": q, "k": k, "qw": qw, "kw": kw, "pos": pos, "table": table, "eps": 1e-6}


def _layout_inputs(case, seed):
    g = _gen(seed)
    B, T = case["batch"], case["nodes"]
    rng = np.random.default_rng([seed, B, T])
    nodes = rng.integers(max(1, T // 2), T + 1, B).astype(np.int32)
    return {"parents": torch.from_numpy(_parents(case, seed)).cuda(),
            "n_nodes": torch.from_numpy(nodes).cuda(),
            "base": torch.randint(0, 131072, (B,), generator=g, device="cuda").int()}


def _inputs(case, seed):
    op = case["op"]
    if op == "layout":
        return _layout_inputs(case, seed)
    if op == "norm":
        return _norm_inputs(case, seed)
    return _commit_inputs(case, seed) if op == "commit" else _cache_inputs(case, seed)


def prepare(case, seed):
    st = _inputs(case, seed)
    st["case"] = case
    B, op = case["batch"], case["op"]
    if op == "attention":
        st["out"] = torch.zeros_like(st["q"])
        st["lse"] = torch.zeros(st["q"].shape[:3], device="cuda")
    if own:
        from tiered_mixed_precision_gb300 import fade as F

        st["F"] = F
        if op in ("layout", "norm"):
            kw = {} if op == "layout" else {"rope_rotary_dim": case["rotary"]}
            if op == "norm":
                kw.update(num_q_heads=case["hq"], num_kv_heads=case["h"], head_dim=case["d"])
            base = dict(num_q_heads=8, num_kv_heads=2, head_dim=64, mid_capacity=64)
            st["cfg"] = F.Config(batch=B, **{**base, **kw})
            if op == "layout":
                T = case["nodes"]
                st["mask"] = torch.zeros((B, T), dtype=torch.int64, device="cuda")
                st["pos"] = torch.zeros((B, T), dtype=torch.int32, device="cuda")
            else:
                st["q_rot"] = torch.empty(st["q"].shape, dtype=torch.float16, device="cuda")
                st["k_rot"] = torch.empty(st["k"].shape, dtype=torch.float16, device="cuda")
            return st
        policy = case.get("policy", "none")
        cfg = F.Config(batch=B, num_q_heads=case["hq"], num_kv_heads=case["h"],
                       head_dim=case["d"], n_sink=SINKS, recent_window=WINDOW,
                       int4_budget=-1 if policy == "none" else case["mid"],
                       middle_k_bits=case["kb"], middle_v_bits=case["vb"],
                       mid_capacity=st["cap"], policy=policy, ema_decay=EMA_DECAY,
                       v_codec="pq" if case["pq"] else "int")
        L = st["layer"] = F.TieredLayer(cfg, 1, "cuda")
        cur = st["cur"] = 1
        for name in ("sink_k", "sink_v", "recent_k", "recent_v"):
            getattr(L, name).copy_(st[name])
        for name in ("mid_k_codes", "mid_v_codes", "mid_k_scales", "mid_v_scales"):
            getattr(L, name)[cur].copy_(st[name])
        if case["pq"]:
            L.set_pq_codebook(st["codebook"])
        meta = torch.zeros_like(L.meta)
        meta[..., F.META["n_sink"]] = SINKS
        meta[..., F.META["n_mid"]] = torch.tensor(st["lens"], device="cuda").int()[:, None]
        meta[..., F.META["n_recent"]] = WINDOW - 1
        meta[..., F.META["head"]] = st["head"]
        meta[..., F.META["cur"]] = cur
        st["meta"] = meta
        st["h_mid"] = np.array(st["lens"], np.int32)
        _put_back(st)
        st["ws"] = torch.empty(F.fade_tree_ws_bytes(cfg, case["nodes"]), dtype=torch.uint8,
                               device="cuda")
    return st


def _put_back(st):
    """The layer at the counts (and scores) it had when the tokens were drafted."""
    L = st["layer"]
    L.meta.copy_(st["meta"])
    L.h_n_sink[:], L.h_n_mid[:], L.h_n_recent[:] = SINKS, st["h_mid"], WINDOW - 1
    if "policy" in st["case"] and st["case"]["policy"] != "position":
        L.sink_scores.copy_(st["sink_scores"])
        L.mid_scores[st["cur"]].copy_(st["mid_scores"])
        L.recent_scores.copy_(st["recent_scores"])


# --------------------------------------------------------------------------- one pass
def run(st):
    op = st["case"]["op"]
    if not own:
        return {"layout": _plain_layout, "norm": _plain_norm, "attention": _plain_attention,
                "commit": _plain_commit}[op](st["case"], st)
    F = st["F"]
    if op == "layout":
        F.fade_tree_layout(st["cfg"], st["parents"], st["n_nodes"], st["base"], st["mask"],
                           st["pos"])
        return [st["mask"], st["pos"]]
    if op == "norm":
        F.fade_qk_norm_rope(st["cfg"], st["table"], st["case"]["maxpos"], st["q"], st["k"],
                            st["qw"], st["kw"], st["eps"], st["pos"], st["q_rot"], st["k_rot"])
        return [st["q_rot"], st["k_rot"]]
    L = st["layer"]
    if op == "attention":
        F.fade_tree_attention(L, st["q"], st["tree_k"], st["tree_v"], st["mask"], st["n_nodes"],
                              st["out"], st["lse"], st["ws"])
        return [st["out"], st["lse"]]
    _put_back(st)
    F.fade_tree_commit(L, st["q"], st["lse"], st["tree_k"], st["tree_v"], st["path"],
                       st["n_path"], st["ws"])
    cur = st["cur"]
    return [L.recent_k, L.recent_v, L.mid_k_codes[cur], L.mid_k_scales[cur], L.mid_v_codes[cur],
            L.mid_v_scales[cur], L.sink_scores, L.mid_scores[cur], L.recent_scores,
            L.meta[..., :4]]


# --------------------------------------------------------------------------- plain forms
def _plain_layout(case, st):
    """Node by node: a node's mask is its parent's and itself, its depth its parent's plus 1."""
    par, n, base = st["parents"], st["n_nodes"], st["base"]
    B, T = par.shape
    mask = torch.zeros((B, T), dtype=torch.int64, device="cuda")
    pos = base[:, None].repeat(1, T)
    for i in range(T):
        p = par[:, i:i + 1].long()
        root = p < 0
        up = torch.where(root, 0, mask.gather(1, p.clamp(min=0)))
        dep = torch.where(root, base[:, None], pos.gather(1, p.clamp(min=0)) + 1)
        live = (n > i)[:, None]
        bit = -(1 << 63) if i == 63 else 1 << i
        mask[:, i:i + 1] = torch.where(live, up | bit, 0)
        pos[:, i:i + 1] = torch.where(live, dep, base[:, None])
    return [mask, pos]


def _plain_norm(case, st):
    d = case["d"]
    r = case["rotary"] or d
    rows = st["table"][st["pos"].long(), :r // 4]                   # [B][T][r/4][4]
    cos = rows[..., 0:2].reshape(*rows.shape[:2], 1, r // 2)
    sin = rows[..., 2:4].reshape(*rows.shape[:2], 1, r // 2)

    def one(x, w):
        x = x.float()
        y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + st["eps"]) * w.float()
        a, b = y[..., :r // 2], y[..., r // 2:r]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., r:]], -1).half()

    return [one(st["q"], st["qw"]), one(st["k"], st["kw"])]


def _ring(st):
    return [(st["head"] + i) % WINDOW for i in range(WINDOW - 1)]


def _row_kv(case, st, b, values=True):
    """Row b's keys and values in cache order, then the drafted ones: fp32 [H][N][d]."""
    n, ring = st["lens"][b], _ring(st)
    H, d = case["h"], case["d"]

    def middle(codes, scales, bits):
        q = _unpack(codes[b, :, :n], bits).float().reshape(H, n, d // GROUP, GROUP)
        return (q * scales[b, :, :n].float()[..., None]).reshape(H, n, d)

    k = torch.cat([st["sink_k"][b].float(),
                   middle(st["mid_k_codes"], st["mid_k_scales"], case["kb"]),
                   st["recent_k"][b][:, ring].float(),
                   st["tree_k"][b].transpose(0, 1).float()], 1)
    if not values:
        return k, None
    if case["pq"]:
        sub = torch.arange(d // 4, device="cuda")
        mid = st["codebook"].float()[sub, st["mid_v_codes"][b, :, :n].long()].reshape(H, n, d)
    else:
        mid = middle(st["mid_v_codes"], st["mid_v_scales"], case["vb"])
    v = torch.cat([st["sink_v"][b].float(), mid, st["recent_v"][b][:, ring].float(),
                   st["tree_v"][b].transpose(0, 1).float()], 1)
    return k, v


def _plain_attention(case, st):
    B, H, Hq, d, T = case["batch"], case["h"], case["hq"], case["d"], case["nodes"]
    G = Hq // H
    out = st["out"] if "out" in st else torch.zeros_like(st["q"])
    lse_out = st["lse"] if "out" in st else torch.zeros((B, T, Hq), device="cuda")
    for b in range(B):
        n = st["nodes"][b]
        k, v = _row_kv(case, st, b)
        k, v = k[:, :k.shape[1] - T + n], v[:, :v.shape[1] - T + n]
        q = st["q"][b, :n].float().reshape(n, H, G, d).permute(1, 0, 2, 3).reshape(H, n * G, d)
        s = (q @ k.transpose(1, 2)) * (1.0 / math.sqrt(d))
        seen = (st["mask"][b, :n, None] >> torch.arange(n, device="cuda")) & 1
        tail = s[..., s.shape[-1] - n:].reshape(H, n, G, n)
        tail.masked_fill_((seen == 0)[None, :, None, :], -math.inf)
        m = s.amax(-1, keepdim=True)
        e = (s - m).exp_()
        z = e.sum(-1, keepdim=True)
        o = (e @ v) / z
        lse = (m + z.log())[..., 0]
        out[b, :n] = o.reshape(H, n, G, d).permute(1, 0, 2, 3).reshape(n, Hq, d).half()
        lse_out[b, :n] = lse.reshape(H, n, G).permute(1, 0, 2).reshape(n, Hq)
    return [out, lse_out]


def _plain_commit(case, st):
    B, H, Hq, d, T = case["batch"], case["h"], case["hq"], case["d"], case["nodes"]
    G = Hq // H
    ring, free = _ring(st), (st["head"] + WINDOW - 1) % WINDOW
    sink_sc, mid_sc = st["sink_scores"].clone(), st["mid_scores"].clone()
    rec_sc = st["recent_scores"].clone()
    meta = torch.zeros((B, H, 4), dtype=torch.int32, device="cuda")
    for b in range(B):
        nodes, n = st["paths"][b], st["lens"][b]
        a = len(nodes)
        new_sc = torch.zeros((H, a), device="cuda")
        if case["policy"] != "position":
            k, _ = _row_kv(case, st, b, values=False)
            held = k.shape[1] - T
            k = torch.cat([k[:, :held], k[:, held:][:, nodes]], 1)
            q = st["q"][b, nodes].float().reshape(a, H, G, d).permute(1, 0, 2, 3)
            s = torch.einsum("hagd,hnd->hagn", q, k) * (1.0 / math.sqrt(d))
            lse = st["lse"][b, nodes].reshape(a, H, G).permute(1, 0, 2)
            p = (s - lse[..., None]).exp().sum(2)                      # [H][a][held + a]
            order = torch.arange(a, device="cuda")
            p[:, :, held:].masked_fill_(order[None, :] > order[:, None], 0.0)
            old = torch.cat([sink_sc[b], mid_sc[b, :, :n], rec_sc[b][:, ring], new_sc], 1)
            for i in range(a):
                if case["policy"] == "h2o":
                    old = old + p[:, i]
                else:
                    old[:, :held + i + 1] = (EMA_DECAY * old[:, :held + i + 1]
                                             + (1 - EMA_DECAY) * p[:, i, :held + i + 1])
            sink_sc[b], mid_sc[b, :, :n] = old[:, :SINKS], old[:, SINKS:SINKS + n]
            rec_sc[b][:, ring] = old[:, SINKS + n:held]
            new_sc = old[:, held:]
        # the oldest a - 1 tokens of the window are demoted, the accepted ones take their slots
        out = ring[:a - 1]
        if out:
            for src, codes, scales, bits in (
                    ("recent_k", st["mid_k_codes"], st["mid_k_scales"], case["kb"]),
                    ("recent_v", st["mid_v_codes"], st["mid_v_scales"], case["vb"])):
                q, s = _quantize(st[src][b][:, out], bits)
                codes[b, :, n:n + a - 1], scales[b, :, n:n + a - 1] = _pack(q, bits), s
            mid_sc[b, :, n:n + a - 1] = rec_sc[b][:, out]
        slots = [free] + out
        st["recent_k"][b][:, slots] = st["tree_k"][b, nodes].transpose(0, 1)
        st["recent_v"][b][:, slots] = st["tree_v"][b, nodes].transpose(0, 1)
        rec_sc[b][:, slots] = new_sc
        meta[b] = torch.tensor([SINKS, n + a - 1, WINDOW, (st["head"] + a - 1) % WINDOW],
                               dtype=torch.int32, device="cuda")
    return [st["recent_k"], st["recent_v"], st["mid_k_codes"], st["mid_k_scales"],
            st["mid_v_codes"], st["mid_v_scales"], sink_sc, mid_sc, rec_sc, meta]


# --------------------------------------------------------------------------- definitions
def exact(case, seed):
    """What run() returns, from the definitions in 64 bits (whole numbers as they are)."""
    st = _inputs(case, seed)
    return {"layout": _exact_layout, "norm": _exact_norm, "attention": _exact_attention,
            "commit": _exact_commit}[case["op"]](case, st)


def _exact_layout(case, st):
    par, n = st["parents"].cpu().tolist(), st["n_nodes"].cpu().tolist()
    base = st["base"].cpu().tolist()
    mask = np.zeros((case["batch"], case["nodes"]), np.uint64)
    pos = np.zeros((case["batch"], case["nodes"]), np.int32)
    for b, row in enumerate(par):
        pos[b] = base[b]
        for i in range(n[b]):
            chain, j = [i], row[i]
            while j >= 0:
                chain.append(j)
                j = row[j]
            mask[b, i] = sum(1 << c for c in chain)
            pos[b, i] = base[b] + len(chain) - 1
    return [torch.from_numpy(mask.view(np.int64)).cuda(), torch.from_numpy(pos).cuda()]


def _exact_norm(case, st):
    d = case["d"]
    r = case["rotary"] or d
    t = st["table"].double()[st["pos"].long()]
    outs = []
    for x, w in ((st["q"], st["qw"]), (st["k"], st["kw"])):
        y = x.double()
        y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / d + st["eps"]) * w.double()
        z = torch.view_as_complex(torch.stack([y[..., :r // 2], y[..., r // 2:r]], -1).contiguous())
        turn = torch.complex(t[:, :, :r // 4, 0:2].flatten(2), t[:, :, :r // 4, 2:4].flatten(2))
        z = z * turn[:, :, None]
        outs.append(torch.cat([z.real, z.imag, y[..., r:]], -1))
    return outs


def _exact_codes(codes, bits, d):
    """Signed codes of packed rows [N][bytes] by arithmetic on the bytes."""
    c = torch.arange(d, device="cuda")
    per = 8 // bits
    u = torch.div(codes.long()[:, c // per], 2 ** (bits * (c % per)), rounding_mode="floor")
    u = u % (2 ** bits)
    return (u - (2 ** bits) * (u >= 2 ** (bits - 1)).long()).double()


def _exact_unit(case, st, b, h, nodes):
    """Keys and values of unit (b, h): cache order, then the drafted nodes; float64."""
    d, n = case["d"], st["lens"][b]
    ring = _ring(st)
    rep = lambda s: s.double().repeat_interleave(GROUP, -1)
    km = _exact_codes(st["mid_k_codes"][b, h, :n], case["kb"], d) * rep(st["mid_k_scales"][b, h, :n])
    if case["pq"]:
        idx = st["mid_v_codes"][b, h, :n].long()
        vm = torch.stack([st["codebook"][s].double()[idx[:, s]] for s in range(d // 4)], 1)
        vm = vm.reshape(n, d)
    else:
        vm = (_exact_codes(st["mid_v_codes"][b, h, :n], case["vb"], d)
              * rep(st["mid_v_scales"][b, h, :n]))
    cat = lambda s, m, r, t: torch.cat([s[b, h].double(), m, r[b, h, ring].double(),
                                        t[b, nodes, h].double()])
    return (cat(st["sink_k"], km, st["recent_k"], st["tree_k"]),
            cat(st["sink_v"], vm, st["recent_v"], st["tree_v"]))


def _exact_attention(case, st):
    B, H, Hq, d, T = case["batch"], case["h"], case["hq"], case["d"], case["nodes"]
    G = Hq // H
    out = torch.zeros((B, T, Hq, d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, T, Hq), dtype=torch.float64, device="cuda")
    for b in range(B):
        n = st["nodes"][b]
        bits = st["mask"][b].cpu().numpy().view(np.uint64)
        seen = torch.tensor([[bool((int(bits[i]) >> j) & 1) for j in range(n)] for i in range(n)],
                            device="cuda")
        for h in range(H):
            k, v = _exact_unit(case, st, b, h, list(range(n)))
            see = torch.ones((n, k.shape[0]), dtype=torch.bool, device="cuda")
            see[:, k.shape[0] - n:] = seen
            for g in range(G):
                s = st["q"][b, :n, h * G + g].double() @ k.T / math.sqrt(d)
                s = torch.where(see, s, torch.full_like(s, -math.inf))
                out[b, :n, h * G + g] = torch.softmax(s, -1) @ v
                lse[b, :n, h * G + g] = torch.logsumexp(s, -1)
    return [out, lse]


def _exact_commit(case, st):
    B, H, Hq, d = case["batch"], case["h"], case["hq"], case["d"]
    G, ring = Hq // H, _ring(st)
    free = (st["head"] + WINDOW - 1) % WINDOW
    scores = [st[n].double() for n in ("sink_scores", "mid_scores", "recent_scores")]
    meta = torch.zeros((B, H, 4), dtype=torch.int32, device="cuda")
    decay, gain = (1.0, 1.0) if case["policy"] == "h2o" else (EMA_DECAY, 1 - EMA_DECAY)
    for b in range(B):
        nodes, n = st["paths"][b], st["lens"][b]
        a = len(nodes)
        slots = [free] + ring[:a - 1]
        for h in range(H):
            new = torch.zeros(a, dtype=torch.float64, device="cuda")
            if case["policy"] != "position":
                k, _ = _exact_unit(case, st, b, h, nodes)
                old = torch.cat([scores[0][b, h], scores[1][b, h, :n], scores[2][b, h, ring], new])
                held = old.numel() - a
                for i, node in enumerate(nodes):
                    heads = slice(h * G, (h + 1) * G)
                    s = st["q"][b, node, heads].double() @ k[:held + i + 1].T / math.sqrt(d)
                    p = torch.exp(s - st["lse"][b, node, heads].double()[:, None]).sum(0)
                    old[:held + i + 1] = decay * old[:held + i + 1] + gain * p
                scores[0][b, h], scores[1][b, h, :n] = old[:SINKS], old[SINKS:SINKS + n]
                scores[2][b, h, ring] = old[SINKS + n:held]
                new = old[held:]
            for i in range(a - 1):
                for src, codes, scales, bits in (
                        ("recent_k", "mid_k_codes", "mid_k_scales", case["kb"]),
                        ("recent_v", "mid_v_codes", "mid_v_scales", case["vb"])):
                    qmax = 2 ** (bits - 1) - 1
                    x = st[src][b, h, ring[i]].double().reshape(-1, GROUP)
                    s = (x.abs().max(1).values / qmax).half()
                    q = torch.round(x / s.double()[:, None]).clamp(-qmax, qmax).long().flatten()
                    per = 8 // bits
                    w = 2 ** (bits * torch.arange(per, device="cuda"))
                    st[codes][b, h, n + i] = ((q % 2 ** bits).reshape(-1, per) * w).sum(1).byte()
                    st[scales][b, h, n + i] = s
                scores[1][b, h, n + i] = scores[2][b, h, ring[i]]
            for i, node in enumerate(nodes):
                st["recent_k"][b, h, slots[i]] = st["tree_k"][b, node, h]
                st["recent_v"][b, h, slots[i]] = st["tree_v"][b, node, h]
                scores[2][b, h, slots[i]] = new[i]
        meta[b] = torch.tensor([SINKS, n + a - 1, WINDOW, (st["head"] + a - 1) % WINDOW],
                               dtype=torch.int32, device="cuda")
    return [st["recent_k"].double(), st["recent_v"].double(), st["mid_k_codes"],
            st["mid_k_scales"].double(), st["mid_v_codes"], st["mid_v_scales"].double(), *scores,
            meta]
