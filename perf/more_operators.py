"""What is measured of the operators of a request's two ends: cases, inputs, plain forms, definitions.

* ``attention``: a prompt's (or a chunk's, or one token's) causal attention, over every earlier token
  or over a sliding window and the first tokens that stay visible (``fade_prompt_attention``);
* ``mass``: the column sums of that attention, from its log-sum-exp: the importance scores that a
  prompt starts with (``fade_prompt_mass``);
* ``verify``: which drafted tokens are accepted under the target's and the drafter's probabilities
  and given random numbers, and the token after them (``fade_tree_verify``).

``own`` false computes them with elementary torch operations; ``own`` true calls the framework.
"""

import math

import numpy as np
import torch

own = False

MASKED_VOCAB = 0.002   # share of the vocabulary whose logits are -inf (padding, forbidden tokens)


# --------------------------------------------------------------------------- cases
def _prompt(name, op, batch, hq, h, d, n_q, n_kv, sink=0, window=0, ragged=False, heads_first=False):
    """n_q queries a row, the last of its n_kv tokens. window 0: every earlier token is seen.
    ragged: rows of n/2 .. n tokens. heads_first: [rows][heads][tokens][d], as prompts lie; otherwise
    slices of a fused projection's output."""
    return {"name": name, "op": op, "batch": batch, "hq": hq, "h": h, "d": d, "n_q": n_q,
            "n_kv": n_kv, "sink": sink, "window": window, "ragged": ragged,
            "heads_first": heads_first}


def _verify(name, batch, nodes, vocab, tree, mode, dtype, depth):
    """mode: "greedy", "certain" (the drafts have no probabilities of their own) or "sampled".
    depth: the longest accepted path (rows keep 1 .. depth nodes)."""
    return {"name": name, "op": "verify", "batch": batch, "nodes": nodes, "vocab": vocab,
            "tree": tree, "mode": mode, "dtype": dtype, "depth": depth}


def listed():
    return [
        # one request's new token over a cache of 4096 that nothing is dropped from: latency
        _prompt("attention_one_token", "attention", 1, 16, 2, 128, 1, 4096),
        # a batch of single tokens over 4 sinks and the last 4160 of 8191 tokens
        _prompt("attention_tokens_window", "attention", 64, 32, 8, 128, 1, 8191, 4, 4160),
        # short prompts of different lengths
        _prompt("attention_short_prompts", "attention", 8, 32, 8, 64, 2048, 2048, ragged=True,
                heads_first=True),
        # one long prompt of an odd length
        _prompt("attention_prompt", "attention", 1, 32, 8, 128, 16383, 16383),
        # long prompts under a window and sinks
        _prompt("attention_prompt_window", "attention", 2, 32, 8, 128, 32768, 32768, 4, 4160,
                heads_first=True),
        # a chunk of a long prompt in a batch of uneven rows
        _prompt("attention_chunk", "attention", 4, 32, 8, 128, 509, 65536, ragged=True),
        # the scores of one short prompt: latency
        _prompt("mass_one_prompt", "mass", 1, 8, 2, 64, 511, 511, heads_first=True),
        # the scores of a batch of prompts that will be evicted from
        _prompt("mass_prompts", "mass", 8, 32, 8, 64, 2048, 2048, ragged=True, heads_first=True),
        # the scores of a long prompt under a window and sinks
        _prompt("mass_window", "mass", 1, 32, 8, 128, 32768, 32768, 4, 4160),
        # a chain of drafts for one request, greedy: latency
        _verify("verify_greedy_chain", 1, 5, 32000, "chain", "greedy", "float16", 5),
        # chains of drafts without probabilities, an odd vocabulary
        _verify("verify_chains", 16, 8, 50257, "chain", "certain", "float32", 8),
        # trees of sampled drafts for a full batch
        _verify("verify_trees", 64, 16, 128256, "tree", "sampled", "bfloat16", 6),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "mass", "verify"])
    if op == "verify":
        mode = rng.choice(["greedy", "certain", "sampled", "sampled"])
        vocab = _log(rng, 1000, 150000)
        nodes = _log(rng, 1, 64)
        batch = _log(rng, 1, max(1, min(128, 120000000 // (nodes * vocab))))
        c = _verify("", batch, nodes, vocab, rng.choice(["chain", "tree", "tree"]), mode,
                    rng.choice(["float16", "bfloat16", "float32"]), rng.randint(1, min(nodes, 8)))
        del c["name"]
        return c
    while True:
        h = rng.choice([1, 2, 4, 8])
        n_kv = _log(rng, 1, 65536)
        n_q = rng.choice([n_kv, _log(rng, 1, n_kv), 1 if op == "attention" else n_kv])
        window = rng.choice([0, _log(rng, 1, 8192)])
        c = _prompt("", op, _log(rng, 1, 64), h * rng.choice([1, 2, 4, 8]), h, rng.choice([64, 128]), n_q,
                    n_kv, rng.randint(0, 200) if window else 0, window, rng.random() < 0.5,
                    rng.random() < 0.5)
        w = work(c)
        # no more than the largest listed case, padding included
        padded = c["batch"] * c["hq"] * n_q * min(n_kv, (window or n_kv) + n_q)
        if w["flops"] < 4e12 and w["bytes"] < 1.5e9 and padded * c["d"] < 1.2e12:
            del c["name"]
            return c


def _lens(case):
    """Every row's queries and tokens (part of the case: the same for every seed)."""
    B, nq, nk = case["batch"], case["n_q"], case["n_kv"]
    kv = np.full(B, nk, np.int32)
    if case["ragged"]:
        rng = np.random.default_rng(nk * 31 + B)
        kv = rng.integers(max(1, nk // 2), nk + 1, B).astype(np.int32)
        kv[0] = nk
    return np.minimum(kv, nq).astype(np.int32), kv


def _seen(case, i):
    """Tokens that a query at position i sees (i: an array)."""
    i = np.asarray(i, np.int64)
    if not case["window"]:
        return i + 1
    first = np.maximum(i - case["window"] + 1, 0)
    return i + 1 - first + np.minimum(first, case["sink"])


def work(case):
    B = case["batch"]
    if case["op"] == "verify":
        size = 4 if case["dtype"] == "float32" else 2
        rows = sum(len(p) for p in _plan(case)[1])
        side = {"greedy": 1, "certain": 1, "sampled": 2}[case["mode"]]
        noise = 0 if case["mode"] == "greedy" else 4 * B * case["vocab"]
        return {"bytes": rows * side * case["vocab"] * size + noise + 12 * B * case["nodes"] + 8 * B,
                "flops": 0}
    hq, h, d = case["hq"], case["h"], case["d"]
    q_len, kv_len = _lens(case)
    pairs = keys = 0
    for a, n in zip(q_len.tolist(), kv_len.tolist()):
        pairs += int(_seen(case, np.arange(n - a, n)).sum())
        first = max(n - a - case["window"] + 1, 0) if case["window"] else 0
        keys += n - first + min(first, case["sink"])
    tokens = int(q_len.sum())
    if case["op"] == "mass":
        return {"bytes": tokens * hq * (2 * d + 4) + keys * h * 2 * d + B * h * case["n_kv"] * 4,
                "flops": 2 * d * hq * pairs}
    return {"bytes": tokens * hq * (4 * d + 4) + keys * h * 4 * d, "flops": 4 * d * hq * pairs}


# --------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(shape, g, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).half()


def _prompt_inputs(case, seed):
    """Rotated queries and keys and the values of a layer; a channel of large keys, as models have."""
    g = _gen(seed)
    B, nq, nk, hq, h, d = (case[x] for x in ("batch", "n_q", "n_kv", "hq", "h", "d"))
    st = {}
    if case["heads_first"]:
        q = _normal((B, hq, nq, d), g).transpose(1, 2)
        k, v = (_normal((B, h, nk, d), g).transpose(1, 2) for _ in range(2))
    else:
        q = _normal((B, nq, hq, d), g)
        kv = _normal((B, nk, 2 * h, d), g)
        k, v = kv[:, :, :h], kv[:, :, h:]
    k[..., int(torch.randint(d, (1,), generator=g, device="cuda"))] *= 6
    st["q"], st["k"], st["v"] = q, k, v
    st["q_len"], st["kv_len"] = _lens(case)
    if case["op"] == "attention":
        st["out"] = torch.zeros((B, nq, hq, d), dtype=torch.float16, device="cuda")
        st["lse"] = torch.zeros((B, nq, hq), device="cuda")
    else:   # what the attention call left with the program
        st["lse"] = torch.zeros((B, nq, hq), device="cuda")
        _plain_attention(case, st)
        st["mass"] = torch.zeros((B, h, nk), device="cuda")
    return st


def _plan(case):
    """Parents of every row's nodes and the path that is accepted (part of the case)."""
    B, T = case["batch"], case["nodes"]
    rng = np.random.default_rng(T * 977 + B)
    par = np.zeros((B, T), np.int32)
    if case["tree"] == "chain":
        par[:] = np.arange(T) - 1
    else:
        par[:, 0] = -1
        for i in range(1, T):
            par[:, i] = rng.integers(max(0, (i - 1) // 3), i, B)
    paths = []
    for b in range(B):
        path, want = [0], int(rng.integers(1, case["depth"] + 1))
        while len(path) < want:
            kids = np.nonzero(par[b] == path[-1])[0]
            kids = kids[kids > path[-1]]
            if not len(kids):
                break
            path.append(int(kids[0] if rng.random() < 0.7 else rng.choice(kids)))
        paths.append(path)
    return par, paths


def _race(weights, g):
    """A draw in proportion to the weights [rows][V]."""
    e = torch.empty(weights.shape, device="cuda").exponential_(generator=g)
    return (weights / e).argmax(-1)


def _verify_inputs(case, seed):
    """Target and drafter logits, tokens and uniform numbers under which the planned paths are what
    is accepted: a kept draft is drawn from what both distributions share, a refused one from what
    the drafter has too much of, and its uniform number on that side of the ratio."""
    g = _gen(seed)
    B, T, V, mode = case["batch"], case["nodes"], case["vocab"], case["mode"]
    dt = getattr(torch, case["dtype"])
    par, paths = _plan(case)
    st = {"parents": torch.from_numpy(par).cuda(), "paths": paths}
    target = torch.randn((B, T, V), generator=g, device="cuda").mul_(4)
    draft = None
    if mode == "sampled":
        draft = torch.randn((B, T, V), generator=g, device="cuda").add_(target).to(dt)
    off = torch.rand(V, generator=g, device="cuda") < MASKED_VOCAB
    target = target.to(dt).masked_fill_(off, -math.inf)
    if draft is not None:
        draft.masked_fill_(off, -math.inf)
    st["target"], st["draft"] = target, draft
    st["temperature"] = 0.7 + 0.6 * torch.rand(B, generator=g, device="cuda")
    tokens = torch.randint(V, (B, T), generator=g, device="cuda").int()
    u = torch.rand((B, T), generator=g, device="cuda")
    keep = np.zeros((B, T), bool)
    for b, p in enumerate(paths):
        keep[b, p] = True
    keep = torch.from_numpy(keep).cuda()
    rows = torch.arange(B, device="cuda")
    cur = torch.zeros(B, dtype=torch.long, device="cuda")
    p, q, a, w = _fresh(case, st, cur)
    gone = torch.zeros((B, V), dtype=torch.bool, device="cuda")
    for i in range(1, T):
        here = st["parents"][:, i] == cur
        yes = here & keep[:, i]
        r = (p - a[:, None] * q).clamp_(min=0)
        if mode == "greedy":
            best = p.argmax(-1)
            x = torch.where(yes, best, (best + 1 + tokens[:, i] % (V - 1)) % V)
            ratio = torch.zeros(B, device="cuda")
        elif mode == "certain":
            r = r.masked_fill(gone, 0.0)
            x = _race(r, g)
            ratio = r[rows, x] / w
        else:
            x = torch.where(yes, _race(torch.minimum(q * w[:, None], r), g),
                            _race((q * w[:, None] - r).clamp_(min=0), g))
            ratio = (r[rows, x] / (q[rows, x] * w)).clamp_(max=1)
        x = torch.where(here, x, tokens[:, i].long())
        tokens[:, i] = x.int()
        f = u[:, i]
        there = torch.where(yes, 0.98 * f * ratio, ratio + (1 - ratio) * (0.02 + 0.97 * f))
        u[:, i] = torch.where(here, there, f).clamp_(0, 0.9999)
        # what the walk knows after this node
        no = here & ~keep[:, i]
        if mode == "certain":
            gone[rows, x] |= no
            w = torch.where(no, w - r[rows, x], w)
        elif mode == "sampled":
            a = torch.where(no, a + w, a)
            w = torch.where(no, (p - a[:, None] * q).clamp_(min=0).sum(-1), w)
        if bool(yes.any()):
            cur = torch.where(yes, i, cur)
            p2, q2, a2, w2 = _fresh(case, st, cur)
            p, q = torch.where(yes[:, None], p2, p), torch.where(yes[:, None], q2, q)
            a, w = torch.where(yes, a2, a), torch.where(yes, w2, w)
            gone &= ~yes[:, None]
    st["tokens"], st["u"] = tokens, u
    if mode == "greedy":
        st["u"] = st["temperature"] = st["noise"] = None
    else:
        st["noise"] = torch.empty((B, V), device="cuda").exponential_(generator=g)
    return st


def prepare(case, seed):
    st = _verify_inputs(case, seed) if case["op"] == "verify" else _prompt_inputs(case, seed)
    st["case"] = case
    B = case["batch"]
    if case["op"] == "verify":
        empty = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
        st["path"], st["n_path"], st["next"] = empty(B, case["nodes"]), empty(B), empty(B)
    if own:
        from tiered_mixed_precision_gb300 import fade as F

        st["F"] = F
        shape = {"num_q_heads": 8, "num_kv_heads": 2, "head_dim": 64}
        if case["op"] != "verify":
            shape = {"num_q_heads": case["hq"], "num_kv_heads": case["h"], "head_dim": case["d"]}
        cfg = st["cfg"] = F.Config(batch=B, mid_capacity=64, **shape)
        if case["op"] != "verify":
            st["ws"] = torch.empty(F.fade_prompt_ws_bytes(cfg, case["n_q"], case["n_kv"]),
                                   dtype=torch.uint8, device="cuda")
    return st


# --------------------------------------------------------------------------- one pass
def run(st):
    case = st["case"]
    if not own:
        return {"attention": _plain_attention, "mass": _plain_mass,
                "verify": _plain_verify}[case["op"]](case, st)
    F = st["F"]
    if case["op"] == "verify":
        F.fade_tree_verify(st["cfg"], st["parents"], None, st["tokens"], st["target"], None,
                           st["draft"], None, st["temperature"], st["u"], st["noise"], st["path"],
                           st["n_path"], st["next"])
        return [st["path"], st["n_path"], st["next"]]
    see = dict(q_len=st["q_len"], kv_len=st["kv_len"], n_sink=case["sink"], window=case["window"],
               ws=st["ws"])
    if case["op"] == "attention":
        F.fade_prompt_attention(st["cfg"], st["q"], st["k"], st["v"], st["out"], st["lse"], **see)
        return [st["out"], st["lse"]]
    F.fade_prompt_mass(st["cfg"], st["q"], st["k"], st["lse"], st["mass"], **see)
    return [st["mass"]]


# --------------------------------------------------------------------------- plain forms
def _blocks(case, st):
    """Blocks of queries small enough for their logits: (i0, i1, the tokens they may see, logits
    fp32 [B][H][G][queries][tokens] with -inf where a query does not see a token)."""
    B, nq, nk, hq, h, d = (case[x] for x in ("batch", "n_q", "n_kv", "hq", "h", "d"))
    W, sink = case["window"], case["sink"]
    q_len = torch.from_numpy(st["q_len"]).cuda().long()
    kv_len = torch.from_numpy(st["kv_len"]).cuda().long()
    far = int((st["kv_len"] - st["q_len"]).max())        # the first query's position at most
    near = int((st["kv_len"] - st["q_len"]).min())
    wide = min(nk, W + far - near + 1024) if W else nk
    step = max(1, min(nq, int(4e8) // (B * hq * wide)))
    keys = st["k"].transpose(1, 2)                       # [B][H][nk][d]
    for i0 in range(0, nq, step):
        i1 = min(nq, i0 + step)
        lo = max(0, near + i0 - W + 1) if W else 0
        hi = min(nk, far + i1)
        cols = torch.arange(lo, hi, device="cuda")
        k = keys[:, :, lo:hi]
        if W and sink and lo:
            cols = torch.cat([torch.arange(min(sink, lo), device="cuda"), cols])
            k = torch.cat([keys[:, :, :min(sink, lo)], k], 2)
        k = k.float()
        q = st["q"][:, i0:i1].float().reshape(B, i1 - i0, h, hq // h, d).permute(0, 2, 3, 1, 4)
        s = (q.reshape(B, h, -1, d) @ k.transpose(2, 3)).mul_(1 / math.sqrt(d))
        s = s.reshape(B, h, hq // h, i1 - i0, -1)
        i = torch.arange(i0, i1, device="cuda")
        at = (kv_len - q_len)[:, None] + i               # [B][queries]
        see = cols <= at[..., None]
        if W:
            see &= (cols < sink) | (cols > at[..., None] - W)
        live = i < q_len[:, None]
        yield i0, i1, cols, s.masked_fill_(~(see & live[..., None])[:, None, None], -math.inf), live


def _plain_attention(case, st):
    B, hq, d = case["batch"], case["hq"], case["d"]
    values = st["v"].transpose(1, 2) if "out" in st else None
    for i0, i1, cols, s, live in _blocks(case, st):
        m = s.amax(-1, keepdim=True).clamp_(min=-1e30)
        e = s.sub_(m).exp_()
        z = e.sum(-1, keepdim=True)
        back = lambda x: x.permute(0, 3, 1, 2, 4).reshape(B, i1 - i0, hq, -1)
        lse = back(m + z.log())[..., 0]
        st["lse"][:, i0:i1] = torch.where(live[..., None], lse, st["lse"][:, i0:i1])
        if values is None:
            continue
        o = (e.flatten(2, 3) @ values[:, :, cols].float()).reshape(*e.shape[:4], d) / z
        st["out"][:, i0:i1] = torch.where(live[..., None, None], back(o).half(), st["out"][:, i0:i1])
    return [st.get("out"), st["lse"]]


def _plain_mass(case, st):
    B, h, hq = case["batch"], case["h"], case["hq"]
    st["mass"].zero_()
    for i0, i1, cols, s, live in _blocks(case, st):
        lse = st["lse"][:, i0:i1].reshape(B, i1 - i0, h, hq // h).permute(0, 2, 3, 1)
        st["mass"][:, :, cols] += s.sub_(lse[..., None]).exp_().sum((2, 3))
    return [st["mass"]]


def _probs(logits, st):
    """fp32 probabilities of logits [B][V] at every row's temperature."""
    x = logits.float()
    if st["temperature"] is not None:
        x = x / st["temperature"][:, None]
    return torch.softmax(x, -1)


def _fresh(case, st, node):
    """The distributions after every row's node, nothing refused there yet: target, drafter, what the
    refused drafts took (in drafter's units) and what is left."""
    rows = torch.arange(case["batch"], device="cuda")
    p = _probs(st["target"][rows, node], st)
    q = _probs(st["draft"][rows, node], st) if st["draft"] is not None else torch.zeros_like(p)
    return p, q, torch.zeros(case["batch"], device="cuda"), torch.ones(case["batch"], device="cuda")


def _plain_verify(case, st):
    """Node by node: one whose parent is the path's end is kept if u q w < max(p - a q, 0); a refused
    one adds w to a, and w becomes the sum of max(p - a q, 0). Drafts without probabilities: kept if
    u w < p, a refused one's p leaves w. At the end the greatest max(p - a q, 0) / noise is next."""
    B, T, V, mode = (case[x] for x in ("batch", "nodes", "vocab", "mode"))
    rows = torch.arange(B, device="cuda")
    cur = torch.zeros(B, dtype=torch.long, device="cuda")
    path = torch.zeros((B, T), dtype=torch.int32, device="cuda")
    n = torch.ones(B, dtype=torch.long, device="cuda")
    if mode == "greedy":
        best = st["target"].argmax(-1)
        for i in range(1, T):
            yes = (st["parents"][:, i] == cur) & (st["tokens"][:, i] == best[rows, cur])
            path[rows, n.clamp(max=T - 1)] = torch.where(yes, i, path[rows, n.clamp(max=T - 1)])
            cur, n = torch.where(yes, i, cur), n + yes
        return [path, n.int(), best[rows, cur].int()]
    p, q, a, w = _fresh(case, st, cur)
    for i in range(1, T):
        here = st["parents"][:, i] == cur
        x = st["tokens"][:, i].long()
        r = (p[rows, x] - a * q[rows, x]).clamp_(min=0)
        yes = here & (st["u"][:, i] * w * (q[rows, x] if mode == "sampled" else 1.0) < r)
        no = here & ~yes
        if mode == "sampled":
            a = torch.where(no, a + w, a)
            w = torch.where(no, (p - a[:, None] * q).clamp_(min=0).sum(-1), w)
        else:
            w = torch.where(no, w - r, w)
            p[rows, x] = torch.where(no, 0.0, p[rows, x])
        path[rows, n.clamp(max=T - 1)] = torch.where(yes, i, path[rows, n.clamp(max=T - 1)])
        cur, n = torch.where(yes, i, cur), n + yes
        p2, q2, a2, w2 = _fresh(case, st, cur)
        p, q = torch.where(yes[:, None], p2, p), torch.where(yes[:, None], q2, q)
        a, w = torch.where(yes, a2, a), torch.where(yes, w2, w)
    nxt = ((p - a[:, None] * q).clamp_(min=0) / st["noise"]).argmax(-1)
    return [path, n.int(), nxt.int()]


# --------------------------------------------------------------------------- definitions
def exact(case, seed):
    """What run() returns, from the definitions in 64 bits (whole numbers as they are)."""
    if case["op"] == "verify":
        return _exact_verify(case, _verify_inputs(case, seed))
    st = _prompt_inputs(case, seed)
    B, nq, nk, hq, h, d = (case[x] for x in ("batch", "n_q", "n_kv", "hq", "h", "d"))
    out = torch.zeros((B, nq, hq, d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, nq, hq), dtype=torch.float64, device="cuda")
    mass = torch.zeros((B, h, nk), dtype=torch.float64, device="cuda")
    sink, W = case["sink"], case["window"] or nk
    for b in range(B):
        a, n = int(st["q_len"][b]), int(st["kv_len"][b])
        for i0 in range(0, a, 2048):
            i1 = min(a, i0 + 2048)
            pos = torch.arange(n - a + i0, n - a + i1, device="cuda")[:, None]
            lo = max(0, int(pos[0, 0]) - W + 1)
            j = torch.cat([torch.arange(min(sink, lo), device="cuda"),
                           torch.arange(lo, int(pos[-1, 0]) + 1, device="cuda")])
            away = pos - j
            see = (away >= 0) & ((away < W) | (j < sink))
            for x in range(hq):
                k, v = st["k"][b, j, x * h // hq].double(), st["v"][b, j, x * h // hq].double()
                s = st["q"][b, i0:i1, x].double() @ k.T / math.sqrt(d)
                s = torch.where(see, s, -math.inf)
                if case["op"] == "mass":
                    p = torch.exp(s - st["lse"][b, i0:i1, x].double()[:, None])
                    mass[b, x * h // hq].index_add_(0, j, p.sum(0))
                else:
                    out[b, i0:i1, x] = torch.softmax(s, -1) @ v
                    lse[b, i0:i1, x] = torch.logsumexp(s, -1)
    return [mass] if case["op"] == "mass" else [out, lse]


def _exact_verify(case, st):
    """Row by row: the residual distribution after every refused draft, normalised each time."""
    B, T, mode = case["batch"], case["nodes"], case["mode"]
    path = torch.zeros((B, T), dtype=torch.int32, device="cuda")
    n_path, nxt = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
    par, tokens = st["parents"].cpu().tolist(), st["tokens"].cpu().tolist()
    u = None if mode == "greedy" else st["u"].double().cpu().tolist()
    for b in range(B):
        at, kept = 0, [0]
        while True:
            x = st["target"][b, at].double()
            if mode == "greedy":
                best = int((x == x.max()).nonzero()[0])
                child = next((i for i in range(at + 1, T) if par[b][i] == at and tokens[b][i] == best),
                             None)
            else:
                t = st["temperature"][b].double()
                r = torch.softmax(x / t, -1)
                q = torch.softmax(st["draft"][b, at].double() / t, -1) if mode == "sampled" else None
                child = None
                for i in range(at + 1, T):
                    if par[b][i] != at:
                        continue
                    tok = tokens[b][i]
                    share = float(q[tok]) if mode == "sampled" else 1.0
                    if u[b][i] * share < float(r[tok]):
                        child = i
                        break
                    if mode == "sampled":
                        r = torch.relu(r - q)
                    else:
                        r[tok] = 0.0
                    r = r / r.sum()
            if child is None:
                break
            kept.append(child)
            at = child
        path[b, :len(kept)] = torch.tensor(kept, dtype=torch.int32, device="cuda")
        n_path[b] = len(kept)
        nxt[b] = best if mode == "greedy" else int((r / st["noise"][b].double()).argmax())
    return [path, n_path, nxt]
