"""Drafted-token entry points without a GPU: argument, shape and capacity errors, returned before
anything is enqueued (the layers' buffers are host memory; no kernel is launched)."""

import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def T():
    from tiered_mixed_precision_gb300 import build

    build.build()
    import tiered_mixed_precision_gb300 as T

    return T


class _S:  # a stream handle that is never used (no launch happens)
    cuda_stream = 0


def _layer(T, **kw):
    base = dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=64, n_sink=2, recent_window=4,
                int4_budget=3, middle_k_bits=4, middle_v_bits=2, mid_capacity=8, policy="h2o")
    base.update(kw)
    return T.TieredLayer(T.Config(**base), 32, device="cpu")


def _args(L, n=5, ws=None):
    c = L.cfg
    z = lambda *s, dt=torch.float16: torch.zeros(s, dtype=dt)
    return dict(q_rot=z(c.batch, n, c.num_q_heads, c.head_dim),
                tree_k=z(c.batch, n, c.num_kv_heads, c.head_dim),
                tree_v=z(c.batch, n, c.num_kv_heads, c.head_dim),
                lse=z(c.batch, n, c.num_q_heads, dt=torch.float32),
                ws=z(1 << 20 if ws is None else ws, dt=torch.uint8))


def _raises(T, status, fn, *a, **kw):
    with pytest.raises(T.FadeError) as e:
        fn(*a, stream=_S(), **kw)
    assert e.value.status == status, str(e.value)
    return str(e.value)


def _attend(T, L, a, mask=None, n_nodes=None, **kw):
    a = {**a, **kw}
    B, n = a["q_rot"].shape[:2]
    mask = torch.zeros((B, n), dtype=torch.int64) if mask is None else mask
    out = torch.zeros_like(a["q_rot"])
    T.fade_tree_attention(L, a["q_rot"], a["tree_k"], a["tree_v"], mask, n_nodes, out, a["lse"],
                          a["ws"], stream=_S())


def _commit(T, status, L, a, lens, path=None, **kw):
    a = {**a, **kw}
    if path is None:
        path = torch.zeros(a["q_rot"].shape[:2], dtype=torch.int32)
    return _raises(T, status, T.fade_tree_commit, L, a["q_rot"], a["lse"], a["tree_k"],
                   a["tree_v"], path, lens, a["ws"])


@pytest.mark.parametrize("n", [0, 65, -1])
def test_tree_sizes_outside_the_limits_are_refused(T, n):
    L = _layer(T)
    with pytest.raises(T.FadeError) as e:
        T.fade_tree_ws_bytes(L.cfg, n)
    assert "tree nodes" in str(e.value)
    if n == 65:
        with pytest.raises(T.FadeError):
            _attend(T, L, _args(L, n))
        z = torch.zeros((2, n), dtype=torch.int32)
        _raises(T, 1, T.fade_tree_layout, L.cfg, z, None, torch.zeros(2, dtype=torch.int32),
                torch.zeros((2, n), dtype=torch.int64), z)


def test_workspace_size_and_alignment(T):
    L = _layer(T)
    need = T.fade_tree_ws_bytes(L.cfg, 64)
    assert need >= T.fade_tree_ws_bytes(L.cfg, 1) > 0
    a = _args(L, ws=8)
    with pytest.raises(T.FadeError) as e:
        _attend(T, L, a)
    assert e.value.status == 3 and "workspace" in str(e.value)
    a = _args(L)
    off = torch.zeros(1 << 20, dtype=torch.uint8)[2:]
    with pytest.raises(T.FadeError) as e:
        _attend(T, L, a, ws=off)
    assert e.value.status == 1
    assert _commit(T, 1, L, a, [1, 1], ws=off)
    assert "workspace" in _commit(T, 3, L, _args(L, ws=16), [1, 1])


def test_unaligned_vectors_are_refused(T):
    L = _layer(T)
    a = _args(L)
    c = L.cfg
    flat = torch.zeros(c.batch * 5 * c.num_kv_heads * 64 + 8, dtype=torch.float16)
    odd = flat[4:4 + a["tree_k"].numel()].view(a["tree_k"].shape)
    with pytest.raises(T.FadeError) as e:
        _attend(T, L, a, tree_k=odd)
    assert e.value.status == 1 and "aligned" in str(e.value)
    wide = torch.zeros((c.batch, 5, c.num_kv_heads, 68), dtype=torch.float16)[..., :64]
    with pytest.raises(T.FadeError):
        _attend(T, L, a, tree_v=wide)


def test_wrong_dtypes_shapes_and_devices_are_value_errors(T):
    L = _layer(T)
    a = _args(L)
    for kw in (dict(tree_k=a["tree_k"].float()), dict(tree_v=a["tree_v"][:, :4]),
               dict(q_rot=a["q_rot"].transpose(1, 2)), dict(lse=a["lse"].double()),
               dict(mask=torch.zeros((2, 5), dtype=torch.int32)),
               dict(n_nodes=torch.zeros(3, dtype=torch.int32))):
        with pytest.raises(ValueError):
            _attend(T, L, a, **kw)
    with pytest.raises(ValueError):   # host tensors on the current stream
        T.fade_tree_attention(L, a["q_rot"], a["tree_k"], a["tree_v"],
                              torch.zeros((2, 5), dtype=torch.int64), None,
                              torch.zeros_like(a["q_rot"]), a["lse"], a["ws"])
    with pytest.raises(ValueError):
        T.fade_tree_commit(L, a["q_rot"], a["lse"], a["tree_k"], a["tree_v"],
                           torch.zeros((2, 5), dtype=torch.int32), [1], a["ws"], stream=_S())
    pq = _layer(T, v_codec="pq")
    with pytest.raises(ValueError):   # no codebook installed
        _attend(T, pq, _args(pq))


def test_commit_refusals_leave_the_mirror(T):
    L = _layer(T)
    L.h_n_sink[:], L.h_n_mid[:], L.h_n_recent[:] = 2, 6, 4
    a = _args(L)
    assert "outside" in _commit(T, 1, L, a, [6, 0])
    assert "outside" in _commit(T, 1, L, a, [0, -1])
    assert "middle slots" in _commit(T, 3, L, a, [2, 3])
    assert "H2O and EMA" in _commit(T, 1, L, a, [1, 1], ws=None)
    assert "H2O and EMA" in _commit(T, 1, L, a, [1, 1], lse=None)
    assert (L.h_n_mid.tolist(), L.h_n_recent.tolist()) == ([6, 6], [4, 4])
    sh = _layer(T, shared_rows=True)
    assert "equal path lengths" in _commit(T, 1, sh, _args(sh), [1, 2])
    # paths of no tokens: nothing to do, nothing enqueued
    T.fade_tree_commit(L, a["q_rot"], a["lse"], a["tree_k"], a["tree_v"],
                       torch.zeros((2, 5), dtype=torch.int32), [0, 0], a["ws"], stream=_S())


def test_norm_refusals(T):
    cfg = T.Config(batch=1, num_q_heads=4, num_kv_heads=1, head_dim=64, mid_capacity=16)
    tab = torch.zeros(32 * 64)
    q = torch.zeros((1, 40, 4, 64), dtype=torch.float16)
    k = torch.zeros((1, 40, 1, 64), dtype=torch.float16)
    w = torch.ones(64, dtype=torch.float16)
    pos = torch.zeros((1, 40), dtype=torch.int32)
    f = T.fade_qk_norm_rope
    _raises(T, 3, f, cfg, tab, 32, q, k, w, w, 1e-6, None, q, k)       # 40 positions, 32 held
    _raises(T, 1, f, cfg, None, 32, q, k, w, w, 1e-6, pos, q, k)
    for eps in (0.0, -1.0, float("inf"), float("nan")):
        _raises(T, 1, f, cfg, tab, 32, q, k, w, w, eps, pos, q, k)
    _raises(T, 1, f, cfg, tab, 32, q, None, w, w, 1e-6, pos, None, None)   # no output
    over = torch.zeros((1, 1, 4, 64), dtype=torch.float16).expand(1, 40, 4, 64)
    assert "overlap" in _raises(T, 1, f, cfg, tab, 32, q, None, w, w, 1e-6, pos, over, None)
    wo = torch.ones(72, dtype=torch.float16)[4:68]
    _raises(T, 1, f, cfg, tab, 32, q, k, wo, w, 1e-6, pos, q, k)
    with pytest.raises(ValueError):
        f(cfg, tab, 32, q, k, w[:32], w, 1e-6, pos, q, k, stream=_S())
    with pytest.raises(ValueError):
        f(cfg, tab, 32, q, k, w, w, 1e-6, pos.long(), q, k, stream=_S())
    for bad in (tab[:-1], tab.double(), torch.zeros(64 * 64)[::2]):   # short, wrong type, strided
        with pytest.raises(ValueError):
            f(cfg, bad, 32, q, k, w, w, 1e-6, pos, q, k, stream=_S())
    # no tokens: nothing to do
    f(cfg, tab, 32, q[:, :0], k[:, :0], w, w, 1e-6, pos[:, :0].contiguous(), q[:, :0], k[:, :0],
      stream=_S())


def test_model_refusals(T):
    from tiered_mixed_precision_gb300.model import FadeCache

    cfg = T.Config(batch=2, num_q_heads=4, num_kv_heads=1, head_dim=64, mid_capacity=16,
                   rope_kind="none")
    fc = FadeCache(cfg, 1, 8, 64, device="cpu")
    with pytest.raises(ValueError):
        fc.set_qk_norm(torch.ones(64), None)
    with pytest.raises(ValueError):
        fc.tree_begin(torch.zeros((1, 4), dtype=torch.int32))
    with pytest.raises(T.FadeError):
        fc.tree_begin(torch.zeros((2, 65), dtype=torch.int32))
    assert np.all(fc.layers[0].h_n_sink == 0)


def test_a_strided_workspace_is_refused(T):
    L = _layer(T)
    a = _args(L)
    a["ws"] = torch.zeros(1 << 21, dtype=torch.uint8)[::2]
    with pytest.raises(ValueError):
        _attend(T, L, a)
    with pytest.raises(ValueError):
        T.fade_tree_commit(L, a["q_rot"], a["lse"], a["tree_k"], a["tree_v"],
                           torch.zeros((2, 5), dtype=torch.int32), [1, 1], a["ws"], stream=_S())


def test_pointers_off_their_type_are_refused(T):
    """What a kernel would read or write in words that do not start on a multiple of their size."""
    import ctypes

    from tiered_mixed_precision_gb300 import fade as F

    L = _layer(T)
    a = _args(L)
    c, lib, n = L.cfg, T.lib(), 5
    cfg, layer = ctypes.byref(c.c()), ctypes.byref(L.c)
    room = torch.zeros(1 << 16, dtype=torch.uint8)
    at = (room.data_ptr() + 15) // 16 * 16
    q, out = a["q_rot"].data_ptr(), torch.zeros_like(a["q_rot"])
    k, v, ws, size = F._heads(a["tree_k"]), F._heads(a["tree_v"]), a["ws"].data_ptr(), 1 << 20
    lens = np.ones(2, np.int32)

    def attend(mask=at, n_nodes=at, lse=at):
        return lib.fade_tree_attention(cfg, layer, n, q, k, v, mask, n_nodes, out.data_ptr(), lse,
                                       ws, size, None)

    def commit(path=at, lse=at):
        return lib.fade_tree_commit(cfg, layer, n, q, lse, k, v, path, lens.ctypes.data, ws, size,
                                    None)

    def layout(**kw):
        p = {**dict(parents=at, n_nodes=at, base=at, mask=at, pos=at), **kw}
        return lib.fade_tree_layout(cfg, n, p["parents"], p["n_nodes"], p["base"], p["mask"],
                                    p["pos"], None)

    for call in (lambda: attend(mask=at + 4), lambda: attend(lse=at + 2),
                 lambda: attend(n_nodes=at + 2), lambda: commit(path=at + 2),
                 lambda: commit(lse=at + 2), lambda: layout(mask=at + 4),
                 *(lambda x=x: layout(**{x: at + 2}) for x in ("parents", "n_nodes", "base", "pos")),
                 lambda: lib.fade_qk_norm_rope(cfg, at, 8, k, k, None, None, None, None,
                                               ctypes.c_float(1.0), at + 2, 2, n, None)):
        assert call() == 1
        assert "aligned" in F.fade_last_error()
    scores = L.c.recent_scores
    L.c.recent_scores = scores + 2
    assert commit() == 1 and "scores" in F.fade_last_error()
    L.c.recent_scores = scores
