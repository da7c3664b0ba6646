"""Verification at temperatures near 0 and of logits far from 0: probabilities depend on differences from the
largest logit alone, which have to be taken before they are scaled."""

import numpy as np
import pytest
import torch

from test_gpu_verify import F, _call, _compare, _inputs  # noqa: F401  (F: the fixture)

pytestmark = pytest.mark.gpu

DTYPES = [torch.float16, torch.bfloat16, torch.float32]
LOW = [1e-2, 1e-4, 1e-5, 1e-6, 1e-7, 1e-9, 1e-30, 1e-38]


def _peaked(B, V, dtype, seed):
    """Root and two nodes in a chain (target, drafter), each with one logit of 15 to 25 above all others
    (below 10), and the tokens that have it."""
    g = torch.Generator().manual_seed(seed)
    target = (torch.randn((B, 3, V), generator=g) * 3).clamp(max=9.5)
    draft = (target + torch.randn((B, 3, V), generator=g)).clamp(max=9.5)
    top = torch.randint(V, (B, 3), generator=g)
    for x in (target, draft):
        x.scatter_(2, top[..., None], 15 + 10 * torch.rand((B, 3, 1), generator=g))
    return target.to(dtype), draft.to(dtype), top.int()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("mode", ["sampled", "certain"])
@pytest.mark.parametrize("V", [1000, 50257, 150001])
def test_a_sure_token_is_kept_at_any_low_temperature(F, V, mode, dtype):
    """5 below the top at T = 1e-2 or less is e^-500: p of the top token is 1 (q too), so a draft of it is
    kept under u = 0.9999 and the next sure token comes after it."""
    B, T = 4 * len(LOW), 2
    target, draft, top = _peaked(B, V, dtype, V)
    st = dict(parents=torch.tensor([[-1, 0]] * B, dtype=torch.int32), n_nodes=None,
              tokens=top[:, :2].contiguous(), target=target[:, 1:], target_root=target[:, 0],
              draft=draft[:, 1:] if mode == "sampled" else None,
              draft_root=draft[:, 0] if mode == "sampled" else None,
              temperature=torch.tensor(LOW, dtype=torch.float32).repeat(4),
              u=torch.full((B, T), 0.9999),
              noise=torch.empty((B, V)).exponential_(generator=torch.Generator().manual_seed(V)))
    path, n_path, nxt = _call(F, st, B, T)
    assert n_path.tolist() == [2] * B and path.tolist() == [[0, 1]] * B
    assert nxt.tolist() == top[:, 2].tolist()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("mode", ["sampled", "certain"])
def test_two_tied_tokens_have_one_half_each(F, mode, dtype):
    """At any low temperature: a draft of one of them, sure for the drafter, is kept under u = 0.499 and
    refused under 0.501, and then the other one comes."""
    V, T = 5003, 1
    temps = [t for t in LOW for _ in range(2)]
    B = len(temps)
    target, draft, top = _peaked(B, V, dtype, 7)
    target, draft, top = target[:, 0], draft[:, 0], top[:, 0].long()
    other = (top + 1234) % V
    rows = torch.arange(B)
    target[rows, other] = target[rows, top]
    u = torch.tensor([0.499, 0.501] * len(LOW))
    st = dict(parents=torch.full((B, T), -1, dtype=torch.int32), n_nodes=None,
              tokens=top[:, None].int(), target=target[:, None].clone(), target_root=target,
              draft=draft[:, None].clone() if mode == "sampled" else None,
              draft_root=draft if mode == "sampled" else None,
              temperature=torch.tensor(temps, dtype=torch.float32), u=u[:, None].contiguous(),
              noise=torch.ones((B, V)))
    st["noise"][rows, other] = 1e-2   # (also what comes after a kept one)
    path, n_path, nxt = _call(F, st, B, T)
    assert n_path.tolist() == [1, 0] * len(LOW)
    assert nxt.tolist() == other.tolist()


@pytest.mark.parametrize("mode", ["sampled", "certain", "greedy"])
def test_low_temperatures_against_definition(F, mode):
    """Drafts are the drafter's (or the target's) likeliest tokens, as at such temperatures they are."""
    B, T, V = 4 * len(LOW), 7, 3001
    for seed in (1, 2):
        st = _inputs(B, T, V, torch.float32, seed, mode)
        at = (st["parents"].long() + 1, torch.arange(B)[:, None])
        like = "draft" if mode == "sampled" else "target"
        both = torch.cat([st[like + "_root"][:, None], st[like]], 1)
        st["tokens"] = both[at[1], at[0]].argmax(-1).int()
        if mode != "greedy":
            st["temperature"] = torch.tensor(LOW, dtype=torch.float32).repeat(4)
        _compare(F, st, B, T, near=0.1)


@pytest.mark.parametrize("mode", ["sampled", "certain", "greedy"])
@pytest.mark.parametrize("V", [1003, 50257])
def test_a_common_offset_changes_nothing(F, V, mode):
    """fp32 logits in eighths plus an offset that keeps them exact (below 2^21, where a step is an eighth):
    the same differences, so the same bits and tokens as without."""
    B, T = 16, 8
    st = _inputs(B, T, V, torch.float32, V, mode)
    for x in ("target", "target_root", "draft", "draft_root"):
        if st[x] is not None:
            st[x] = (8 * st[x]).round() / 8
    plain = _call(F, st, B, T)
    if V < 2000:
        _compare(F, st, B, T, near=0.2)
    for ot, od in ((1e4, 1e4), (1e5, -1e5), (-1e6, 1e6), (2.0 ** 20, 0.0)):
        moved = dict(st)
        for x, o in (("target", ot), ("target_root", ot), ("draft", od), ("draft_root", od)):
            if st[x] is not None:
                moved[x] = st[x] + o
                assert torch.equal(moved[x] - o, st[x])
        for a, b in zip(_call(F, moved, B, T), plain):
            assert np.array_equal(a, b), (ot, od)
