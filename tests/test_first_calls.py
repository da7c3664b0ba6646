"""The first calls of a process, from several threads at once."""

import threading

import numpy as np
import pytest
import torch


def test_types_are_there_before_torch_is(monkeypatch):
    """What another thread takes as the sign that a first call has been made comes last."""
    from tiered_mixed_precision_gb300 import fade as F

    class Watched(dict):
        def __setitem__(self, k, v):
            assert F._torch is None, k
            super().__setitem__(k, v)

    monkeypatch.setattr(F, "_torch", None)
    monkeypatch.setattr(F, "_dtypes", Watched())
    F._device(None)
    assert F._torch is torch and set(F._dtypes) == {"float16", "bfloat16", "float32", "int32", "int64"}


@pytest.mark.gpu
def test_calls_from_several_threads():
    """Each with a stream, tensors and workspace of its own: the bits of the same calls alone."""
    from tiered_mixed_precision_gb300 import build

    build.build()
    from tiered_mixed_precision_gb300 import fade as F

    cfg = F.Config(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=64, mid_capacity=64)
    B, n, V, T = 2, 700, 3001, 6
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn((B, n, h, 64), generator=g).half().cuda() for h in (8, 2, 2))
    logits = torch.randn((B, T + 1, V), generator=g).half().cuda()
    draft = torch.randn((B, T + 1, V), generator=g).half().cuda()
    parents = torch.tensor([[-1, 0, 0, 1, 2, 2]] * B, dtype=torch.int32, device="cuda")
    tokens = draft.argmax(-1)[:, :T].int().contiguous()
    u, noise = torch.rand((B, T), generator=g).cuda(), torch.rand((B, V), generator=g).cuda() + 0.1
    lens = np.array([n, 333], np.int32)

    def calls(got, i, rounds):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(rounds):
                out, lse = torch.zeros_like(q), torch.zeros((B, n, 8), device="cuda")
                mass = torch.zeros((B, 2, n), device="cuda")
                path = torch.zeros((B, T), dtype=torch.int32, device="cuda")
                n_path, nxt = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
                F.fade_prompt_attention(cfg, q, k, v, out, lse, lens, lens, 4, 90)
                F.fade_prompt_mass(cfg, q, k, lse, mass, lens, lens, 4, 90)
                F.fade_tree_verify(cfg, parents, None, tokens, logits[:, 1:], logits[:, 0], draft[:, 1:],
                                   draft[:, 0], None, u, noise, path, n_path, nxt)
            torch.cuda.current_stream().synchronize()
        got[i] = (out, lse, mass, path, n_path, nxt)

    torch.cuda.synchronize()
    got = [None] * 5
    threads = [threading.Thread(target=calls, args=(got, i, 20)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    calls(got, 4, 1)
    for one in got[:4]:
        for x, y in zip(one, got[4]):
            assert torch.equal(x, y)
