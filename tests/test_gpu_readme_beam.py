"""The README's beam search example runs as it is printed, and gives what the calls' oracle-tested parts give."""
import numpy as np
import pytest
import torch

from test_gpu_beam import check_select
from test_gpu_cross import check, exact
from test_gpu_readme import _block

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


def test_the_beam_search_example(lib):
    B, K, Hq, Hkv, d, vocab, cp, columns = 3, 4, 8, 2, 64, 5003, 2, 6
    g = torch.Generator(device="cuda").manual_seed(3)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    S = [70, 1, 200]
    lens, pool = torch.tensor([37, 90, 16], **I32), B * K * columns
    bt = torch.randperm(pool, generator=g, device="cuda").int().reshape(1, B * K, columns).repeat(cp, 1, 1)
    names = dict(
        torch=torch, cpa=lib, B=B, K=K, vocab=vocab, S=max(S), eos=7, logits=3 * normal(B, K, vocab), lens=lens, bt=bt, own=bt.clone(),
        scores=torch.randn(B, K, generator=g, device="cuda"), kc=normal(cp, pool, Hkv, 16, d), vc=normal(cp, pool, Hkv, 16, d),
        q=normal(B * K, Hq, d), k=normal(B * K, Hkv, d), v=normal(B * K, Hkv, d), qx=normal(B * K, Hq, d),
        kx=normal(sum(S), Hkv, d), vx=normal(sum(S), Hkv, d), cu_kv=torch.tensor(np.cumsum([0] + S), **I32), max_len=100,
        f=10000.0 ** (-torch.arange(d // 2, device="cuda").double() / (d // 2)))
    logits, scores = names["logits"], names["scores"]
    exec(_block("Beam search with K beams a source"), names)
    check_select([names["scores"], names["parents"], names["tokens"], *names["candidates"]], logits, scores, 2 * K, 7)
    assert names["lens"].tolist() == [38, 91, 17]
    spans = [(b * K, K, sum(S[:b]), S[b]) for b in range(B)]
    check(names["out"], names["lse"], exact(names["qx"], names["kx"], names["vx"], spans, d ** -0.5), False)
    # full columns are the parents', the page being filled each beam's own
    at = (lens.cpu().numpy() // 2) // 16
    for b in range(B):
        for j, p in enumerate(names["parents"][b].tolist()):
            row, now = names["own"][0, b * K + p], names["bt"][0, b * K + j]
            c = min(int(at[b]), columns)
            assert torch.equal(now[:c], row[:c])
