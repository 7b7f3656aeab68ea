"""Beam selection's log-sums where logits are far from 0 and rise along a row, so that what a thread's sum is relative to
moves: beams of the same logits in another order have the same sum, whatever the order.

Tolerances as in test_gpu_beam: 2^-19 for the sum's logarithm, 2^-24 of the score."""
import numpy as np
import pytest
import torch

from oracle import beam_oracle as bo
from test_gpu_beam import DEV, DT, _np, check_select

pytestmark = pytest.mark.gpu


def stairs(V, base, steps, period, reverse):
    """`period` logits of one height after another: a thread takes its logits from all heights in turn."""
    at = torch.arange(V, device=DEV) % (period * len(steps)) // period
    s = torch.tensor(steps, dtype=torch.float64, device=DEV)
    return (base + (s.flip(0) if reverse else s)[at]).float()


@pytest.mark.parametrize("base", [0, -90, 300, -300, 3000, -3000, 30000, 90000, -90000])
@pytest.mark.parametrize("steps", [(0, 15.875, 16.125, 16.125), (0, 10.75, 11.25, 11.25), (0, 17, 34, 51), (0, 0.5, 1, 12)])
@pytest.mark.parametrize("period", [4096, 1024])
def test_sums_of_rising_rows(lib, base, steps, period):
    """One sequence of 32 beams: every other one falls where the others rise."""
    K, V, M = 32, 32768, 64
    x = torch.stack([stairs(V, base, steps, period, k % 2 == 1) for k in range(K)])[None].contiguous()
    for k in range(K):                                       # one of each's highest logits stands out
        x[0, k, 100 + 7 * k + (0 if k % 2 else 3 * period)] = base + max(steps) + 4.0
    scores = -1 - torch.arange(K, device=DEV).float()[None] * 2.0 ** -17           # beams' scores lie this close
    check_select(lib.cp_beam_select(x, scores, num_candidates=M), x, scores, M, -1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("base", [0, 256, 4096, -32768])
def test_sums_of_many_short_and_long_rows(lib, dtype, base):
    """Rows that are one chunk, and rows of many; each candidate's score against the oracle's for that continuation."""
    for B, K, V, M in ((1, 4, 32000, 8), (160, 4, 20001, 8), (2, 32, 2048, 64)):
        g = torch.Generator(device=DEV).manual_seed(V)
        x = base + torch.linspace(0, 40, V, device=DEV) + torch.randn(B, K, V, generator=g, device=DEV)
        x = x.to(DT[dtype]).contiguous()
        scores = -5 + torch.randn(B, K, generator=g, device=DEV)
        *_, cs, cb, ct = (y.cpu().numpy() for y in lib.cp_beam_select(x, scores, num_candidates=M))
        for b in range(0, B, 53):
            a, s = _np(x[b]), _np(scores[b])
            top = a.max(-1, keepdims=True)
            exact = s[:, None] + (a - top - np.log(np.exp(a - top).sum(-1, keepdims=True)))
            mine = exact[cb[b], ct[b]]
            e = 2.0 ** -19 + 2.0 ** -24 * np.abs(mine)
            assert (np.abs(cs[b] - mine) <= e).all()
            best = np.array([c[0] for c in bo.select(a, s, M)[0]])
            assert (np.abs(mine - best) <= 2 * e).all() and len(set(zip(cb[b], ct[b]))) == M
