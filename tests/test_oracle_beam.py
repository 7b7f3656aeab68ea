"""Pins of the beam oracle: cross attention against torch in float64 and the serving oracle, selection against
hand-worked cases and torch, reordering against the logical rows that the tables describe."""
import math

import numpy as np
import pytest
import torch

from oracle import beam_oracle as bo
from oracle import serving_oracle as so


def test_cross_attention_against_torch_and_the_causal_oracle():
    r = np.random.default_rng(1)
    q, k, v = r.normal(size=(5, 6, 8)), r.normal(size=(7, 2, 8)), r.normal(size=(7, 2, 8))
    ranges = np.array([[0, 7], [2, 5], [3, 3], [-4, 99], [6, 7]])
    out, lse, _, _ = bo.cross(q, k, v, 0.3, ranges)
    Q, K, V = (torch.tensor(x).transpose(0, 1) for x in (q, k, v))
    s = 0.3 * Q @ K.repeat_interleave(3, 0).transpose(1, 2)
    for i, (a, b) in enumerate(ranges):
        a, b = max(0, a), min(7, b)
        if a >= b:
            assert (out[i] == 0).all() and np.isneginf(lse[i]).all()
            continue
        x = s[:, i, a:b]
        assert np.allclose(lse[i], torch.logsumexp(x, -1).numpy())
        assert np.allclose(out[i], (x.softmax(-1)[:, None] @ V.repeat_interleave(3, 0)[:, a:b])[:, 0].numpy())
    o = so.attend(q[4], k.transpose(1, 0, 2), v.transpose(1, 0, 2), 6, 0, 7, 0.3)
    last = bo.cross(q[4:], k, v, 0.3)
    assert np.allclose(o[0], last[0][0]) and np.allclose(o[1], last[1][0])   # the last position sees all


def test_selection_by_hand():
    x = np.log(np.array([[0.5, 0.25, 0.25, 0.0], [0.1, 0.1, 0.1, 0.7]]) + 1e-300)
    x[0, 3] = -np.inf
    best, on = bo.select(x, np.array([math.log(0.5), math.log(0.5)]), 4, eos=3)
    assert [c[1:] for c in best] == [(1, 3), (0, 0), (0, 1), (0, 2)]         # 0.35, 0.25, then equal: lower first
    assert np.allclose([math.exp(c[0]) for c in best], [0.35, 0.25, 0.125, 0.125])
    assert [c[1:] for c in on] == [(0, 0), (0, 1)]


def test_selection_of_what_has_no_probability():
    inf = np.inf
    x = np.array([[-inf, np.nan, -inf], [1.0, -inf, 1.0], [inf, 0.0, inf]])
    best, _ = bo.select(x, np.array([-1.0, -2.0, -3.0]), 7)
    assert [c[1:] for c in best] == [(1, 0), (1, 2), (2, 0), (2, 2), (0, 0), (0, 1), (0, 2)]
    assert np.allclose([c[0] for c in best[:4]], [-2 - math.log(2)] * 2 + [-3 - math.log(2)] * 2)
    assert all(c[0] == -inf for c in best[4:])
    best, _ = bo.select(np.zeros((2, 3)), np.array([-inf, 0.0]), 5)
    assert [c[1:] for c in best] == [(1, 0), (1, 1), (1, 2), (0, 0), (0, 1)]
    best, on = bo.select(np.zeros((3, 2)), np.array([inf, np.nan, 1.0]), 4, eos=0)
    assert [c[1:] for c in best] == [(2, 0), (2, 1), (0, 0), (0, 1)] and [c[1:] for c in on] == [(2, 1), (0, 1)]


def test_selection_against_torch():
    r = np.random.default_rng(2)
    x, s = r.normal(size=(4, 50)) * 3, r.normal(size=4)
    want = torch.topk((torch.tensor(x).log_softmax(-1) + torch.tensor(s)[:, None]).reshape(-1), 8)
    best, _ = bo.select(x, s, 8)
    assert np.allclose([c[0] for c in best], want.values.numpy())
    assert [c[1] * 50 + c[2] for c in best] == want.indices.tolist()


@pytest.mark.parametrize("cp,I", [(1, 16), (2, 3), (4, 8)])
def test_reordered_tables_describe_the_parents_rows(cp, I):
    """Generation by generation: each beam's rows, read through its table, are its history's."""
    r = np.random.default_rng(cp)
    K, prompt, steps, cols = 3, 21, 60, 8
    own = np.arange(cp * K * cols).reshape(cp, K, cols) % (K * cols) + 10
    tables = np.full((cp, K, cols), -1)
    for k in range(cp):
        tables[k, :, :-(-bo.held(prompt, k, cp, I) // 16)] = np.arange(-(-bo.held(prompt, k, cp, I) // 16))
    cache = np.full((cp, 10 + K * cols, 1, 16, 1), np.nan)
    hist = [[float(p) for p in range(prompt)] for _ in range(K)]
    for p in range(prompt):
        rank, page, row = so.slot(p, cp, I, tables[:, 0])
        cache[rank, page, 0, row] = p
    for n in range(prompt, prompt + steps):
        parents = [r.integers(0, K, K).tolist()]
        tables, (cache,) = bo.reorder(parents, [n], tables, own, [cache], cp, I)
        hist = [list(hist[p]) for p in parents[0]]
        for j in range(K):
            value = 1000.0 * n + j
            rank, page, row = so.slot(n, cp, I, tables[:, j])
            cache[rank, page, 0, row] = value
            hist[j].append(value)
        for j in range(K):
            got = [cache[(*so.slot(p, cp, I, tables[:, j])[:2], 0, so.slot(p, cp, I, tables[:, j])[2])][0]
                   for p in range(n + 1)]
            assert got == hist[j]
