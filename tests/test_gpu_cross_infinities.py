"""Cross attention with infinities and numbers near the largest in what a row sees: a key whose score is -inf has no
weight, one of +inf makes the row NaN, and other rows are as they are without it; in every type, for few rows and many,
whole and in parts.

The tolerances are test_gpu_cross's, with the largest scale sum |q||k| of the keys that have a finite score."""
import math

import pytest
import torch

from test_gpu_cross import DEV, DT, I32, _cu, check

pytestmark = pytest.mark.gpu


def reference(q, k, v, scale):
    """Float64, one sequence: (out, lse, weight-averaged |v|, largest scale sum |q||k| of a finite score)."""
    q, k, v = (x.double().cpu() for x in (q, k, v))
    G = q.shape[1] // k.shape[1]
    k, v = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    s = torch.full((q.shape[0], q.shape[1], k.shape[0]), 0.0, dtype=torch.float64)
    for h in range(q.shape[1]):
        for c in range(q.shape[2]):         # (a sum of infinities of one sign, not of a blocked product's 0 times one)
            s[:, h] += q[:, h, c, None] * k[None, :, h, c]
    s *= scale
    b = scale * torch.einsum("ihd,jhd->ihj", q.abs(), k.abs())
    lse = torch.logsumexp(s, -1)
    w = torch.exp(s - lse[..., None])
    return [x.numpy() for x in (torch.einsum("ihj,jhd->ihd", w, v), lse, torch.einsum("ihj,jhd->ihd", w, v.abs()),
                                b.masked_fill(~s.isfinite(), 0).amax(-1))]


# rows, keys, Hq, Hkv, d, dtype, workspace
SIZES = [(1, 40, 2, 1, 64, "f32", True), (5, 700, 4, 2, 64, "f32", True), (6, 333, 4, 2, 128, "f32", True),
         (20, 130, 2, 2, 128, "f32", True), (70, 90, 6, 2, 64, "f32", True), (3, 9000, 2, 1, 64, "f32", True),
         (3, 9000, 2, 1, 64, "f32", False), (1, 40, 2, 1, 64, "bf16", True), (4, 1500, 4, 2, 64, "bf16", True),
         (20, 130, 2, 2, 128, "bf16", True), (3, 20000, 2, 1, 128, "bf16", True), (200, 700, 4, 2, 128, "bf16", True),
         (300, 2000, 2, 2, 64, "bf16", True), (150, 333, 4, 2, 64, "bf16", False)]


def data(T, S, Hq, Hkv, d, dtype):
    g = torch.Generator(device=DEV).manual_seed(T + S)
    return [torch.randn(n, h, d, generator=g, device=DEV).to(DT[dtype]) for n, h in ((T, Hq), (S, Hkv), (S, Hkv))]


def run(lib, q, k, v, ws, ranges=None):
    err = torch.zeros(1, **I32)
    got = lib.cp_cross_attention(q, _cu([len(q)]), k, v, _cu([len(k)]), max_seqlen_q=len(q), max_seqlen_kv=len(k), err=err,
                                 key_ranges=ranges, workspace=None if ws else torch.empty(0, dtype=torch.uint8, device=DEV))
    assert int(err) == 0
    return got


@pytest.mark.parametrize("T,S,Hq,Hkv,d,dtype,ws", SIZES)
@pytest.mark.parametrize("ranged", [False, True])
def test_visible_keys_with_infinities(lib, T, S, Hq, Hkv, d, dtype, ws, ranged):
    q, k, v = data(T, S, Hq, Hkv, d, dtype)
    q[..., 7] = q[..., 7].abs() + 0.25                    # (and 1 somewhere: its lower parts are 0)
    q[..., d - 1] = -1
    k[S // 3, :, 7] = -math.inf
    k[S - 1, :, d - 1] = math.inf
    ranges = torch.tensor([[0, S]] * T, **I32) if ranged else None
    out, lse = run(lib, q, k, v, ws, ranges)
    want = reference(q, k, v, d ** -0.5)
    check(out, lse, want, dtype == "f32")
    # a score of +inf in one row and head: that row is NaN, the others are as they were
    j, h = T // 2, Hq - 1
    q[j, h, 7] = -q[j, h, 7]
    o2, l2 = run(lib, q, k, v, ws, ranges)
    assert bool(o2[j, h].isnan().all()) and not bool(l2[j, h].isfinite())
    o2[j, h], l2[j, h] = out[j, h], lse[j, h]
    check(o2, l2, want, dtype == "f32")


@pytest.mark.parametrize("T,S,Hq,Hkv,d,dtype,ws", SIZES)
def test_queries_with_infinities(lib, T, S, Hq, Hkv, d, dtype, ws):
    """Row 0 has +inf in a head: scores of -inf alone leave it without weights, one of +inf makes it NaN."""
    q, k, v = data(T, S, Hq, Hkv, d, dtype)
    k[..., 7] = -k[..., 7].abs() - 0.25
    want = reference(q, k, v, d ** -0.5)
    clean, cl = run(lib, q, k, v, ws)
    check(clean, cl, want, dtype == "f32")
    q[0, 0, 7] = math.inf
    out, lse = run(lib, q, k, v, ws)
    assert bool((out[0, 0] == 0).all()) and bool(lse[0, 0].isneginf())
    out[0, 0], lse[0, 0] = clean[0, 0], cl[0, 0]
    check(out, lse, want, dtype == "f32")
    k[S // 2, 0, 7] = 1
    out, lse = run(lib, q, k, v, ws)
    assert bool(out[0, 0].isnan().all()) and not bool(lse[0, 0].isfinite())
    keep = torch.ones(T, Hq, dtype=torch.bool, device=DEV)
    keep[0, 0] = False
    assert bool(out[keep].isfinite().all()) and bool(lse[keep].isfinite().all())


@pytest.mark.parametrize("T,S,Hq,Hkv,d", [x[:5] for x in SIZES if x[5] == "f32" and x[6]])
def test_finite_numbers_that_round_to_infinities(lib, T, S, Hq, Hkv, d):
    """Above 3.39e38 the nearest bf16 is an infinity."""
    q, k, v = data(T, S, Hq, Hkv, d, "f32")
    q[..., 3] = 2.0 ** -125
    k[S // 2, :, 3], k[0, :, 3] = 3.4e38, -3.4028234e38
    out, lse = run(lib, q, k, v, True)
    check(out, lse, reference(q, k, v, d ** -0.5), True)
    q[0, 0, 5], k[..., 5] = -3.3999e38, 2.0 ** -124
    out, lse = run(lib, q, k, v, True)
    check(out, lse, reference(q, k, v, d ** -0.5), True)
