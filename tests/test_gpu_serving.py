"""Parity of the rotate-and-append, read-back, 4-bit and modified-score calls with the float64
serving oracle, with whatever lies outside a row's keys poisoned.

Tolerances, fixed before the first run:
  * fp32 sums of up to 128 products, each addition off by at most 2^-23 of partial sums that
    `big` = max scale sum |q||k| bounds: a score is off by at most 2^-16 big; the cap adds
    cap 2^-20 (two approximate special functions of 2^-22 each, and a rounding), the bias 2^-22 of
    itself, which is at most slope * length.  The LSE inherits that and 2^-22 of itself (SCORE).
  * outputs: a score error e changes every weight by at most a factor e^2e, so the output by
    2 e |v|_avg; probabilities enter the PV product as bf16: 2^-8 |v|_avg; bf16 output: 2^-8 |O|;
    fp32 sums over the keys: 2^-18 |v|_avg.
  * 4-bit values: the rounded factor is probability times scale, against code * scale =
    value - minimum, so its 2^-8 multiplies |value - minimum|_avg, at most |v|_avg + |minimum|_avg.
  * rotation: angles off by 2^-26 turns and cosines by 2^-22 together, two products and a sum of
    2^-24 each: 2^-20.5 of the pair's length, below 1e-6 of it.
"""
import math

import numpy as np
import pytest
import torch

from oracle import serving_oracle as so

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _np(t):
    return t.detach().double().cpu().numpy()


def _score_tol(big, lse, cap, slopes, length):
    lse = np.where(np.isfinite(lse), np.abs(lse), 0)
    return 2.0 ** -16 * big + cap * 2.0 ** -20 + (max(slopes) * length * 2.0 ** -22 if slopes is not None else 0) + \
        2.0 ** -22 * lse + 1e-6


def _check(out, lse, O, L, absv, big, cap=0.0, slopes=None, length=1, f32=False, what=""):
    out, lse = _np(out), _np(lse)
    assert np.array_equal(np.isneginf(lse), np.isneginf(L)), f"{what}: rows without keys differ"
    e = _score_tol(big, L, cap, slopes, length)
    fin = np.isfinite(L)
    assert np.isfinite(out).all(), f"{what}: not finite"
    assert (np.abs(lse - np.where(fin, L, 0))[fin] <= e[fin]).all(), f"{what}: lse off by " \
        f"{np.abs(lse - np.where(fin, L, 0))[fin].max()} against {e[fin].min()}"
    tol = 2 * e[..., None] * absv + 2.0 ** -18 * absv + 1e-30
    if not f32:
        tol = tol + 2.0 ** -8 * absv + 2.0 ** -8 * np.abs(O)
    assert (np.abs(out - O) <= tol).all(), f"{what}: out off by {np.abs(out - O).max()}, worst ratio " \
        f"{(np.abs(out - O) / tol).max()}"
    assert (out[~fin] == 0).all()


# ------------------------------------------------------------------------------ paged caches
class Cache:
    """Pools with every slot poisoned, block tables over a shuffled pool, and the logical rows."""

    def __init__(self, lens, Hkv, d, cp, I, dtype, q4, seed=0, cols=None):
        r = np.random.default_rng(seed)
        self.B, self.Hkv, self.d, self.cp, self.I, self.q4 = len(lens), Hkv, d, cp, I, q4
        need = [max(1, -(-(-(-max(n, 1) // (I * cp)) * I) // 16)) for n in lens]
        cols = cols or max(need)
        self.pool = sum(need) + 3
        t = np.full((cp, self.B, cols), -1, np.int32)
        for k in range(cp):
            ids = iter(r.permutation(self.pool))
            for b, n in enumerate(need):
                t[k, b, :n] = [next(ids) for _ in range(n)]
        self.tables = t
        if q4:   # codes 15, scale and minimum NaN
            self.k, self.v = (np.full((cp, self.pool, Hkv, 9 * d), 0xFF, np.uint8) for _ in range(2))
        else:
            self.k, self.v = (np.full((cp, self.pool, Hkv, 16, d), np.nan) for _ in range(2))
        self.dtype = dtype

    def at(self, b, p):
        return so.slot(p, self.cp, self.I, self.tables[:, b])

    def put(self, b, p, k, v):
        rank, page, row = self.at(b, p)
        for c, x in ((self.k, k), (self.v, v)):
            for h in range(self.Hkv):
                if self.q4:
                    so.q4_write(c[rank, page, h], row, x[h])
                else:
                    c[rank, page, h, row] = x[h]

    def get(self, b, p):
        rank, page, row = self.at(b, p)
        if self.q4:
            return [np.stack([so.q4_read(c[rank, page, h], row, self.d) for h in range(self.Hkv)])
                    for c in (self.k, self.v)]
        return [c[rank, page, :, row] for c in (self.k, self.v)]

    def minima(self, b, p):
        rank, page, row = self.at(b, p)
        return np.stack([so.q4_minima(self.v[rank, page, h], row, self.d) for h in range(self.Hkv)])

    def device(self):
        t = torch.tensor(self.tables).to(DEV)
        if self.q4:
            return torch.tensor(self.k).to(DEV), torch.tensor(self.v).to(DEV), t
        return (torch.tensor(x, dtype=torch.float32).to(self.dtype).to(DEV) for x in (self.k, self.v)), t


def _dev(c):
    x = c.device()
    if c.q4:
        return x
    (k, v), t = x
    return k, v, t


def _rows(r, shape, dtype):
    return _np(torch.tensor(r.normal(size=shape), dtype=torch.float32).to(dtype))


# ------------------------------------------------------------------------------ append and read
WRITES = [
    # lens new, context, Hq, Hkv, d, dtype, q4, rot, style, cp, I, slices of one projection
    ([1, 1, 1], [40, 0, 17], 8, 2, 128, "bf16", False, 128, "half", 2, 8, True),
    ([5, 0, 37], [3, 9, 100], 3, 3, 64, "bf16", False, 64, "pairs", 3, 5, False),
    ([33], [1 << 20], 4, 1, 128, "f32", False, 64, "half", 4, 1, True),
    ([19, 2], [7, 1 << 19], 6, 2, 64, "f32", False, 32, "pairs", 1, 8, True),
    ([40, 1], [11, 0], 4, 2, 128, "bf16", True, 128, "half", 2, 8, True),
    ([21, 18], [0, 90], 2, 1, 128, "f32", True, 64, "pairs", 2, 16, False),
    ([3, 70], [5, 6], 2, 2, 64, "bf16", True, 64, "half", 4, 8, True),
    ([9], [1000], 0, 2, 64, "f32", True, 0, "half", 1, 8, False),
    ([300, 1, 260], [8, 8, 8], 16, 2, 128, "bf16", False, 96, "half", 2, 8, True),
]


def _write_case(lib, new, ctx, Hq, Hkv, d, dt, q4, rot, style, cp, I, sliced, seed=7, pad=3):
    r = np.random.default_rng(seed)
    dtype, N = DT[dt], sum(new)
    c = Cache([a + b for a, b in zip(new, ctx)], Hkv, d, cp, I, dtype, q4, seed) if max(ctx) < 4096 else None
    if c is None:   # far positions: a wide table that only holds the pages in use
        cols = (max(a + b for a, b in zip(new, ctx)) // cp + I) // 16 + 2
        c = Cache([400] * len(new), Hkv, d, cp, I, dtype, q4, seed, cols)
        ids = [list(r.permutation(c.pool)) for _ in range(cp)]
        c.tables[:] = -1
        for b, (n, x) in enumerate(zip(new, ctx)):
            for p in range(x, x + n):
                rank, local = (p // I) % cp, p // (I * cp) * I + p % I
                if c.tables[rank, b, local // 16] < 0:
                    c.tables[rank, b, local // 16] = ids[rank].pop()
    f = 10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))
    rows = torch.tensor(r.normal(size=(N + pad, Hq + 2 * Hkv, d)), dtype=torch.float32).to(dtype).to(DEV)
    rows[N:] = float("nan")
    q, k, v = rows.split([Hq, Hkv, Hkv], 1)
    if not sliced:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    kc, vc, t = _dev(c)
    cu = torch.tensor(np.cumsum([0] + new), dtype=torch.int32, device=DEV)
    st = torch.tensor(ctx, dtype=torch.int32, device=DEV)
    return c, f, q, k, v, kc, vc, t, cu, st, N


@pytest.mark.parametrize("case", WRITES, ids=[str(i) for i in range(len(WRITES))])
def test_write_against_the_oracle(lib, case):
    new, ctx, Hq, Hkv, d, dt, q4, rot, style, cp, I, sliced = case
    c, f, q, k, v, kc, vc, t, cu, st, N = _write_case(lib, *case)
    dtype = DT[dt]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    q_out = torch.full((N + 3, Hq, d), 77.0, dtype=dtype, device=DEV) if Hq else None
    k_out = torch.full((N + 3, Hkv, d), 77.0, dtype=dtype, device=DEV)
    kc0, vc0 = kc.clone(), vc.clone()
    lib.cp_rope_kv_cache_write(k, v, cu, st, kc, vc, t, cp, I,
                               inv_freq=torch.tensor(f, device=DEV) if rot else None,
                               rope_style=lib.CP_ROPE_PAIRS if style == "pairs" else lib.CP_ROPE_HALF,
                               q=q if Hq else None, q_out=q_out, k_out=k_out, err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    pos = np.concatenate([np.arange(x, x + n) for n, x in zip(new, ctx)])
    half = 2.0 ** -8 if dt == "bf16" else 2.0 ** -24
    want_k = so.rotate(_np(k)[:N], pos, f, style == "pairs")
    for got, want, src in ((q_out, so.rotate(_np(q)[:N], pos, f, style == "pairs") if Hq else None, q),
                           (k_out, want_k, k)):
        if got is None:
            continue
        pair = np.sqrt((_np(src)[:N] ** 2).sum(-1, keepdims=True))     # no pair is longer than its row
        assert (np.abs(_np(got)[:N] - want) <= 1e-6 * pair + half * np.abs(want)).all()
        assert bool((got[N:] == 77.0).all())                            # rows behind the last sequence
    # the cache: written slots as the oracle writes them, everything else untouched bit for bit
    kn, vn = kc.cpu(), vc.cpu()
    seen = set()
    for b, (n, x) in enumerate(zip(new, ctx)):
        for i in range(n):
            row = int(cu[b]) + i
            rank, page, s = c.at(b, x + i)
            seen.add((rank, page, s))
            for h in range(Hkv):
                wk, wv = want_k[row, h], _np(v)[row, h]
                if not q4:
                    assert torch.equal(vn[rank, page, h, s].to(v.device), v[row, h])
                    assert torch.equal(kn[rank, page, h, s].to(DEV), k_out[row, h])
                else:
                    rec = np.zeros(9 * d, np.uint8)
                    so.q4_write(rec, s, wv)
                    got = vn[rank, page, h].numpy()
                    for lo, hi in ((s * d // 2, (s + 1) * d // 2), (8 * d + s * d // 16, 8 * d + (s + 1) * d // 16)):
                        assert np.array_equal(got[lo:hi], rec[lo:hi]), (b, i, h)
                    # keys: the rotation's 1e-6 may move a code at a tie or a bf16 rounding of the
                    # scale: within half a step and one rounding of the group's ends
                    val = so.q4_read(kn[rank, page, h].numpy(), s, d)
                    _, sc, mn = so.q4_codes(wk)
                    tol = np.repeat(sc / 2 + 2.0 ** -7 * (np.abs(mn) + 15 * sc), 64)
                    assert (np.abs(val - wk) <= tol).all()
    for got, old in ((kn, kc0.cpu()), (vn, vc0.cpu())):
        a, o = got.view(torch.uint8), old.view(torch.uint8)
        if q4:
            a = torch.cat([a[..., :8 * d].unflatten(-1, (16, d // 2)), a[..., 8 * d:].unflatten(-1, (16, d // 16))], -1)
            o = torch.cat([o[..., :8 * d].unflatten(-1, (16, d // 2)), o[..., 8 * d:].unflatten(-1, (16, d // 16))], -1)
        keep = torch.ones(cp, c.pool, 16, dtype=torch.bool)
        for rank, page, s in seen:
            keep[rank, page, s] = False
        assert torch.equal(a.transpose(2, 3)[keep], o.transpose(2, 3)[keep])


def test_write_in_place_and_without_queries(lib):
    args = ([7, 12], [5, 0], 4, 2, 128, "bf16", False, 128, "half", 2, 8, True)
    c, f, q, k, v, kc, vc, t, cu, st, N = _write_case(lib, *args)
    fr = torch.tensor(f, device=DEV)
    q_out, _ = lib.cp_rope_kv_cache_write(k, v, cu, st, kc, vc, t, 2, 8, inv_freq=fr, q=q)
    kc2, vc2 = kc.clone(), vc.clone()
    got, none = lib.cp_rope_kv_cache_write(k, v, cu, st, kc2, vc2, t, 2, 8, inv_freq=fr, q=q, q_out=q)
    assert got.data_ptr() == q.data_ptr() and none is None
    assert torch.equal(q[:N], q_out[:N])
    none, _ = lib.cp_rope_kv_cache_write(k, v, cu, st, kc2, vc2, t, 2, 8, inv_freq=fr)
    assert none is None and torch.equal(kc2.view(torch.int16), kc.view(torch.int16))


@pytest.mark.parametrize("q4", [False, True])
def test_write_reports_what_has_no_page(lib, q4):
    args = ([20], [5], 2, 2, 64, "bf16", q4, 64, "half", 2, 8, False)
    c, f, q, k, v, kc, vc, t, cu, st, N = _write_case(lib, *args)
    fr = torch.tensor(f, device=DEV)
    for bad in (-1, c.pool, 1 << 30):
        t2, k2, v2 = t.clone(), kc.clone(), vc.clone()
        t2[1, 0, 0] = bad
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        q_out, _ = lib.cp_rope_kv_cache_write(k, v, cu, st, k2, v2, t2, 2, 8, inv_freq=fr, q=q, err=err)
        assert int(err) == 5
        assert torch.equal(k2[1].view(torch.uint8), kc[1].view(torch.uint8))   # rank 1: nothing written
        assert not torch.equal(k2[0].view(torch.uint8), kc[0].view(torch.uint8))
        assert bool(torch.isfinite(q_out[:N].float()).all())                    # queries are rotated all the same
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    k2, v2 = kc.clone(), vc.clone()
    lib.cp_rope_kv_cache_write(k, v, cu, torch.full_like(st, -30), k2, v2, t, 2, 8, inv_freq=fr, err=err)
    assert int(err) == 5 and torch.equal(k2.view(torch.uint8), kc.view(torch.uint8))


def test_infinities_and_nan_in_a_4bit_row(lib):
    d = 128
    c = Cache([3], 1, d, 1, 8, torch.float32, True)
    kc, vc, t = _dev(c)
    x = torch.randn(3, 1, d, device=DEV)
    x[0, 0, 3], x[1, 0, 70], x[2, 0, 5] = float("inf"), float("nan"), 3e38
    x[2, 0, 6] = -3e38
    cu, st = torch.tensor([0, 3], dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    lib.cp_rope_kv_cache_write(x, x, cu, st, kc, vc, t, 1, 8)
    k, v = lib.cp_kv_cache_read(kc, vc, cu, st, t, 1, 8, out_dtype=torch.float32)
    assert torch.equal(torch.isnan(k), torch.isnan(v))
    bad = torch.zeros(3, 2, dtype=torch.bool)
    bad[0, 0] = bad[1, 1] = bad[2, 0] = True      # the group with it, not the other one
    assert torch.equal(torch.isnan(k).view(3, 2, 64).all(-1).cpu(), bad)
    assert torch.equal(torch.isnan(k).view(3, 2, 64).any(-1).cpu(), bad)


READS = [([1], 1, 128, "bf16", False, 1, 8), ([0, 37, 130], 3, 64, "bf16", False, 2, 8),
         ([50, 3], 2, 128, "f32", False, 3, 5), ([21], 8, 64, "f32", False, 4, 1),
         ([70, 1, 0, 18], 2, 128, "bf16", True, 2, 8), ([33, 47], 1, 64, "f32", True, 4, 16),
         ([90], 2, 128, "f32", True, 1, 3)]


@pytest.mark.parametrize("lens,Hkv,d,dt,q4,cp,I", READS)
def test_read_against_the_oracle(lib, lens, Hkv, d, dt, q4, cp, I):
    r = np.random.default_rng(9)
    skip = [min(n, 2 * i) for i, n in enumerate(lens)]           # start past the first positions
    c = Cache(lens, Hkv, d, cp, I, DT[dt], q4, 3)
    want = [[], []]
    for b, n in enumerate(lens):
        for p in range(n):
            k, v = (_rows(r, (Hkv, d), DT[dt]) for _ in range(2))
            c.put(b, p, k, v)
            if p >= skip[b]:
                for w, x in zip(want, c.get(b, p)):
                    w.append(x)
    kc, vc, t = _dev(c)
    cu = torch.tensor(np.cumsum([0] + [n - s for n, s in zip(lens, skip)]), dtype=torch.int32, device=DEV)
    st = torch.tensor(skip, dtype=torch.int32, device=DEV)
    N = int(cu[-1])
    outs = [torch.full((N + 2, Hkv, d), 5.0, dtype=DT[dt], device=DEV) for _ in range(2)]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    lib.cp_kv_cache_read(kc, vc, cu, st, t, cp, I, k_out=outs[0], v_out=outs[1], err=err)
    assert int(err) == 0
    for o, w in zip(outs, want):
        assert bool((o[N:] == 5.0).all())
        w = np.array(w).reshape(N, Hkv, d)
        if q4:     # one fp32 rounding of minimum + scale n (the product is exact), one to the output
            tol = 2.0 ** -24 * np.abs(w) + (2.0 ** -8 * np.abs(w) if dt == "bf16" else 0)
            assert (np.abs(_np(o[:N]) - w) <= tol).all()
        else:
            assert np.array_equal(_np(o[:N]), w)
    two = lib.cp_kv_cache_read(kc, vc, cu, st, t, cp, I, out_dtype=DT[dt])   # allocated here
    assert torch.equal(two[0], outs[0][:N]) and torch.equal(two[1], outs[1][:N])


def test_read_reports_what_has_no_page(lib):
    c = Cache([40], 2, 64, 2, 8, torch.float32, False)
    kc, vc, t = _dev(c)
    kc.normal_(), vc.normal_()
    cu = torch.tensor([0, 40], dtype=torch.int32, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    good, _ = lib.cp_kv_cache_read(kc, vc, cu, st, t, 2, 8)
    t2 = t.clone()
    t2[1, 0, 1] = c.pool            # rank 1's second page: positions 40 .. (none), 24..31 stay on its first
    t2[0, 0, 1] = -7                # rank 0's second page: local 16.. = positions 32..39
    k = torch.full_like(good, 5.0)
    v = torch.full_like(good, 5.0)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    lib.cp_kv_cache_read(kc, vc, cu, st, t2, 2, 8, k_out=k, v_out=v, err=err)
    assert int(err) == 5
    assert torch.equal(k[:32], good[:32]) and bool((k[32:] == 5.0).all())


# ------------------------------------------------------------------------------ decode
def _decode_case(lens, Hq, Hkv, d, cp, I, dt, q4, cap, window, alibi, docs, seed=1):
    """Cache with only the visible positions written, and the oracle's result."""
    r = np.random.default_rng(seed)
    dtype = DT[dt]
    c = Cache(lens, Hkv, d, cp, I, dtype, q4, seed)
    q = _rows(r, (len(lens), Hq, d), dtype)
    slopes = np.array([2.0 ** (-8 * (h + 1) / Hq) for h in range(Hq)]) if alibi else None
    start = None
    if docs:   # somewhere inside, at the end, and behind it (an empty row)
        start = [int(r.integers(0, max(1, n))) if i % 3 else n + 4 * (i % 2) for i, n in enumerate(lens)]
    O, L, A, big = [], [], [], 0.0
    for b, n in enumerate(lens):
        lo, hi = so.bounds(n - 1, n, window, start[b] if start else None)
        k, v, mn = np.zeros((Hkv, max(n, 1), d)), np.zeros((Hkv, max(n, 1), d)), np.zeros((Hkv, max(n, 1), d))
        for p in range(max(lo, 0), max(hi, 0)):
            c.put(b, p, _rows(r, (Hkv, d), dtype), _rows(r, (Hkv, d), dtype))
            k[:, p], v[:, p] = c.get(b, p)
            if q4:
                mn[:, p] = c.minima(b, p)
        o, l, a, m = so.attend(q[b], k, v, n - 1, lo, hi, 1 / math.sqrt(d), cap, slopes)
        if q4:
            a = a + so.attend(q[b], k, np.abs(mn), n - 1, lo, hi, 1 / math.sqrt(d), cap, slopes)[0]
        O.append(o), L.append(l), A.append(a)
        big = max(big, m)
    return c, q, slopes, start, np.array(O), np.array(L), np.array(A), big


DECODES = [
    # lens, Hq, Hkv, d, cp, I, dtype, q4, cap, window, alibi, docs
    ([1], 8, 1, 128, 1, 8, "bf16", True, 0.0, 0, False, False),
    ([1, 2, 17, 16, 300], 16, 2, 128, 2, 8, "bf16", True, 0.0, 0, False, False),
    ([257, 0, 63], 6, 2, 64, 3, 5, "bf16", True, 20.0, 0, True, False),
    ([500, 33], 32, 2, 128, 2, 8, "bf16", True, 0.0, 100, False, False),
    ([129, 40, 77, 200], 18, 2, 64, 4, 1, "bf16", True, 2.0, 31, True, True),
    ([200, 90], 22, 2, 128, 1, 16, "bf16", True, 5.0, 0, True, True),
    ([1], 1, 1, 64, 1, 8, "bf16", False, 30.0, 0, False, False),
    ([300, 5, 64], 16, 2, 128, 2, 8, "bf16", False, 3.0, 0, False, False),
    ([257, 0, 63], 9, 3, 64, 3, 5, "bf16", False, 20.0, 0, True, False),
    ([500, 33], 32, 2, 128, 2, 8, "bf16", False, 0.0, 1, False, False),
    ([129, 40, 77, 200], 20, 2, 64, 8, 1, "bf16", False, 2.0, 31, True, True),
    ([400], 8, 8, 128, 1, 8, "bf16", False, 0.0, 4000, True, False),
    ([1, 300], 8, 2, 64, 4, 8, "f32", False, 0.0, 50, True, False),
    ([100, 0, 17, 250], 14, 2, 128, 2, 3, "f32", False, 4.0, 0, True, True),
    ([333], 3, 3, 128, 1, 8, "f32", False, 30.0, 0, False, False),
    ([90, 16], 10, 2, 64, 2, 8, "f32", False, 0.0, 16, False, False),
]


@pytest.mark.parametrize("case", DECODES, ids=[str(i) for i in range(len(DECODES))])
def test_decode_against_the_oracle(lib, case):
    lens, Hq, Hkv, d, cp, I, dt, q4, cap, window, alibi, docs = case
    c, q, slopes, start, O, L, A, big = _decode_case(*case)
    kc, vc, t = _dev(c)
    dq = torch.tensor(q, dtype=torch.float32).to(DT[dt]).to(DEV)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    kw = dict(softcap=cap, window=window,
              alibi_slopes=torch.tensor(slopes, dtype=torch.float32, device=DEV) if alibi else None,
              kv_start=torch.tensor(start, dtype=torch.int32, device=DEV) if docs else None)
    if alibi:
        slopes = _np(kw["alibi_slopes"])
    fused, part = ((lib.cp_decode_attention_q4, lib.cp_partial_attn_decode_q4) if q4 else
                   (lib.cp_decode_attention_mod, lib.cp_partial_attn_decode_mod))
    chk = dict(cap=cap, slopes=slopes, length=max(lens), f32=dt == "f32")
    share = max(1, -(-max(lens) // (I * cp)) * I)
    for plan in (None, (1, (share + 31) // 16 * 16), (-(-(share + 15) // 16), 16)):
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        p = {} if plan is None else dict(num_splits=plan[0], split_tokens=plan[1])
        if plan is None or cp * plan[0] <= 256:
            out, lse = fused(dq, kc, vc, t, sl, cp, I, err=err, **kw, **p)
            _check(out, lse, O, L, A, big, what=f"fused {plan}", **chk)
        po, pl = part(dq, kc, vc, t, sl, cp, I, err=err, **kw, **p)
        mo, ml = lib.cp_lse_merge(po, pl, out_dtype=DT[dt])
        _check(mo, ml, O, L, A, big, what=f"partials {plan}", **chk)
        assert int(err) == 0


@pytest.mark.parametrize("q4,dt", [(True, "bf16"), (False, "bf16"), (False, "f32")])
def test_decode_workspace_is_left_reusable_and_calls_repeat_bitwise(lib, q4, dt):
    case = ([200, 64, 1, 333], 16, 2, 128, 2, 8, dt, q4, 30.0, 0, False, False)
    c, q, _, _, O, L, A, big = _decode_case(*case)
    kc, vc, t = _dev(c)
    dq = torch.tensor(q, dtype=torch.float32).to(DT[dt]).to(DEV)
    sl = torch.tensor([200, 64, 1, 333], dtype=torch.int32, device=DEV)
    f = lib.cp_decode_attention_q4 if q4 else lib.cp_decode_attention_mod
    ws = torch.zeros(lib.cp_decode_workspace_size(4, 16, 2, 128, 2, 11), dtype=torch.uint8, device=DEV)
    kw = dict(num_splits=11, split_tokens=16, softcap=30.0, workspace=ws)
    first = f(dq, kc, vc, t, sl, 2, 8, **kw)
    again = [f(dq, kc, vc, t, sl, 2, 8, **kw) for _ in range(5)]
    assert all(torch.equal(first[i], x[i]) for x in again for i in range(2))
    assert not ws[:4 * 4 * 2].any()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    out, lse = torch.empty_like(first[0]), torch.empty_like(first[1])
    with torch.cuda.graph(g):
        f(dq, kc, vc, t, sl, 2, 8, out=out, out_lse=lse, **kw)
    for _ in range(3):
        out.zero_(), lse.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    sl.copy_(torch.tensor([10, 64, 1, 0], dtype=torch.int32))    # shorter lengths in the same graph
    g.replay()
    torch.cuda.synchronize()
    assert torch.isneginf(lse[3]).all() and not out[3].any()
    assert torch.equal(out[1:3], first[0][1:3])


@pytest.mark.parametrize("q4,dt", [(True, "bf16"), (False, "bf16"), (False, "f32")])
def test_decode_reports_bad_pages_and_short_plans(lib, q4, dt):
    case = ([400], 4, 1, 64, 2, 8, dt, q4, 0.0, 0, False, False)
    c, q, *_ = _decode_case(*case)
    kc, vc, t = _dev(c)
    dq = torch.tensor(q, dtype=torch.float32).to(DT[dt]).to(DEV)
    sl = torch.tensor([400], dtype=torch.int32, device=DEV)
    f = lib.cp_decode_attention_q4 if q4 else lib.cp_decode_attention_mod
    for bad in (-5, c.pool, 1 << 30):
        t2 = t.clone()
        t2[1, 0, 3] = bad
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        out, _ = f(dq, kc, vc, t2, sl, 2, 8, err=err)
        assert int(err) == 5 and bool(torch.isfinite(out.float()).all())
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    f(dq, kc, vc, t, sl, 2, 8, err=err, num_splits=2, split_tokens=64)      # covers 128 of 200
    assert int(err) == 5
    err.zero_()
    f(dq, kc, vc, t, sl, 2, 8, err=err, window=200, num_splits=2, split_tokens=64)
    assert int(err) == 0                                                      # 100 of a window


@pytest.mark.parametrize("q4", [True, False])
def test_nan_and_infinite_keys_reach_exactly_the_rows_that_see_them(lib, q4):
    d, lens = 128, [100, 100, 100]
    r = np.random.default_rng(5)
    c = Cache(lens, 1, d, 2, 8, torch.bfloat16, q4)
    for b in range(3):
        for p in range(100):
            k, v = _rows(r, (1, d), torch.bfloat16), _rows(r, (1, d), torch.bfloat16)
            if b == 1 and p == 50:
                v[0, 9] = np.nan
            if b == 2 and p == 50:
                k[0, 9] = np.nan
            c.put(b, p, k, v)
    kc, vc, t = _dev(c)
    q = torch.randn(3, 8, d, device=DEV).to(torch.bfloat16)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    f = lib.cp_decode_attention_q4 if q4 else lib.cp_decode_attention_mod
    out, lse = f(q, kc, vc, t, sl, 2, 8)
    assert bool(torch.isfinite(out[0].float()).all())
    nan = torch.isnan(out[1].float())
    assert bool(nan[:, 9].all()) and not bool(nan[:, 64:].any())
    assert q4 or int(nan.sum()) == 8
    assert bool(torch.isnan(out[2].float()).all()) and bool(torch.isnan(lse[2]).all())
    out, lse = f(q, kc, vc, t, sl, 2, 8, window=49)       # past the bad ones
    assert bool(torch.isfinite(out.float()).all()) and bool(torch.isfinite(lse).all())


# ------------------------------------------------------------------------------ prefill
PREFILLS = [
    # new, context, Hq, Hkv, d, cap, window, alibi, doc, prefix
    ([1], [0], 2, 1, 128, 0.0, 0, False, False, 0),
    ([1, 129, 0, 300], [0, 0, 5, 0], 4, 2, 128, 0.0, 0, False, False, 0),
    ([257], [0], 8, 2, 128, 50.0, 0, False, False, 0),
    ([200, 130], [33, 300], 6, 2, 64, 2.0, 0, False, False, 0),
    ([300, 77], [0, 150], 4, 2, 128, 0.0, 100, False, False, 0),
    ([513], [0], 3, 1, 128, 0.5, 1, False, False, 0),
    ([300], [40], 4, 4, 64, 0.0, 0, True, False, 0),
    ([290, 40], [0, 10], 6, 2, 128, 4.0, 0, True, False, 200),
    ([400, 1, 33], [0, 100, 7], 4, 2, 128, 0.0, 0, False, True, 0),
    ([300, 260], [20, 0], 10, 2, 64, 8.0, 150, True, True, 90),
    ([140], [500], 2, 2, 128, 0.0, 64, False, False, 600),
    ([600], [0], 2, 1, 64, 1.0, 300, False, True, 0),
    ([200, 31], [0, 60], 4, 2, 128, 100.0, 0, False, False, 0),     # a cap past the fixed reference's
    ([333], [0], 3, 1, 64, 55.0, 0, False, True, 40),
    ([150], [20], 2, 1, 128, 0.02, 0, False, False, 0),
]


def _prefill_inputs(new, ctx, Hq, Hkv, d, cap, window, alibi, doc, prefix, seed=3, pad=37):
    r = np.random.default_rng(seed)
    N, Nk = sum(new), sum(new) + sum(ctx)
    q = _rows(r, (N, Hq, d), torch.bfloat16) * (3.0 if cap else 1.0)     # scores past the cap's linear part
    k, v = _rows(r, (Nk, Hkv, d), torch.bfloat16), _rows(r, (Nk, Hkv, d), torch.bfloat16)
    slopes = np.array([2.0 ** (-8 * (h + 1) / Hq) for h in range(Hq)], np.float32).astype(float) if alibi else None
    pre = [min(prefix - 30 * b, n + x) for b, (n, x) in enumerate(zip(new, ctx))] if prefix else None
    start = None
    if doc:
        start = []
        for n, x in zip(new, ctx):
            at = 0
            for i in range(n):
                if r.random() < 0.02:
                    at = x + i
                start.append(x + n + 3 if r.random() < 0.03 else at)       # some rows see nothing
    return q, k, v, slopes, pre, start


def _prefill_oracle(new, ctx, q, k, v, d, cap, window, slopes, pre, start):
    O, L, A, big, r0, k0 = [], [], [], 0.0, 0, 0
    for b, (n, x) in enumerate(zip(new, ctx)):
        kk, vv = k[k0:k0 + n + x].transpose(1, 0, 2), v[k0:k0 + n + x].transpose(1, 0, 2)
        for i in range(n):
            lo, hi = so.bounds(x + i, x + n, window, start[r0 + i] if start else None, pre[b] if pre else 0)
            o, l, a, m = so.attend(q[r0 + i], kk, vv, x + i, lo, hi, 1 / math.sqrt(d), cap, slopes)
            O.append(o), L.append(l), A.append(a)
            big = max(big, m)
        r0, k0 = r0 + n, k0 + n + x
    return np.array(O), np.array(L), np.array(A), big


def _bf(x, pad=0, fill=float("nan")):
    t = torch.tensor(x, dtype=torch.float32).to(torch.bfloat16).to(DEV)
    if pad:
        t = torch.cat([t, torch.full((pad,) + t.shape[1:], fill, dtype=t.dtype, device=DEV)])
    return t


@pytest.mark.parametrize("case", PREFILLS, ids=[str(i) for i in range(len(PREFILLS))])
def test_prefill_against_the_oracle(lib, case):
    new, ctx, Hq, Hkv, d, cap, window, alibi, doc, prefix = case
    q, k, v, slopes, pre, start = _prefill_inputs(*case)
    dq, dk, dv = _bf(q, 37), _bf(k, 37), _bf(v, 37)      # NaN behind the last sequence
    q, k, v = _np(dq)[:len(q)], _np(dk)[:len(k)], _np(dv)[:len(v)]
    O, L, A, big = _prefill_oracle(new, ctx, q, k, v, d, cap, window, slopes, pre, start)
    N = len(q)
    i32 = dict(dtype=torch.int32, device=DEV)
    cu = torch.tensor(np.cumsum([0] + new), **i32)
    cukv = torch.tensor(np.cumsum([0] + [a + b for a, b in zip(new, ctx)]), **i32)
    out = torch.full((N + 37, Hq, d), 9.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((N + 37, Hq), 9.0, device=DEV)
    err = torch.zeros(1, **i32)
    lib.cp_attn_prefill_mod(dq, cu, dk, dv, cu_seqlens_kv=cukv, softcap=cap, window=window,
                            alibi_slopes=torch.tensor(slopes, dtype=torch.float32, device=DEV) if alibi else None,
                            kv_start=torch.tensor(start + [0] * 37, **i32) if doc else None,
                            prefix_lens=torch.tensor(pre, **i32) if prefix else None, max_seqlen_q=max(new), out=out,
                            out_lse=lse, err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    assert bool((out[N:] == 9.0).all()) and bool((lse[N:] == 9.0).all())
    _check(out[:N], lse[:N], O, L, A, big, cap=cap, slopes=slopes, length=max(a + b for a, b in zip(new, ctx)))


@pytest.mark.parametrize("d,Hq,Hkv", [(128, 4, 2), (64, 3, 1)])
@pytest.mark.parametrize("what", ["v_nan", "v_inf", "k_nan", "k_inf"])
def test_prefill_infinities_and_nan_stay_with_the_rows_that_see_them(lib, d, Hq, Hkv, what):
    """One bad key in the middle: rows before it (causal), of other documents, past the window and of
    the neighbouring sequences come out bit for bit as without it; rows that see it show it."""
    new = [150, 400, 60]
    r = np.random.default_rng(8)
    q, k, v = (_bf(r.normal(size=(610, h, d))) for h in (Hq, Hkv, Hkv))
    start = np.zeros(610, np.int32)
    start[150 + 300:550] = 300                      # a second document in the middle sequence
    i32 = dict(dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 150, 550, 610], **i32)
    kw = dict(window=120, kv_start=torch.tensor(start, **i32), max_seqlen_q=400)
    clean = lib.cp_attn_prefill_mod(q, cu, k, v, **kw)
    at = 150 + 230                                   # position 230 of the middle sequence
    k2, v2 = k.clone(), v.clone()
    bad = float("nan") if what.endswith("nan") else float("inf")
    (v2 if what[0] == "v" else k2)[at, 0, 5] = bad
    out, lse = lib.cp_attn_prefill_mod(q, cu, k2, v2, **kw)
    sees = torch.zeros(610, dtype=torch.bool, device=DEV)
    sees[at:150 + 300] = True                        # own document, from the key on, 120 keys wide
    G = Hq // Hkv
    heads = torch.arange(Hq, device=DEV) // G == 0
    same = ~(sees[:, None] & heads[None])
    assert torch.equal(out[same], clean[0][same]) and torch.equal(lse[same], clean[1][same])
    hit = out[sees][:, heads]
    if what == "v_nan":
        assert bool(torch.isnan(hit[..., 5].float()).all())
        assert torch.equal(lse, clean[1])
    elif what == "v_inf":
        assert bool((hit[..., 5] == float("inf")).all())
    elif what == "k_nan":
        assert bool(torch.isnan(hit.float()).all()) and bool(torch.isnan(lse[sees][:, heads]).all())
    else:   # a score of +inf (NaN weights) or -inf (no weight), by the sign of the query's component
        up = q[sees][:, heads][..., 5] > 0
        assert bool(torch.isnan(hit.float()).all(-1)[up].all())
        assert bool(torch.isfinite(hit.float()).all(-1)[q[sees][:, heads][..., 5] < 0].all())


def test_prefill_without_modification_is_the_fused_prefill(lib):
    r = np.random.default_rng(4)
    q, k, v = (_bf(r.normal(size=(700, h, 128))) for h in (8, 2, 2))
    cu = torch.tensor([0, 300, 700], dtype=torch.int32, device=DEV)
    a = lib.cp_attn_prefill_mod(q, cu, k, v)
    b = lib.cp_attn_prefill_fused(q, cu, 2, k, v)
    assert (a[1] - b[1]).abs().max() < 1e-4
    assert bool(((a[0].float() - b[0].float()).abs() <= 2.0 ** -6 * (1e-2 + b[0].float().abs())).all())


def test_prefill_flags_fewer_kv_tokens_than_queries(lib):
    q, k = torch.randn(20, 2, 64, device=DEV).to(torch.bfloat16), torch.randn(15, 2, 64, device=DEV).to(torch.bfloat16)
    i32 = dict(dtype=torch.int32, device=DEV)
    err = torch.zeros(1, **i32)
    lib.cp_attn_prefill_mod(q, torch.tensor([0, 20], **i32), k, k, cu_seqlens_kv=torch.tensor([0, 15], **i32), err=err)
    assert int(err) == 5


def test_prefill_in_a_cuda_graph_and_on_another_stream(lib):
    r = np.random.default_rng(6)
    q, k, v = (_bf(r.normal(size=(500, h, 128))) for h in (4, 2, 2))
    cu = torch.tensor([0, 500], dtype=torch.int32, device=DEV)
    want = lib.cp_attn_prefill_mod(q, cu, k, v, softcap=20.0, window=200, max_seqlen_q=500)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = lib.cp_attn_prefill_mod(q, cu, k, v, softcap=20.0, window=200, max_seqlen_q=500, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.cp_attn_prefill_mod(q, cu, k, v, softcap=20.0, window=200, max_seqlen_q=500, out=out, out_lse=lse)
    for _ in range(2):
        out.zero_(), lse.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


# ------------------------------------------------------------------------------ as they are used
@pytest.mark.parametrize("q4", [False, True])
def test_a_serving_run(lib, q4):
    """A prompt in two chunks and then single tokens: append with rotation, read the context back,
    attend it with capped scores, and decode over the cache; every step against attention in 64 bits
    over what the cache stands for."""
    Hq, Hkv, d, cp, I, cap, W = 8, 2, 128, 2, 8, 15.0, 90
    steps = [[70, 33], [41, 60], [1, 1], [1, 1], [1, 1]]
    r = np.random.default_rng(12)
    c = Cache([120, 110], Hkv, d, cp, I, torch.bfloat16, q4)
    kc, vc, t = _dev(c)
    f = 10000.0 ** (-np.arange(64) / 64)
    freq = torch.tensor(f, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    done = [0, 0]
    for new in steps:
        N = sum(new)
        q, k, v = (_bf(r.normal(size=(N, h, d))) for h in (Hq, Hkv, Hkv))
        cu, st = torch.tensor(np.cumsum([0] + new), **i32), torch.tensor(done, **i32)
        qr, _ = lib.cp_rope_kv_cache_write(k, v, cu, st, kc, vc, t, cp, I, inv_freq=freq, q=q)
        done = [a + b for a, b in zip(done, new)]
        cukv = torch.tensor(np.cumsum([0] + done), **i32)
        K, V = lib.cp_kv_cache_read(kc, vc, cukv, torch.zeros(2, **i32), t, cp, I, out_dtype=torch.bfloat16)
        ctx = [a - b for a, b in zip(done, new)]
        if max(new) > 1:
            out, lse = lib.cp_attn_prefill_mod(qr, cu, K, V, cu_seqlens_kv=cukv, softcap=cap, window=W)
            kn, vn = _np(K), _np(V)
        else:
            call = lib.cp_decode_attention_q4 if q4 else lib.cp_decode_attention_mod
            out, lse = call(qr, kc, vc, t, torch.tensor(done, **i32), cp, I, softcap=cap, window=W)
            if q4:   # decode reads the records themselves, not their rounding to bf16
                K, V = lib.cp_kv_cache_read(kc, vc, cukv, torch.zeros(2, **i32), t, cp, I, out_dtype=torch.float32)
            kn, vn = _np(K), _np(V)
        O, L, A, big = _prefill_oracle(new, ctx, _np(qr), kn, vn, d, cap, W, None, None, None)
        # 4-bit: the minima are at most as far out as the largest value
        A = A + (np.abs(vn).max() if q4 else 0)
        _check(out, lse, O, L, A, big, cap=cap, what=f"{new} after {ctx}")
