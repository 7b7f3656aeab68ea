"""The serving calls at sizes that fill many tiles, splits, clusters and waves, against attention in
float64 on the GPU (torch, over the rows cp_kv_cache_read gives, which the small tests pin), with the
tolerances of test_gpu_serving; pools past 32-bit offsets, hundreds of sequences, two streams at once."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
I32 = dict(dtype=torch.int32, device=DEV)


def _cu(lens):
    return torch.tensor(np.cumsum([0] + list(lens)), **I32)


def _pool(lens, Hkv, d, cp, I, dtype, q4, seed, extra=0):
    """A paged cache whose tables take their pages from the top of each rank's pool."""
    need = [max(1, -(-(-(-n // (I * cp)) * I) // 16)) for n in lens]
    pool = sum(need) + extra
    t = torch.full((cp, len(lens), max(need)), -1, dtype=torch.int32)
    g = torch.Generator().manual_seed(seed)
    for r in range(cp):
        ids = (extra + torch.randperm(sum(need), generator=g)).to(torch.int32)
        at = 0
        for b, n in enumerate(need):
            t[r, b, :n] = ids[at:at + n]
            at += n
    shape = (cp, pool, Hkv) + ((9 * d,) if q4 else (16, d))
    k, v = (torch.empty(shape, dtype=torch.uint8 if q4 else dtype, device=DEV) for _ in range(2))
    return k, v, t.to(DEV)


def _fill(lib, lens, Hkv, d, cp, I, dtype, q4, seed, extra=0):
    """The cache, filled with N(0, 1) rows of every position, and its rows in float64."""
    k, v, t = _pool(lens, Hkv, d, cp, I, dtype, q4, seed, extra)
    g = torch.Generator(device=DEV).manual_seed(seed)
    N = sum(lens)
    kn, vn = (torch.randn(N, Hkv, d, generator=g, device=DEV).to(dtype) for _ in range(2))
    zero = torch.zeros(len(lens), **I32)
    lib.cp_rope_kv_cache_write(kn, vn, _cu(lens), zero, k, v, t, cp, I)
    K, V = lib.cp_kv_cache_read(k, v, _cu(lens), zero, t, cp, I, out_dtype=torch.float32 if q4 else dtype)
    return k, v, t, K.double(), V.double()


def _attend(q, k, v, lo, hi, at, cap, slopes):
    """Queries q [i, Hq, d] over keys k, v [j, Hkv, d] (float64); out, lse, |v| average, largest
    scale sum |q||k|."""
    G, d = q.shape[1] // k.shape[1], q.shape[2]
    j = torch.arange(k.shape[0], device=DEV)
    seen = (j >= lo[:, None]) & (j < hi[:, None])
    kk, vv = (x.repeat_interleave(G, 1).permute(1, 0, 2) for x in (k, v))
    s = q.permute(1, 0, 2) @ kk.transpose(1, 2) / math.sqrt(d)
    big = float((q.abs().permute(1, 0, 2) @ kk.abs().transpose(1, 2)).max() / math.sqrt(d)) if s.numel() else 0.0
    if cap:
        s = cap * torch.tanh(s / cap)
    if slopes is not None:
        s = s - slopes.double()[:, None, None] * (at[:, None] - j).abs()
    s = s.masked_fill(~seen, -torch.inf)
    lse = torch.logsumexp(s, -1)
    w = torch.exp(s - lse.clamp(min=-1e300)[..., None])
    return (w @ vv).permute(1, 0, 2), lse.T, (w @ vv.abs()).permute(1, 0, 2), big


def _check(out, lse, O, L, A, big, cap, slopes, length, f32=False, extra=0.0, what=""):
    out, lse = out.double(), lse.double()
    fin = torch.isfinite(L)
    assert torch.equal(torch.isneginf(lse), ~fin), what
    e = 2.0 ** -16 * big + cap * 2.0 ** -20 + (float(slopes.max()) * length * 2.0 ** -22 if slopes is not None else 0) + \
        2.0 ** -22 * torch.where(fin, L.abs(), 0) + 1e-6
    assert bool(((lse - L).abs() <= e)[fin].all()), (what, float((lse - L).abs()[fin].max()))
    A = A + extra
    tol = (2 * e[..., None] + 2.0 ** -18) * A + (0 if f32 else 2.0 ** -8 * A + 2.0 ** -8 * O.abs()) + 1e-30
    d = (out - O).abs()
    assert bool((d <= tol).all()), (what, float((d / tol).max()))


LONG = [
    # B, longest, Hq, Hkv, d, cp, I, dtype, q4, cap, window, alibi, docs
    (1, 9000, 16, 2, 128, 2, 8, "bf16", True, 0.0, 0, False, False),       # several clusters per head
    (40, 3000, 32, 8, 128, 2, 8, "bf16", True, 0.0, 0, False, False),      # no clusters
    (3, 20000, 8, 8, 64, 4, 5, "bf16", True, 30.0, 5000, True, True),
    (70, 700, 24, 2, 128, 1, 16, "bf16", True, 0.0, 0, False, True),
    (1, 9000, 8, 1, 128, 8, 8, "bf16", False, 50.0, 0, False, False),
    (40, 3000, 32, 8, 128, 2, 8, "bf16", False, 0.0, 1111, True, False),
    (64, 1500, 32, 2, 64, 3, 1, "bf16", False, 5.0, 0, False, True),
    (2, 12000, 4, 2, 128, 2, 8, "f32", False, 0.0, 0, True, False),
    (60, 900, 16, 4, 64, 2, 8, "f32", False, 20.0, 333, False, True),
    # one to five query heads to a kv head: a tile of scores shared by two pages, and not
    (5, 400, 3, 3, 128, 2, 8, "bf16", True, 0.0, 0, False, True),
    (7, 300, 4, 2, 64, 1, 16, "bf16", True, 0.0, 100, True, False),
    (6, 1200, 6, 2, 128, 2, 1, "bf16", True, 15.0, 0, True, True),
    (9, 700, 8, 2, 64, 3, 5, "bf16", True, 0.0, 0, False, False),
    (5, 900, 10, 2, 128, 1, 8, "bf16", True, 0.0, 0, False, True),
    (64, 40, 4, 1, 128, 1, 8, "bf16", True, 0.0, 0, False, False),
]


@pytest.mark.parametrize("case", LONG, ids=[str(i) for i in range(len(LONG))])
def test_decode_of_long_and_many_sequences(lib, case):
    B, longest, Hq, Hkv, d, cp, I, dt, q4, cap, window, alibi, docs = case
    r = np.random.default_rng(B + longest)
    lens = [longest] + [int(n) for n in r.integers(1, longest + 1, B - 1)]
    kc, vc, t, K, V = _fill(lib, lens, Hkv, d, cp, I, DT[dt], q4, 1)
    q = torch.randn(B, Hq, d, device=DEV).to(DT[dt])
    slopes = 2.0 ** (-8 * (torch.arange(Hq, device=DEV, dtype=torch.float32) + 1) / Hq) if alibi else None
    start = torch.tensor([int(r.integers(0, n)) if i % 5 else n for i, n in enumerate(lens)], **I32) if docs else None
    sl = torch.tensor(lens, **I32)
    O, L, A, big, at = [], [], [], 0.0, 0
    for b, n in enumerate(lens):
        lo = max(0, n - window if window else 0, int(start[b]) if docs else 0)
        one = torch.tensor([n - 1], device=DEV)
        o, l, a, m = _attend(q[b:b + 1].double(), K[at:at + n], V[at:at + n], torch.tensor([lo], device=DEV), one + 1,
                             one, cap, slopes)
        O.append(o), L.append(l), A.append(a)
        big, at = max(big, m), at + n
    O, L, A = torch.cat(O), torch.cat(L), torch.cat(A)
    fused, part = ((lib.cp_decode_attention_q4, lib.cp_partial_attn_decode_q4) if q4 else
                   (lib.cp_decode_attention_mod, lib.cp_partial_attn_decode_mod))
    kw = dict(softcap=cap, window=window, alibi_slopes=slopes, kv_start=start)
    # 4-bit: what P's rounding meets is value - minimum; no minimum is further out than the largest value
    chk = dict(cap=cap, slopes=slopes, length=longest, f32=dt == "f32", extra=float(V.abs().max()) if q4 else 0.0)
    err = torch.zeros(1, **I32)
    plan = lib.cp_decode_mod_plan(B, Hkv, cp, I, longest, window=window, q4=q4)
    for splits, tokens in (plan, (256 // cp, -(-(-(-longest // (I * cp)) * I + 15) // (256 // cp) // 16) * 16 + 16)):
        out, lse = fused(q, kc, vc, t, sl, cp, I, num_splits=splits, split_tokens=tokens, err=err, **kw)
        _check(out, lse, O, L, A, big, what=f"fused {splits} x {tokens}", **chk)
    po, pl = part(q, kc, vc, t, sl, cp, I, num_splits=plan[0], split_tokens=plan[1], err=err, **kw)
    mo, ml = lib.cp_lse_merge(po, pl, out_dtype=DT[dt])
    _check(mo, ml, O, L, A, big, what="partials", **chk)
    assert int(err) == 0


PREFILL = [
    # new, context, Hq, Hkv, d, cap, window, alibi, doc, prefix
    ([1500, 700], [0, 900], 8, 2, 128, 0.0, 0, False, 0, 0),
    ([2048], [0], 4, 2, 128, 50.0, 0, False, 0, 0),
    ([1111, 1, 530], [3, 700, 0], 6, 2, 64, 30.0, 400, False, 0, 0),
    ([1900], [100], 3, 1, 128, 0.0, 0, True, 0, 500),
    ([900, 1300], [0, 0], 10, 2, 128, 3.0, 700, True, 150, 0),
    ([1700], [0], 9, 3, 64, 20.0, 0, False, 60, 0),
    ([1024], [1024], 2, 2, 128, 0.0, 1024, False, 0, 1500),
    ([640] * 3, [0, 640, 1280], 16, 8, 64, 100.0, 0, True, 300, 64),
]


@pytest.mark.parametrize("case", PREFILL, ids=[str(i) for i in range(len(PREFILL))])
def test_prefill_of_many_tiles(lib, case):
    new, ctx, Hq, Hkv, d, cap, window, alibi, doc, prefix = case
    r = np.random.default_rng(sum(new))
    tot = [a + b for a, b in zip(new, ctx)]
    q = (torch.randn(sum(new), Hq, d, device=DEV) * (2 if cap else 1)).to(torch.bfloat16)
    k, v = (torch.randn(sum(tot), Hkv, d, device=DEV).to(torch.bfloat16) for _ in range(2))
    slopes = 2.0 ** (-8 * (torch.arange(Hq, device=DEV, dtype=torch.float32) + 1) / Hq) if alibi else None
    pre = [int(r.integers(0, prefix + 1)) for _ in new] if prefix else None
    start = []
    for n, x in zip(new, ctx):
        at = 0
        for i in range(n):
            at = x + i if doc and r.random() < 1.0 / doc else at
            start.append(x + n if doc and r.random() < 0.01 else at)
    start = torch.tensor(start, **I32)
    err = torch.zeros(1, **I32)
    out, lse = lib.cp_attn_prefill_mod(q, _cu(new), k, v, cu_seqlens_kv=_cu(tot), softcap=cap, window=window,
                                       alibi_slopes=slopes, kv_start=start if doc else None,
                                       prefix_lens=torch.tensor(pre, **I32) if prefix else None, max_seqlen_q=max(new),
                                       err=err)
    assert int(err) == 0
    r0 = k0 = 0
    for b, (n, x) in enumerate(zip(new, ctx)):
        at = torch.arange(x, x + n, device=DEV)
        lo = (at - window + 1).clamp(min=0) if window else torch.zeros_like(at)
        if doc:
            lo = torch.maximum(lo, start[r0:r0 + n].long())
        hi = (at + 1).clamp(min=min(pre[b], n + x) if prefix else 0)
        O, L, A, big = _attend(q[r0:r0 + n].double(), k[k0:k0 + n + x].double(), v[k0:k0 + n + x].double(), lo, hi, at,
                               cap, slopes)
        _check(out[r0:r0 + n], lse[r0:r0 + n], O, L, A, big, cap, slopes, n + x, what=f"sequence {b}")
        r0, k0 = r0 + n, k0 + n + x


@pytest.mark.parametrize("q4,dt,d", [(True, "bf16", 128), (True, "bf16", 64), (False, "bf16", 128), (False, "f32", 64)])
def test_pools_past_32_bit_offsets(lib, q4, dt, d):
    """The same cache with its pages behind more than 2^32 bytes (2^31 elements) of each rank's pool."""
    Hkv, cp, I, lens = 8, 2, 8, [700, 33]
    page = Hkv * (9 * d if q4 else 16 * d * (2 if dt == "bf16" else 4))
    q = torch.randn(2, 16, d, device=DEV).to(DT[dt])
    got = []
    for extra in (0, (1 << 32) // page + 1000):
        k, v, t, K, V = _fill(lib, lens, Hkv, d, cp, I, DT[dt], q4, 3, extra)
        call = lib.cp_decode_attention_q4 if q4 else lib.cp_decode_attention_mod
        err = torch.zeros(1, **I32)
        out, lse = call(q, k, v, t, torch.tensor(lens, **I32), cp, I, num_splits=3, split_tokens=128, err=err)
        assert int(err) == 0
        got.append((K, V, out, lse))
        del k, v
        torch.cuda.empty_cache()
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("q4", [False, True])
def test_hundreds_of_sequences_some_empty(lib, q4):
    """More sequences than a warp compares at once (the search for a row's sequence)."""
    r = np.random.default_rng(2)
    for B in (31, 300, 1000):
        lens = [int(n) if n < 9 else 0 for n in r.integers(0, 12, B)]
        lens[-1] = lens[-1] or 3
        k, v, t, K, V = _fill(lib, lens, 2, 64, 2, 8, torch.bfloat16, q4, 5)
        g = torch.Generator(device=DEV).manual_seed(5)
        kn, vn = (torch.randn(sum(lens), 2, 64, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
        for a, b in ((K, kn), (V, vn)):
            if not q4:
                assert torch.equal(a, b.double())
            else:   # within half a step of a group's range / 15, and its ends' rounding to bf16
                span = (b.double().amax(-1, keepdim=True) - b.double().amin(-1, keepdim=True))
                assert bool(((a - b.double()).abs() <= span / 30 + 2.0 ** -6 * b.double().abs().amax(-1, keepdim=True)).all())


def test_a_large_cap_leaves_the_scores_as_they_are(lib):
    """tanh of a small argument keeps its relative accuracy: with a cap of 10^5 the scores change by
    less than s^3 / (3 cap^2) < 2^-20, and the cap's arithmetic by 2^-20 of a score (below 2^4)."""
    for q4, dt in ((True, "bf16"), (False, "bf16"), (False, "f32")):
        k, v, t, K, V = _fill(lib, [900], 2, 128, 2, 8, DT[dt], q4, 7)
        q = torch.randn(1, 8, 128, device=DEV).to(DT[dt])
        call = lib.cp_decode_attention_q4 if q4 else lib.cp_decode_attention_mod
        a, b = (call(q, k, v, t, torch.tensor([900], **I32), 2, 8, softcap=c)[1] for c in (0.0, 1e5))
        assert float((a - b).abs().max()) <= 2.0 ** -16 + 2.0 ** -20
    q, k, v = (torch.randn(300, h, 128, device=DEV).to(torch.bfloat16) for h in (4, 2, 2))
    a, b = (lib.cp_attn_prefill_mod(q, _cu([300]), k, v, softcap=c)[1] for c in (0.0, 1e5))
    assert float((a - b).abs().max()) <= 2.0 ** -16 + 2.0 ** -20


def test_two_streams_at_once(lib):
    """Decode, prefill and append on two streams, each with its own workspace and cache, give what they
    give alone."""
    runs = []
    for seed in (1, 2):
        lens = [1500, 700 * seed]
        k, v, t, K, V = _fill(lib, lens, 2, 128, 2, 8, torch.bfloat16, True, seed)
        q = torch.randn(2, 16, 128, device=DEV).to(torch.bfloat16)
        plan = lib.cp_decode_mod_plan(2, 2, 2, 8, 1500, q4=True)
        ws = torch.zeros(lib.cp_decode_workspace_size(2, 16, 2, 128, 2, plan[0]), dtype=torch.uint8, device=DEV)
        pq, pk, pv = (torch.randn(600, h, 128, device=DEV).to(torch.bfloat16) for h in (4, 2, 2))
        cu, sl, cu1 = _cu([600]), torch.tensor(lens, **I32), _cu([1, 1])
        kn = torch.randn(2, 2, 128, device=DEV).to(torch.bfloat16)
        freq = torch.tensor(10000.0 ** (-np.arange(64) / 64), device=DEV)

        def step(k=k, v=v, t=t, q=q, plan=plan, ws=ws, pq=pq, pk=pk, pv=pv, cu=cu, sl=sl, cu1=cu1, kn=kn, freq=freq):
            q2, _ = lib.cp_rope_kv_cache_write(kn, kn, cu1, sl - 1, k, v, t, 2, 8, inv_freq=freq, q=q)
            a = lib.cp_decode_attention_q4(q2, k, v, t, sl, 2, 8, num_splits=plan[0], split_tokens=plan[1], workspace=ws)
            b = lib.cp_attn_prefill_mod(pq, cu, pk, pv, softcap=30.0, window=200, max_seqlen_q=600)
            return a + b
        runs.append(step)
    want = [s() for s in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(20):
        got = []
        for s, f in zip(streams, runs):
            with torch.cuda.stream(s):
                got.append(f())
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_a_decode_step_in_a_cuda_graph(lib):
    """Append and decode captured together: each replay appends at the position in device memory and
    attends what is there, as the eager calls do."""
    B, Hq, Hkv, d, cp, I = 3, 16, 2, 128, 2, 8
    lens = [900, 40, 333]
    for q4 in (True, False):
        k, v, t, _, _ = _fill(lib, [n + 8 for n in lens], Hkv, d, cp, I, torch.bfloat16, q4, 4)
        k2, v2 = k.clone(), v.clone()
        call = lib.cp_decode_attention_q4 if q4 else lib.cp_decode_attention_mod
        plan = lib.cp_decode_mod_plan(B, Hkv, cp, I, 1000, q4=q4)
        ws = torch.zeros(lib.cp_decode_workspace_size(B, Hq, Hkv, d, cp, plan[0]), dtype=torch.uint8, device=DEV)
        qkv = torch.empty(B, Hq + 2 * Hkv, d, dtype=torch.bfloat16, device=DEV)
        sl, start, cu = torch.tensor(lens, **I32), torch.tensor(lens, **I32), _cu([1] * B)
        freq = torch.tensor(10000.0 ** (-np.arange(64) / 64), device=DEV)

        def step(k, v, ws):
            q, kn, vn = qkv.split([Hq, Hkv, Hkv], 1)
            q, _ = lib.cp_rope_kv_cache_write(kn, vn, cu, start, k, v, t, cp, I, inv_freq=freq, q=q)
            return call(q, k, v, t, sl, cp, I, softcap=50.0, num_splits=plan[0], split_tokens=plan[1], workspace=ws)
        qkv.normal_()
        step(k2, v2, torch.zeros_like(ws))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out, lse = step(k, v, ws)
        for i in range(4):
            qkv.normal_()
            start.copy_(torch.tensor([n + i for n in lens], dtype=torch.int32))
            sl.copy_(torch.tensor([n + i + 1 for n in lens], dtype=torch.int32))
            g.replay()
            want = step(k2, v2, torch.zeros_like(ws))
            torch.cuda.synchronize()
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("dt,d", [("f32", 128), ("bf16", 64), ("f32", 64)])
def test_nearly_constant_rows_in_four_bits(lib, dt, d):
    """A group whose minimum rounds above its greatest value is stored as that minimum with scale 0, and
    decodes as such (a negative scale would make infinite weights of zero codes)."""
    cp, I, lens = 2, 8, [50, 33]
    k, v, t = _pool(lens, 2, d, cp, I, torch.uint8, True, 6)
    k.zero_(), v.zero_()        # (pages end behind the sequences: their last rows are never written)
    g = torch.Generator(device=DEV).manual_seed(6)
    level = torch.tensor([257.3, -0.70123, 1000.9, 3e-5], device=DEV)
    kn, vn = (level[torch.randint(0, 4, (sum(lens), 2, 1), generator=g, device=DEV)].expand(-1, -1, d) *
              (1 + 1e-5 * torch.rand(sum(lens), 2, d, generator=g, device=DEV)) for _ in range(2))
    kn, vn = kn.to(DT[dt]).contiguous(), vn.to(DT[dt]).contiguous()
    zero = torch.zeros(2, **I32)
    lib.cp_rope_kv_cache_write(kn, vn, _cu(lens), zero, k, v, t, cp, I)
    scales = [x[..., 8 * d:].contiguous().view(torch.bfloat16)[..., ::2] for x in (k, v)]
    assert all(bool((s.float()[torch.isfinite(s.float())] >= 0).all()) for s in scales)
    K, V = lib.cp_kv_cache_read(k, v, _cu(lens), zero, t, cp, I, out_dtype=torch.float32)
    assert bool(((V - vn.float()).abs() <= 2.0 ** -8 * vn.float().abs()).all())
    q = torch.randn(2, 8, d, device=DEV, generator=g).to(torch.bfloat16) * 0.02
    out, lse = lib.cp_decode_attention_q4(q, k, v, t, torch.tensor(lens, **I32), cp, I)
    at = 0
    for b, n in enumerate(lens):
        one = torch.tensor([n - 1], device=DEV)
        o, l, a, big = _attend(q[b:b + 1].double(), K[at:at + n].double(), V[at:at + n].double(), 0 * one, one + 1, one, 0.0, None)
        _check(out[b:b + 1], lse[b:b + 1], o, l, a, big, 0.0, None, n, extra=float(V.abs().max()), what=f"sequence {b}")
        at += n


def test_calls_that_feed_one_another(lib):
    """Append, decode, read-back and prefill one after the other, each on what the one before it wrote,
    with nothing between them, give what they give with a synchronization after each."""
    B, Hq, Hkv, d, cp, I, L = 3, 8, 2, 128, 2, 8, 40
    g = torch.Generator(device=DEV).manual_seed(8)
    first = torch.randn(B, Hq + 2 * Hkv, d, generator=g, device=DEV).to(torch.bfloat16)
    freq = torch.tensor(10000.0 ** (-np.arange(64) / 64), device=DEV)
    cu1 = _cu([1] * B)
    starts = [torch.full((B,), i, **I32) for i in range(L + 1)]
    cus = [_cu([i] * B) for i in range(L + 1)]
    for q4 in (False, True):
        results = []
        for wait in (True, False, False, False):
            k, v, t = _pool([L] * B, Hkv, d, cp, I, torch.bfloat16, q4, 1)
            k.zero_(), v.zero_()
            call = lib.cp_decode_attention_q4 if q4 else lib.cp_decode_attention_mod
            ws = torch.zeros(lib.cp_decode_workspace_size(B, Hq, Hkv, d, cp, 2), dtype=torch.uint8, device=DEV)
            x, seen = first, []
            for i in range(L):
                q, kn, vn = x.split([Hq, Hkv, Hkv], 1)
                q, _ = lib.cp_rope_kv_cache_write(kn, vn, cu1, starts[i], k, v, t, cp, I, inv_freq=freq, q=q)
                if wait:
                    torch.cuda.synchronize()
                o, l = call(q, k, v, t, starts[i + 1], cp, I, num_splits=2, split_tokens=16, workspace=ws)
                if wait:
                    torch.cuda.synchronize()
                rk, rv = lib.cp_kv_cache_read(k, v, cus[i + 1], starts[0], t, cp, I, total=B * (i + 1), out_dtype=torch.bfloat16)
                if wait:
                    torch.cuda.synchronize()
                p, pl = lib.cp_attn_prefill_mod(o, cu1, rk, rv, cu_seqlens_kv=cus[i + 1], max_seqlen_q=1, softcap=9.0)
                if wait:
                    torch.cuda.synchronize()
                x = torch.cat([p, rk.view(B, i + 1, Hkv, d)[:, i], o[:, :Hkv]], 1)
                seen += [o, l, rk, rv, p, pl]
            torch.cuda.synchronize()
            results.append(seen)
        for other in results[1:]:
            assert all(torch.equal(a, b) for a, b in zip(results[0], other))


@pytest.mark.parametrize("q4", [True, False])
def test_two_graphs_share_a_workspace(lib, q4):
    """Two captured decodes of different shapes over one workspace, replayed in turn with eager calls
    between: every call leaves the workspace as the next one, of whatever shape, needs it."""
    graphs, wants, outs = [], [], []
    shapes = [(2, [900, 333], 16, 2, 6, 96), (40, [700] * 40, 16, 2, 3, 128)]      # in one cluster's reach, and not
    need = max(lib.cp_decode_workspace_size(B, Hq, Hkv, 128, 2, S) for B, _, Hq, Hkv, S, _ in shapes)
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    call = lib.cp_decode_attention_q4 if q4 else lib.cp_decode_attention_mod
    runs = []
    for B, lens, Hq, Hkv, S, tokens in shapes:
        k, v, t, _, _ = _fill(lib, lens, Hkv, 128, 2, 8, torch.bfloat16, q4, 1)
        q, sl = torch.randn(B, Hq, 128, device=DEV).to(torch.bfloat16), torch.tensor(lens, **I32)

        def run(q=q, k=k, v=v, t=t, sl=sl, S=S, tokens=tokens):
            return call(q, k, v, t, sl, 2, 8, num_splits=S, split_tokens=tokens, workspace=ws)
        runs.append(run)
        wants.append([x.clone() for x in run()])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run())
        graphs.append(g)
    for i in (0, 1, 1, 0, 0, 1, 0, 1, 1, 0):
        for x in outs[i]:
            x.zero_()
        graphs[i].replay()
        between = runs[1 - i]()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs[i], wants[i]))
        assert all(torch.equal(a, b) for a, b in zip(between, wants[1 - i]))
    assert int(ws[:4 * 80].max()) == 0              # the counters are back at zero


def test_the_plain_decode_shares_a_workspace_between_shapes(lib):
    """cp_decode_attention, and the calls with modified scores after it, over one workspace."""
    ws, runs = None, []
    for B, L, S, tokens in ((2, 900, 6, 96), (40, 700, 6, 64)):
        k, v, t, _, _ = _fill(lib, [L] * B, 2, 128, 2, 8, torch.bfloat16, False, 1)
        q, sl = torch.randn(B, 16, 128, device=DEV).to(torch.bfloat16), torch.full((B,), L, **I32)
        for call in (lib.cp_decode_attention, lib.cp_decode_attention_mod):
            def run(ws, call=call, q=q, k=k, v=v, t=t, sl=sl, S=S, tokens=tokens):
                return call(q, k, v, t, sl, 2, 8, num_splits=S, split_tokens=tokens, workspace=ws)
            runs.append((run, [x.clone() for x in run(None)]))
    ws = torch.zeros(max(lib.cp_decode_workspace_size(B, 16, 2, 128, 2, 6) for B in (2, 40)), dtype=torch.uint8, device=DEV)
    for i in (0, 2, 1, 3, 2, 0, 3, 1, 0, 3):
        run, want = runs[i]
        assert all(torch.equal(a, b) for a, b in zip(run(ws), want))


def test_prefill_reports_a_sequence_past_max_seqlen_q(lib):
    for Hq, Hkv in ((4, 2), (3, 1)):
        q, k, v = (torch.randn(700, h, 64, device=DEV).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
        full, _ = lib.cp_attn_prefill_mod(q, _cu([100, 600]), k, v, max_seqlen_q=600)
        for longest, flagged in ((600, 0), (700, 0), (256, 5)):
            err, out = torch.zeros(1, **I32), torch.zeros_like(q)
            lib.cp_attn_prefill_mod(q, _cu([100, 600]), k, v, max_seqlen_q=longest, out=out, err=err)
            assert int(err) == flagged and torch.equal(out[:356], full[:356])
            assert torch.equal(out[356:], full[356:]) if not flagged else not out[356:].any()


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 128), (3, 1, 64)])
@pytest.mark.parametrize("cap", [0.0, 30.0, 50.0, 100.0])
def test_prefill_rows_of_one_key_are_that_keys_value(lib, Hq, Hkv, d, cap):
    """With a window of one key, and with documents of one token, every output is its own value row bit for
    bit: the weight of a row's only key is 1, wherever in the sequence it lies."""
    n = 700
    q, k, v = (torch.randn(n, h, d, device=DEV).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    want = v.repeat_interleave(Hq // Hkv, 1)
    start = torch.arange(n, **I32)
    for kw in (dict(window=1), dict(kv_start=start), dict(kv_start=start, window=300)):
        out, _ = lib.cp_attn_prefill_mod(q, _cu([n]), k, v, softcap=cap, max_seqlen_q=n, **kw)
        assert torch.equal(out, want)
