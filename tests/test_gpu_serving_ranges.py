"""Values far apart in size, and scores at the ends of their range, in the serving calls."""
import math

import numpy as np
import pytest
import torch

from test_gpu_serving_large import DEV, I32, _attend, _check, _cu, _pool

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------ V's range, 4 bits
def _minima(pool, t, n, cp, I, d):
    """Each value's group minimum of positions 0..n-1 of sequence 0, [n, Hkv, d], in float64."""
    p = np.arange(n)
    turn = p // I
    rank, local = turn % cp, turn // cp * I + p % I
    page = t.cpu().numpy()[rank, 0, local // 16]
    rec = pool[torch.tensor(rank, device=DEV), torch.tensor(page, device=DEV).long()]        # [n, Hkv, 9 d]
    at = torch.tensor(local % 16, device=DEV)
    pairs = rec[..., 8 * d:].reshape(n, rec.shape[1], 16, d // 16).contiguous()
    pairs = pairs[torch.arange(n, device=DEV), :, at].contiguous().view(torch.bfloat16)      # scale, minimum, ..
    return pairs[..., 1::2].double().repeat_interleave(64, -1)


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 1, 128), (8, 1, 128), (16, 1, 128), (6, 2, 64), (14, 1, 64)])
@pytest.mark.parametrize("cap", [0.0, 500.0])
@pytest.mark.parametrize("rise,fall", [(60.0, 16), (60.0, 24), (60.0, 40), (25.0, 30), (12.0, 12), (9.0, 9), (100.0, 50), (30.0, 7), (12.0, 25), (8.5, 20)])
def test_v_scales_that_fall_while_the_scores_rise(lib, Hq, Hkv, d, cap, rise, fall):
    """The tokens of each later part of the sequence score `rise` (in powers of two) more and their V is 2^-fall
    as large: the parts before it count for nothing then, and what they left behind must not cost the later ones
    their bits.  V's smallest value is near 0 in half of the groups, so that the minima do not stand in for it.

    Tolerance: that of the 4-bit decode (see test_gpu_serving), with |value - minimum| <= |value| + |minimum|
    of the tokens that count.  A factor that is 2^k below the largest that counts is off by 2^-25 2^k units: with
    2^-8 allowed and up to a few hundred equal weights, that needs no term of its own."""
    parts, n, cp, I = 3, 3 * 192, 1, 16
    k, v, t = _pool([n], Hkv, d, cp, I, torch.bfloat16, True, 3)
    g = torch.Generator(device=DEV).manual_seed(4)
    part = torch.arange(n, device=DEV) // 192
    # q = c (1, .., 1), k = a (1, .., 1) + little: q.k / sqrt(d) = c a sqrt(d)
    c = 2.0
    level = (part.double() - (parts - 1)) * rise * math.log(2) / (c * math.sqrt(d))
    kn = (level[:, None, None] + 0.02 * torch.randn(n, Hkv, d, generator=g, device=DEV)).to(torch.bfloat16)
    vn = torch.rand(n, Hkv, d, generator=g, device=DEV)
    vn[:, :, :32] = 2 * vn[:, :, :32] - 1
    vn = (vn * (2.0 ** (fall * (parts - 1 - part.double())))[:, None, None]).to(torch.bfloat16)
    lib.cp_rope_kv_cache_write(kn, vn, _cu([n]), torch.zeros(1, **I32), k, v, t, cp, I)
    K, V = (x.double() for x in lib.cp_kv_cache_read(k, v, _cu([n]), torch.zeros(1, **I32), t, cp, I, out_dtype=torch.float32))
    M = _minima(v, t, n, cp, I, d)
    q = torch.full((1, Hq, d), c, dtype=torch.bfloat16, device=DEV)
    one = torch.tensor([n - 1], device=DEV)
    O, L, A, big = _attend(q.double(), K, V, 0 * one, one + 1, one, cap, None)
    extra = _attend(q.double(), K, M.abs(), 0 * one, one + 1, one, cap, None)[0]
    for S, tokens in ((1, 576), (3, 192), (2, 320)):
        out, lse = lib.cp_decode_attention_q4(q, k, v, t, torch.tensor([n], **I32), cp, I, softcap=cap, num_splits=S, split_tokens=tokens)
        _check(out, lse, O, L, A, big, cap, None, n, extra=extra, what=f"{S} x {tokens}")


# ------------------------------------------------------------------------------ capped prefill
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 128), (3, 1, 64)])
@pytest.mark.parametrize("cap", [4.0, 30.0, 100.0, 1e5, 1e9])
@pytest.mark.parametrize("bad", ["inf", "nan", "large", "huge"])
def test_keys_a_row_does_not_see_leave_its_capped_scores_alone(lib, Hq, Hkv, d, cap, bad):
    """One bad key in the middle, and bad rows behind the last sequence: rows that do not see it come out bit for
    bit as without it, with a cap and with a cap and a bias."""
    new = [150, 400, 60]
    r = torch.Generator(device=DEV).manual_seed(8)
    q, k, v = (torch.randn(610, h, d, generator=r, device=DEV).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    start = torch.zeros(610, **I32)
    start[150 + 300:550] = 300                       # a second document in the middle sequence
    at = 150 + 230                                   # position 230 of the middle sequence
    k2 = k.clone()
    k2[at, 0, 5] = dict(inf=float("inf"), nan=float("nan"), large=1e4, huge=1e30)[bad]
    sees = torch.zeros(610, dtype=torch.bool, device=DEV)
    sees[at:150 + 300] = True                        # own document, from the key on, 120 keys wide
    same = ~(sees[:, None] & (torch.arange(Hq, device=DEV) // (Hq // Hkv) == 0)[None])
    slopes = 2.0 ** (-8 * (torch.arange(Hq, device=DEV, dtype=torch.float32) + 1) / Hq)
    for alibi in (None, slopes):
        kw = dict(window=120, kv_start=start, max_seqlen_q=400, softcap=cap, alibi_slopes=alibi)
        clean = lib.cp_attn_prefill_mod(q, _cu(new), k, v, **kw)
        out, lse = lib.cp_attn_prefill_mod(q, _cu(new), k2, v, **kw)
        assert torch.equal(out[same], clean[0][same]) and torch.equal(lse[same], clean[1][same])


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 128), (3, 1, 64)])
@pytest.mark.parametrize("cap", [0.5, 2.0, 20.0, 1e6, 1e9])
def test_small_and_large_scores_under_one_cap(lib, Hq, Hkv, d, cap):
    """Rows whose scores lie far below the cap next to rows (of the same warp) far above it: each to the accuracy
    of its own scores, 2^-16 of the products' sum and 2^-20 of the capped score (tanh x <= x)."""
    n = 300
    g = torch.Generator(device=DEV).manual_seed(6)
    q, k, v = (torch.randn(n, h, d, generator=g, device=DEV) for h in (Hq, Hkv, Hkv))
    q[::2] *= 4 * cap
    q, k, v = (x.to(torch.bfloat16) for x in (q, k, v))
    out, lse = lib.cp_attn_prefill_mod(q, _cu([n]), k, v, softcap=cap, max_seqlen_q=n)
    for i in (0, 1, 2, 129, 200, 298, 299):
        one = torch.tensor([i], device=DEV)
        O, L, A, big = _attend(q[i:i + 1].double(), k.double(), v.double(), 0 * one, one + 1, one, cap, None)
        _check(out[i:i + 1], lse[i:i + 1], O, L, A, min(big, 64 * cap) if i % 2 == 0 else big, min(cap, big), None, n, what=f"row {i}")


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 128), (3, 1, 64)])
@pytest.mark.parametrize("cap,up", [(50.0, 40), (30.0, 40), (55.0, 40), (50.0, 90), (300.0, 90)])
def test_capped_prefill_with_large_values_and_late_high_scores(lib, Hq, Hkv, d, cap, up):
    """Scores at the cap's lower end in the first key tiles and at its upper end behind them, V up to 2^up.

    Caps up to 55: scores past 7 caps, where tanh is 1 to 2^-20 whatever the products' sum is off by."""
    n = 700
    g = torch.Generator(device=DEV).manual_seed(5)
    q = torch.full((n, Hq, d), 8.0, dtype=torch.bfloat16, device=DEV)
    k = torch.full((n, Hkv, d), -8.0, dtype=torch.bfloat16, device=DEV)
    k[200:] = 8.0
    k = k * (1 + 0.25 * torch.rand(n, Hkv, 1, generator=g, device=DEV)).to(torch.bfloat16)
    v = ((0.5 + torch.rand(n, Hkv, d, generator=g, device=DEV) / 2) * 2.0 ** up).to(torch.bfloat16)
    out, lse = lib.cp_attn_prefill_mod(q, _cu([n]), k, v, softcap=cap, max_seqlen_q=n)
    at = torch.arange(n, device=DEV)
    O, L, A, big = _attend(q.double(), k.double(), v.double(), 0 * at, at + 1, at, cap, None)
    # 300: scores of 2 to 3 caps, whose tanh changes by at most 0.07 of what the products' sum is off by
    _check(out, lse, O, L, A, 1.0 if cap < 100 else big, cap, None, n)


@pytest.mark.parametrize("kind", ["bf16", "f32", "q4"])
@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_decode_of_the_largest_values(lib, kind, cap):
    """V just below 2^96, the bound that the header gives, under scores that rise along the sequence."""
    n, Hq, Hkv, d, cp, I = 1500, 8, 2, 128, 2, 8
    dt, q4 = torch.float32 if kind == "f32" else torch.bfloat16, kind == "q4"
    k, v, t = _pool([n], Hkv, d, cp, I, dt, q4, 3)
    g = torch.Generator(device=DEV).manual_seed(4)
    kn = (torch.linspace(-2, 2, n, device=DEV)[:, None, None] + 0.1 * torch.randn(n, Hkv, d, generator=g, device=DEV)).to(dt)
    vn = ((2 * torch.rand(n, Hkv, d, generator=g, device=DEV) - 1) * 2.0 ** 95.9).to(dt)
    zero = torch.zeros(1, **I32)
    lib.cp_rope_kv_cache_write(kn, vn, _cu([n]), zero, k, v, t, cp, I)
    K, V = (x.double() for x in lib.cp_kv_cache_read(k, v, _cu([n]), zero, t, cp, I, out_dtype=torch.float32 if q4 else dt))
    q = torch.full((1, Hq, d), 1.5, dtype=dt, device=DEV)
    one = torch.tensor([n - 1], device=DEV)
    O, L, A, big = _attend(q.double(), K, V, 0 * one, one + 1, one, cap, None)
    fused = lib.cp_decode_attention_q4 if q4 else lib.cp_decode_attention_mod
    for S, tokens in ((1, 752), (6, 128)):
        out, lse = fused(q, k, v, t, torch.tensor([n], **I32), cp, I, softcap=cap, num_splits=S, split_tokens=tokens)
        _check(out, lse, O, L, A, big, cap, None, n, f32=kind == "f32", extra=float(V.abs().max()) if q4 else 0.0, what=f"{S} x {tokens}")


@pytest.mark.parametrize("cap,scale", [(1e-6, 1e3), (1e-3, 1e4), (1e-6, 1e-11), (1e-6, 1e-9), (1e9, 1e4), (1e9, 1e14), (3.0, 1e6)])
def test_capped_prefill_at_the_ends_of_cap_and_scale(lib, cap, scale):
    """Caps and softmax scales at the ends of what the calls take, with rows of zeros (scores of 0 under any of
    them), small and ordinary rows."""
    n, Hq, Hkv, d = 640, 4, 2, 64
    g = torch.Generator(device=DEV).manual_seed(7)
    q, k, v = (torch.randn(n, h, d, generator=g, device=DEV).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    for size in (0.0, min(1.0, 0.02 * cap / scale)):       # all near the middle of the cap, or 0
        qs = (q.float() * size).to(torch.bfloat16)
        out, lse = lib.cp_attn_prefill_mod(qs, _cu([n]), k, v, softcap=cap, softmax_scale=scale, max_seqlen_q=n)
        for i in (0, 1, 270, 500, 639):
            one = torch.tensor([i], device=DEV)
            O, L, A, big = _attend(qs[i:i + 1].double() * (scale * math.sqrt(d)), k.double(), v.double(), 0 * one, one + 1, one, cap, None)
            _check(out[i:i + 1], lse[i:i + 1], O, L, A, big, min(cap, big), None, n, what=f"{size}, row {i}")


@pytest.mark.parametrize("kind", ["bf16", "f32", "q4"])
@pytest.mark.parametrize("cap,scale", [(1e-6, 1e3), (1e-3, 1e4), (1e-6, 1e-11), (1e9, 1e4), (1e9, 1e14), (3.0, 1e6), (0.0, 1e6), (0.0, 1e-20)])
def test_decode_at_the_ends_of_cap_and_scale(lib, kind, cap, scale):
    """As the prefill above, over the caches."""
    n, Hq, Hkv, d, cp, I = 700, 8, 2, 64, 2, 8
    dt, q4 = torch.float32 if kind == "f32" else torch.bfloat16, kind == "q4"
    k, v, t = _pool([n], Hkv, d, cp, I, dt, q4, 3)
    g = torch.Generator(device=DEV).manual_seed(9)
    q, kn, vn = (torch.randn(m, h, d, generator=g, device=DEV).to(dt) for m, h in ((1, Hq), (n, Hkv), (n, Hkv)))
    zero = torch.zeros(1, **I32)
    lib.cp_rope_kv_cache_write(kn, vn, _cu([n]), zero, k, v, t, cp, I)
    K, V = (x.double() for x in lib.cp_kv_cache_read(k, v, _cu([n]), zero, t, cp, I, out_dtype=torch.float32 if q4 else dt))
    one = torch.tensor([n - 1], device=DEV)
    call = lib.cp_decode_attention_q4 if q4 else lib.cp_decode_attention_mod
    for size in (0.0, min(1.0, (0.02 * cap if cap else 0.5) / scale)):
        qs = (q.float() * size).to(dt)
        O, L, A, big = _attend(qs.double() * (scale * math.sqrt(d)), K, V, 0 * one, one + 1, one, cap, None)
        out, lse = call(qs, k, v, t, torch.tensor([n], **I32), cp, I, softcap=cap, softmax_scale=scale)
        _check(out, lse, O, L, A, big, min(cap, big), None, n, f32=kind == "f32", extra=float(V.abs().max()) if q4 else 0.0, what=f"{size}")


# ------------------------------------------------------------------------------ slopes and limits
@pytest.mark.parametrize("Hq,Hkv,d", [(6, 3, 128), (3, 1, 64)])
@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("prefix", [0, 400])
def test_prefill_slopes_of_every_kind(lib, Hq, Hkv, d, cap, prefix):
    """Slopes of 0, gentle, steep, negative (weights that grow with the distance) and past what the exponent takes."""
    n, ctx = 500, 200
    g = torch.Generator(device=DEV).manual_seed(3)
    q = torch.randn(n, Hq, d, generator=g, device=DEV).to(torch.bfloat16)
    k, v = (torch.randn(n + ctx, Hkv, d, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    at = torch.arange(ctx, ctx + n, device=DEV)
    hi = (at + 1).clamp(min=prefix)
    for some in ([0.0, 0.3, 0.9], [1.0, 40.0, -0.01], [-0.2, 300.0, 1e-6]):
        slopes = torch.tensor((some * 2)[:Hq], device=DEV)
        out, lse = lib.cp_attn_prefill_mod(q, _cu([n]), k, v, cu_seqlens_kv=_cu([n + ctx]), softcap=cap, alibi_slopes=slopes, max_seqlen_q=n,
                                           prefix_lens=torch.tensor([prefix], **I32) if prefix else None)
        O, L, A, big = _attend(q.double(), k.double(), v.double(), 0 * at, hi, at, cap, slopes)
        # the bias' own roundings: 2^-22 of the largest one among the keys that count (with a slope below 0, all of
        # them; above 0, those within the scores' spread of the nearest key, which `big` covers)
        far = float((-slopes).clamp(min=0).max()) * (n + ctx)
        beyond = float((slopes * (prefix - ctx)).clamp(min=0).max()) if prefix else 0.0
        _check(out, lse, O, L, A, big + (far + beyond) * 2.0 ** -6, cap, None, n, what=str(some))


@pytest.mark.parametrize("kind", ["bf16", "f32", "q4"])
def test_limits_at_the_ends_of_their_types(lib, kind):
    """Windows, document starts and prefixes of -2^31 and 2^31 - 1: no limit, or no key."""
    n, Hq, Hkv, d, cp, I, top, low = 300, 4, 2, 64, 2, 8, 2 ** 31 - 1, -2 ** 31
    dt, q4 = torch.float32 if kind == "f32" else torch.bfloat16, kind == "q4"
    k, v, t = _pool([n], Hkv, d, cp, I, dt, q4, 3)
    g = torch.Generator(device=DEV).manual_seed(9)
    q, kn, vn = (torch.randn(m, h, d, generator=g, device=DEV).to(dt) for m, h in ((n, Hq), (n, Hkv), (n, Hkv)))
    lib.cp_rope_kv_cache_write(kn, vn, _cu([n]), torch.zeros(1, **I32), k, v, t, cp, I)
    call = lib.cp_decode_attention_q4 if q4 else lib.cp_decode_attention_mod
    sl = torch.tensor([n], **I32)
    full = call(q[:1], k, v, t, sl, cp, I)
    for kw in (dict(window=top), dict(kv_start=torch.tensor([low], **I32)), dict(window=top, kv_start=torch.tensor([-1], **I32))):
        got = call(q[:1], k, v, t, sl, cp, I, **kw)
        assert all(torch.equal(a, b) for a, b in zip(got, full))
    for lens, kw in ((sl, dict(kv_start=torch.tensor([top], **I32))), (torch.tensor([low], **I32), dict(max_seq_len=n)),
                     (torch.tensor([low], **I32), dict(max_seq_len=n, window=5, kv_start=torch.tensor([top], **I32)))):
        out, lse = call(q[:1], k, v, t, lens, cp, I, **kw)
        assert not out.any() and bool(torch.isneginf(lse).all())
    if kind != "bf16":
        return
    cu, full = _cu([n]), lib.cp_attn_prefill_mod(q, _cu([n]), kn, vn)
    whole = lib.cp_attn_prefill_mod(q, cu, kn, vn, prefix_lens=torch.tensor([n], **I32))
    at = lambda x: torch.full((n,), x, **I32)
    for want, kw in ((full, dict(window=top)), (full, dict(kv_start=at(low))), (full, dict(prefix_lens=torch.tensor([low], **I32))),
                     (whole, dict(prefix_lens=torch.tensor([top], **I32))), (whole, dict(prefix_lens=torch.tensor([top], **I32), kv_start=at(-7), window=top))):
        got = lib.cp_attn_prefill_mod(q, cu, kn, vn, **kw)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), kw
    out, lse = lib.cp_attn_prefill_mod(q, cu, kn, vn, kv_start=at(top), softcap=5.0)
    assert not out.any() and bool(torch.isneginf(lse).all())
