"""Cases, plain forms and reference results of the serving operators around the paged round-robin
K/V cache: rotate-and-append, read-back, decode over a 4-bit cache, and attention whose scores are
capped, biased by distance or masked by document, window and prefix (prefill and decode).

Every attention score is
    s = scale q.k;  s = cap tanh(s / cap) if cap;  s -= slope[h] |i - j| if slopes
over the keys j in [lo_i, hi_i): lo_i = max(0, i - window + 1, kv_start_i), hi_i = i + 1, or the
sequence's prefix length where that is larger.  A row without a key gives 0 and LSE -inf.

4-bit cache: one kv head's 16 tokens are a record of 9 d bytes: 16 rows of d / 2 bytes, then for each
token and group of 64 dims the bf16 pair (scale, minimum).  value = minimum + scale * n, n in 0..15.
The 32-bit word w of a row holds 8 consecutive dims (lowest nibble first) from 8 w (d = 64) or
64 (w % 2) + 8 (w // 2) (d = 128).

Position p of a sequence lives on rank (p // I) % cp at local index (p // (I cp)) I + p % I, in the
rank's page pool through its block table, 16 tokens a page.
"""
import math
import random

import torch

own = False

PAGE = 16
BASE = 10000.0  # base of the rotation's frequencies


# ------------------------------------------------------------------------------------ the cases

def listed():
    return [
        # one decode step's append: 64 sequences, one token each, deep in their contexts
        dict(name="write_step", op="write", B=64, new_lo=1, new_hi=1, ctx_lo=1023, ctx_hi=32767, Hq=32, Hkv=8,
             d=128, dtype="bf16", cache="same", rot=128, style="half", cp=2, I=8, lens=11),
        # a long prompt's append: 2 x 32768 tokens into empty caches
        dict(name="write_long", op="write", B=2, new_lo=32768, new_hi=32768, ctx_lo=0, ctx_hi=0, Hq=16, Hkv=2,
             d=128, dtype="bf16", cache="same", rot=128, style="half", cp=4, I=8, lens=12),
        # a chunk of four prompts into a 4-bit cache, read back as the rows that a prefill attends
        dict(name="write_q4_chunk", op="write", B=4, new_lo=2048, new_hi=2048, ctx_lo=30720, ctx_hi=30720, Hq=16,
             Hkv=2, d=128, dtype="bf16", cache="q4", rot=128, style="half", cp=4, I=8, lens=13),
        # the cached context of a chunked prefill (4 x 30720 tokens), back to contiguous rows
        dict(name="read_chunked", op="read", B=4, lo=30720, hi=30720, Hkv=2, d=128, dtype="bf16", cache="same",
             cp=4, I=8, lens=14),
        # ragged short contexts of a 4-bit cache
        dict(name="read_q4_ragged", op="read", B=7, lo=1, hi=2500, Hkv=8, d=128, dtype="bf16", cache="q4", cp=2,
             I=8, lens=15),
        # one user's decode step over a 4-bit cache: latency
        dict(name="decode_q4_one", op="decode", B=1, lo=1777, hi=1777, Hq=16, Hkv=2, d=128, dtype="bf16",
             cache="q4", cap=0.0, window=0, alibi=False, docs=False, cp=2, I=8, lens=16),
        # a full decode batch over a 4-bit cache
        dict(name="decode_q4_batch", op="decode", B=64, lo=1024, hi=32768, Hq=32, Hkv=8, d=128, dtype="bf16",
             cache="q4", cap=0.0, window=0, alibi=False, docs=False, cp=2, I=8, lens=17),
        # a prompt of a model with capped scores
        dict(name="prefill_cap", op="prefill", B=1, lo=8192, hi=8192, ctx_lo=0, ctx_hi=0, Hq=16, Hkv=2, d=128,
             cap=50.0, window=0, alibi=False, doc=0, prefix=0, lens=18),
        # a long prompt through a sliding-window layer with capped scores
        dict(name="prefill_window", op="prefill", B=1, lo=16384, hi=16384, ctx_lo=0, ctx_hi=0, Hq=16, Hkv=2,
             d=128, cap=30.0, window=4096, alibi=False, doc=0, prefix=0, lens=19),
        # ragged prompts with a distance bias, packed documents and a bidirectional prefix, some with a context
        dict(name="prefill_docs", op="prefill", B=5, lo=1, hi=3001, ctx_lo=0, ctx_hi=700, Hq=24, Hkv=8, d=64,
             cap=0.0, window=0, alibi=True, doc=400, prefix=96, lens=20),
        # a full decode batch with capped scores
        dict(name="decode_cap", op="decode", B=64, lo=1024, hi=32768, Hq=32, Hkv=8, d=128, dtype="bf16",
             cache="same", cap=50.0, window=0, alibi=False, docs=False, cp=2, I=8, lens=21),
        # a small fp32 batch with a distance bias and a window
        dict(name="decode_alibi", op="decode", B=8, lo=300, hi=5000, Hq=8, Hkv=2, d=64, dtype="f32", cache="same",
             cap=0.0, window=1500, alibi=True, docs=True, cp=4, I=8, lens=22),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "decode", "decode", "prefill", "prefill"])
    d, Hkv = rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 6, 8])
    c = dict(op=op, Hkv=Hkv, d=d, lens=rng.randrange(1 << 20))
    if op != "prefill":
        c.update(cp=rng.choice([1, 2, 4, 8]), I=rng.choice([1, 5, 8, 16]))
    if op == "write":
        tokens, B = _log(rng, 1, 65536), _log(rng, 1, 64)
        hi = max(1, tokens // B)
        c.update(B=B, new_lo=max(1, hi // 2), new_hi=hi, ctx_lo=0, ctx_hi=_log(rng, 1, 32768 // B), Hq=G * Hkv,
                 dtype=rng.choice(["bf16", "bf16", "f32"]), cache=rng.choice(["same", "q4"]),
                 rot=rng.choice([d, d, d // 2]), style=rng.choice(["half", "pairs"]))
        if B * hi * Hkv * (G + 4) > 65536 * 20:
            c.update(Hkv=2, Hq=2 * G)
    elif op == "read":
        B, hi = _log(rng, 1, 32), _log(rng, 1, 32768)
        hi = max(1, min(hi, 122880 // B))
        q4 = rng.random() < 0.5
        c.update(B=B, lo=max(1, hi // 4), hi=hi, dtype="bf16" if q4 else rng.choice(["bf16", "f32"]),
                 cache="q4" if q4 else "same")
        if B * hi * Hkv * d * (1 if c["dtype"] == "bf16" else 2) > 122880 * 256:
            c.update(Hkv=1, d=64)
    elif op == "decode":
        B, hi = _log(rng, 1, 64), _log(rng, 1, 32768)
        dtype, cache = rng.choice([("bf16", "q4"), ("bf16", "q4"), ("bf16", "same"), ("f32", "same")])
        c.update(B=B, lo=max(1, hi // 32), hi=hi, Hq=G * Hkv, dtype=dtype, cache=cache,
                 cap=rng.choice([0.0, 30.0, 50.0]), window=rng.choice([0, 0, _log(rng, 1, 8192)]),
                 alibi=rng.random() < 0.3, docs=rng.random() < 0.3)
        if dtype == "f32":
            c.update(hi=min(hi, 16384), lo=min(c["lo"], 512))
    else:
        B, hi = _log(rng, 1, 8), _log(rng, 1, 8192)
        hi = max(1, min(hi, int(16384 * math.sqrt(16.0 / (B * G * Hkv)) * 0.7) - 1000))
        c.update(B=B, lo=max(1, hi // 8), hi=hi, ctx_lo=0, ctx_hi=rng.choice([0, 0, _log(rng, 1, 1000)]),
                 Hq=G * Hkv, cap=rng.choice([0.0, 30.0, 50.0]), window=rng.choice([0, 0, _log(rng, 1, 4096)]),
                 alibi=rng.random() < 0.4, doc=rng.choice([0, 0, _log(rng, 8, 2000)]),
                 prefix=rng.choice([0, 0, _log(rng, 1, 512)]))
    return c


def _lens(case, lo, hi, salt):
    r = random.Random(case["lens"] * 7 + salt)
    return [r.randint(lo, hi) for _ in range(case["B"])]


def _decode_spans(case):
    """(length, first visible position) of each sequence of a decode case."""
    L = _lens(case, case["lo"], case["hi"], 0)
    r = random.Random(case["lens"] * 7 + 3)
    doc = [r.randint(0, n - 1) if case["docs"] else 0 for n in L]
    return L, doc, [max(s, n - case["window"] if case["window"] else 0) for n, s in zip(L, doc)]


def _prefill_spans(case):
    """Per sequence: new tokens, context, prefix length, document starts of the new tokens."""
    T = _lens(case, case["lo"], case["hi"], 0)
    C = _lens(case, case["ctx_lo"], case["ctx_hi"], 1)
    r = random.Random(case["lens"] * 7 + 2)
    pre = [min(r.randint(0, case["prefix"]), t + c) if case["prefix"] else 0 for t, c in zip(T, C)]
    starts = []
    for t, c in zip(T, C):
        row, at = [], 0
        for i in range(t):
            if case["doc"] and r.random() < 1.0 / case["doc"]:
                at = c + i
            # now and then a placeholder that belongs to no document: its row sees nothing
            row.append(c + t if case["doc"] and r.random() < 0.002 else at)
        starts.append(row)
    return T, C, pre, starts


# ------------------------------------------------------------------------------------ the inputs

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _dev():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _gen(seed):
    return torch.Generator(device=_dev()).manual_seed(seed)


def _randn(shape, g, dtype):
    return torch.randn(*shape, generator=g, device=_dev(), dtype=torch.float32).to(dtype)


def _cu(lens):
    return torch.tensor([0] + list(lens), device=_dev()).cumsum(0).to(torch.int32)


def _tables(case, lens, seed):
    """Block tables [cp, B, max_blocks] of a shuffled pool on each rank, and the pool's pages."""
    cp, I = case["cp"], case["I"]
    need = [-(-(-(-n // (I * cp)) * I) // PAGE) for n in lens]
    pool, wide = max(1, sum(need)), max(1, max(need))
    at = torch.tensor([0] + need[:-1]).cumsum(0)
    col = torch.arange(wide)
    flat = at[:, None] + col
    g = torch.Generator().manual_seed(seed)
    perm = torch.stack([torch.randperm(pool, generator=g) for _ in range(cp)])
    t = perm[:, flat.clamp(max=pool - 1)]
    t = torch.where(col < torch.tensor(need)[:, None], t, torch.tensor(-1))
    return t.to(torch.int32).to(_dev()), pool


def _quantised_pool(n_pages, d, g):
    """Random 4-bit records [n_pages, 9 d] of N(0, 1) rows."""
    rows = torch.randn(n_pages * PAGE, d // 64, 64, generator=g, device=_dev())
    n, sc, mn = _quantise(rows)
    return _records(n.view(n_pages, PAGE, d // 64, 64), sc.view(n_pages, PAGE, -1), mn.view(n_pages, PAGE, -1))


def _pools(case, pool, g):
    shape = (case["cp"], pool, case["Hkv"])
    if case["cache"] == "q4":
        n = shape[0] * shape[1] * shape[2]
        part = 1 << 17  # pages quantised at a time
        return [torch.cat([_quantised_pool(min(part, n - i), case["d"], g) for i in range(0, n, part)])
                .view(*shape, 9 * case["d"]) for _ in range(2)]
    return [_randn(shape + (PAGE, case["d"]), g, DT[case["dtype"]]) for _ in range(2)]


def _slopes(Hq):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], device=_dev(), dtype=torch.float32)


def prepare(case, seed):
    g, dev = _gen(seed), _dev()
    s = dict(case=case)
    if case["op"] == "prefill":
        T, C, pre, starts = _prefill_spans(case)
        N, Nk = sum(T), sum(T) + sum(C)
        s.update(q=_randn((N, case["Hq"], case["d"]), g, torch.bfloat16),
                 k=_randn((Nk, case["Hkv"], case["d"]), g, torch.bfloat16),
                 v=_randn((Nk, case["Hkv"], case["d"]), g, torch.bfloat16), cu_q=_cu(T),
                 cu_kv=_cu([a + b for a, b in zip(T, C)]), max_q=max(T), max_kv=max(a + b for a, b in zip(T, C)),
                 slopes=_slopes(case["Hq"]) if case["alibi"] else None,
                 kv_start=torch.tensor(sum(starts, []), dtype=torch.int32, device=dev) if case["doc"] else None,
                 prefix=torch.tensor(pre, dtype=torch.int32, device=dev) if case["prefix"] else None)
        return s
    if case["op"] == "decode":
        L, doc, _ = _decode_spans(case)
        tables, pool = _tables(case, L, seed)
        kc, vc = _pools(case, pool, g)
        s.update(q=_randn((case["B"], case["Hq"], case["d"]), g, DT[case["dtype"]]), k_cache=kc, v_cache=vc,
                 tables=tables, seq_lens=torch.tensor(L, dtype=torch.int32, device=dev), max_len=max(L),
                 slopes=_slopes(case["Hq"]) if case["alibi"] else None,
                 kv_start=torch.tensor(doc, dtype=torch.int32, device=dev) if case["docs"] else None)
        return s
    if case["op"] == "read":
        L = _lens(case, case["lo"], case["hi"], 0)
        tables, pool = _tables(case, L, seed)
        kc, vc = _pools(case, pool, g)
        s.update(k_cache=kc, v_cache=vc, tables=tables, cu=_cu(L), total=sum(L),
                 start=torch.zeros(case["B"], dtype=torch.int32, device=dev))
        return s
    new = _lens(case, case["new_lo"], case["new_hi"], 0)
    ctx = _lens(case, case["ctx_lo"], case["ctx_hi"], 1)
    tables, pool = _tables(case, [a + b for a, b in zip(new, ctx)], seed)
    N, dt = sum(new), DT[case["dtype"]]
    # a fused projection's output: q, k and v are its columns
    qkv = _randn((N, case["Hq"] + 2 * case["Hkv"], case["d"]), g, dt)
    q, k, v = qkv.split([case["Hq"], case["Hkv"], case["Hkv"]], 1)
    shape = (case["cp"], pool, case["Hkv"])
    if case["cache"] == "q4":
        kc, vc = (torch.zeros(shape + (9 * case["d"],), dtype=torch.uint8, device=dev) for _ in range(2))
    else:
        kc, vc = (torch.zeros(shape + (PAGE, case["d"]), dtype=dt, device=dev) for _ in range(2))
    half = case["rot"] // 2
    freq = BASE ** (-torch.arange(half, dtype=torch.float64) / half)
    s.update(q=q, k=k, v=v, k_cache=kc, v_cache=vc, tables=tables, cu=_cu(new), total=N, inv_freq=freq.to(dev),
             start=torch.tensor(ctx, dtype=torch.int32, device=dev))
    return s


# ------------------------------------------------------------------------------------ plain forms

def _quantise(x):
    """Groups of 64 (last axis), fp32: codes 0..15 and the bf16 scale and minimum of each group."""
    mn = x.amin(-1, keepdim=True).to(torch.bfloat16).float()
    sc = ((x.amax(-1, keepdim=True) - mn) / 15).to(torch.bfloat16).float()
    n = torch.where(sc > 0, ((x - mn) / torch.where(sc > 0, sc, 1)).round().clamp(0, 15), 0.0)
    return n.to(torch.int32), sc.squeeze(-1), mn.squeeze(-1)


def _row_bytes(n):
    """Codes [..., groups, 64] -> the row's bytes [..., d / 2]: words of 8 codes, the groups' words in turn."""
    w = n.unflatten(-1, (8, 8)).transpose(-2, -3).flatten(-3)
    return (w[..., 0::2] | (w[..., 1::2] << 4)).to(torch.uint8)


def _scale_bytes(sc, mn):
    return torch.stack([sc, mn], -1).to(torch.bfloat16).contiguous().view(torch.uint8).flatten(-2)


def _records(n, sc, mn):
    return torch.cat([_row_bytes(n).flatten(-2), _scale_bytes(sc, mn).flatten(-2)], -1)


def _values(rows, scales):
    """Row bytes [..., d / 2] and scale bytes [..., d / 16] -> the values they stand for, fp32 [..., d]."""
    groups = rows.shape[-1] // 32
    n = torch.stack([rows & 15, rows >> 4], -1).flatten(-2)
    n = n.unflatten(-1, (8, groups, 8)).transpose(-2, -3).flatten(-2).float()
    p = scales.contiguous().view(torch.bfloat16).float().unflatten(-1, (groups, 2))
    return (p[..., 1:] + p[..., :1] * n).flatten(-2)


def _slots(s, seq, pos):
    """(rank, page, row within the page) of positions of sequences."""
    cp, I = s["case"]["cp"], s["case"]["I"]
    r = (pos // I) % cp
    local = (pos // (I * cp)) * I + pos % I
    page = s["tables"][r, seq, (local // PAGE).clamp(max=s["tables"].shape[-1] - 1)].long()
    return r, page.clamp(min=0), local % PAGE


def _rows_of(cu, total):
    """(sequence, index within it) of each token-major row."""
    row = torch.arange(total, device=cu.device)
    seq = torch.searchsorted(cu[1:].long(), row, right=True)
    return seq, row - cu.long()[seq]


def _fetch(s, cache, r, page, slot):
    """Rows of the cache as fp32 [..., Hkv, d]."""
    if s["case"]["cache"] != "q4":
        return cache[r, page, :, slot].float()
    d = s["case"]["d"]
    body = cache[..., :8 * d].unflatten(-1, (PAGE, d // 2))
    tail = cache[..., 8 * d:].unflatten(-1, (PAGE, d // 16))
    return _values(body[r, page, :, slot], tail[r, page, :, slot])


def _rotate(x, angle, style):
    """x [N, H, d] fp32 rotated in its first 2 * angle.shape[-1] dims by the angles [N, rot / 2]."""
    h = angle.shape[-1]
    c, n = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if style == "half":
        a, b = x[..., :h], x[..., h:2 * h]
        return torch.cat([a * c - b * n, b * c + a * n, x[..., 2 * h:]], -1)
    a, b = x[..., 0:2 * h:2], x[..., 1:2 * h:2]
    return torch.cat([torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2), x[..., 2 * h:]], -1)


def _write(s):
    case, dt = s["case"], DT[s["case"]["dtype"]]
    seq, off = _rows_of(s["cu"], s["total"])
    pos = s["start"].long()[seq] + off
    angle = pos.double()[:, None] * s["inv_freq"]
    q, k = (_rotate(s[x].float(), angle, case["style"]) for x in ("q", "k"))
    v = s["v"].float()
    r, page, slot = _slots(s, seq, pos)
    if case["cache"] != "q4":
        s["k_cache"][r, page, :, slot] = k.to(dt)
        s["v_cache"][r, page, :, slot] = v.to(dt)
        return q.to(dt), s["k_cache"], s["v_cache"]
    d = case["d"]
    ca, cb, va, vb = _quant_write(s, "k_cache", k, r, page, slot) + _quant_write(s, "v_cache", v, r, page, slot)
    return q.to(dt), _values(ca[r, page, :, slot], cb[r, page, :, slot]).to(dt), \
        _values(va[r, page, :, slot], vb[r, page, :, slot]).to(dt)


def _quant_write(s, name, x, r, page, slot):
    """Quantises rows [N, Hkv, d] into the cache; its row and scale bytes as views."""
    d = s["case"]["d"]
    body = s[name][..., :8 * d].unflatten(-1, (PAGE, d // 2))
    tail = s[name][..., 8 * d:].unflatten(-1, (PAGE, d // 16))
    n, sc, mn = _quantise(x.unflatten(-1, (-1, 64)))
    body[r, page, :, slot] = _row_bytes(n)
    tail[r, page, :, slot] = _scale_bytes(sc, mn)
    return body, tail


def _read(s):
    seq, off = _rows_of(s["cu"], s["total"])
    r, page, slot = _slots(s, seq, s["start"].long()[seq] + off)
    dt = DT[s["case"]["dtype"]]
    return _fetch(s, s["k_cache"], r, page, slot).to(dt), _fetch(s, s["v_cache"], r, page, slot).to(dt)


def _attend(score, v, cap, bias, mask):
    """Softmax of the scores [..., i, j] (fp32, overwritten) over the keys of `mask`, times v."""
    if cap:
        score = score.div_(cap).tanh_().mul_(cap)
    if bias is not None:
        score -= bias
    score.masked_fill_(~mask, -math.inf)
    m = score.amax(-1, keepdim=True)
    score -= torch.where(m > -math.inf, m, 0.0)
    p = score.exp_()
    total = p.sum(-1, keepdim=True)
    o = p @ v / torch.where(total > 0, total, 1)
    return o, (m + total.log()).squeeze(-1)


def _decode(s):
    case = s["case"]
    B, d, dev = case["B"], case["d"], s["q"].device
    L = s["seq_lens"].long()[:, None]
    pos = torch.arange(s["max_len"], device=dev)[None].expand(B, -1)
    r, page, slot = _slots(s, torch.arange(B, device=dev)[:, None].expand_as(pos), pos)
    k = _fetch(s, s["k_cache"], r, page, slot).permute(0, 2, 3, 1)
    q = s["q"].float().view(B, case["Hkv"], -1, d)
    score = q @ k / math.sqrt(d)
    lo = torch.zeros_like(L)
    if case["window"]:
        lo = torch.maximum(lo, L - case["window"])
    if s["kv_start"] is not None:
        lo = torch.maximum(lo, s["kv_start"].long()[:, None])
    mask = ((pos >= lo) & (pos < L))[:, None, None]
    bias = None
    if s["slopes"] is not None:
        bias = s["slopes"].view(1, case["Hkv"], -1, 1) * (L - 1 - pos).abs().float()[:, None, None]
    v = _fetch(s, s["v_cache"], r, page, slot).permute(0, 2, 1, 3)
    # rows behind a sequence's end are not its values: whatever lies there is left out
    v = v.masked_fill(~((pos >= lo) & (pos < L))[:, None, :, None], 0.0)
    o, lse = _attend(score, v, case["cap"], bias, mask)
    return o.reshape(B, -1, d).to(s["q"].dtype), lse.reshape(B, -1)


def _prefill(s):
    case, dev = s["case"], s["q"].device
    B, d, Hkv = case["B"], case["d"], case["Hkv"]
    cu_q, cu_kv = s["cu_q"].long(), s["cu_kv"].long()
    T, K = (cu_q[1:] - cu_q[:-1])[:, None], (cu_kv[1:] - cu_kv[:-1])[:, None]
    i, j = torch.arange(s["max_q"], device=dev)[None], torch.arange(s["max_kv"], device=dev)[None]
    rows = torch.minimum(cu_q[:-1, None] + i, cu_q[-1:] - 1)
    keys = torch.minimum(cu_kv[:-1, None] + j, cu_kv[-1:] - 1)
    q = s["q"][rows].float().view(B, s["max_q"], Hkv, -1, d).permute(0, 2, 3, 1, 4)
    k = s["k"][keys].float().permute(0, 2, 3, 1)[:, :, None]
    v = s["v"][keys].float().permute(0, 2, 1, 3)[:, :, None]
    at = K - T + i  # position of each query
    lo, hi = torch.zeros_like(at), at + 1
    if case["window"]:
        lo = torch.maximum(lo, at - case["window"] + 1)
    if s["kv_start"] is not None:
        lo = torch.maximum(lo, s["kv_start"].long()[rows])
    if s["prefix"] is not None:
        hi = torch.maximum(hi, s["prefix"].long()[:, None])
    hi = torch.minimum(hi, K)
    j = j[:, None]
    mask = ((j >= lo[..., None]) & (j < hi[..., None]))[:, None, None]
    bias = None
    if s["slopes"] is not None:
        bias = s["slopes"].view(1, Hkv, -1, 1, 1) * (at[..., None] - j).abs().float()[:, None, None]
    score = q @ k
    score *= 1.0 / math.sqrt(d)
    o, lse = _attend(score, v, case["cap"], bias, mask)
    b, t = _rows_of(s["cu_q"], s["q"].shape[0])
    o = o.permute(0, 3, 1, 2, 4)[b, t].reshape(-1, case["Hq"], d)
    return o.to(torch.bfloat16), lse.permute(0, 3, 1, 2)[b, t].reshape(-1, case["Hq"])


# ------------------------------------------------------------------------------------ the framework's calls

def _own_write(s):
    import context_gqa_attention_gb300 as cpa
    case = s["case"]
    style = cpa.CP_ROPE_HALF if case["style"] == "half" else cpa.CP_ROPE_PAIRS
    q, _ = cpa.cp_rope_kv_cache_write(s["k"], s["v"], s["cu"], s["start"], s["k_cache"], s["v_cache"], s["tables"],
                                      case["cp"], case["I"], inv_freq=s["inv_freq"], rope_style=style, q=s["q"])
    if case["cache"] != "q4":
        return q, s["k_cache"], s["v_cache"]
    k, v = cpa.cp_kv_cache_read(s["k_cache"], s["v_cache"], s["cu"], s["start"], s["tables"], case["cp"],
                                case["I"], total=s["total"], out_dtype=DT[case["dtype"]])
    return q, k, v


def _own_read(s):
    import context_gqa_attention_gb300 as cpa
    case = s["case"]
    return cpa.cp_kv_cache_read(s["k_cache"], s["v_cache"], s["cu"], s["start"], s["tables"], case["cp"], case["I"],
                                total=s["total"], out_dtype=DT[case["dtype"]])


def _own_decode(s):
    import context_gqa_attention_gb300 as cpa
    case = s["case"]
    if "plan" not in s:  # a program keeps its split plan and its zero-filled workspace
        plan = cpa.cp_decode_mod_plan(case["B"], case["Hkv"], case["cp"], case["I"], s["max_len"],
                                      window=case["window"], q4=case["cache"] == "q4")
        size = cpa.cp_decode_workspace_size(case["B"], case["Hq"], case["Hkv"], case["d"], case["cp"], plan[0])
        s["plan"] = plan + (torch.zeros(size, dtype=torch.uint8, device=s["q"].device),)
    splits, tokens, workspace = s["plan"]
    call = cpa.cp_decode_attention_q4 if case["cache"] == "q4" else cpa.cp_decode_attention_mod
    return call(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["seq_lens"], case["cp"], case["I"],
                softcap=case["cap"], window=case["window"], alibi_slopes=s["slopes"], kv_start=s["kv_start"],
                num_splits=splits, split_tokens=tokens, workspace=workspace)


def _own_prefill(s):
    import context_gqa_attention_gb300 as cpa
    case = s["case"]
    return cpa.cp_attn_prefill_mod(s["q"], s["cu_q"], s["k"], s["v"], cu_seqlens_kv=s["cu_kv"],
                                   max_seqlen_q=s["max_q"], softcap=case["cap"], window=case["window"],
                                   alibi_slopes=s["slopes"], kv_start=s["kv_start"], prefix_lens=s["prefix"])


def run(state):
    op = state["case"]["op"]
    if own:
        return {"write": _own_write, "read": _own_read, "decode": _own_decode, "prefill": _own_prefill}[op](state)
    return {"write": _write, "read": _read, "decode": _decode, "prefill": _prefill}[op](state)


# ------------------------------------------------------------------------------------ work

def _row_cost(case):
    """Bytes of one cached token and kv head, of K or of V."""
    return case["d"] * 9 / 16 if case["cache"] == "q4" else case["d"] * (2 if case["dtype"] == "bf16" else 4)


def work(case):
    d, Hkv = case["d"], case["Hkv"]
    if case["op"] == "prefill":
        T, C, pre, starts = _prefill_spans(case)
        N, Nk = sum(T), sum(T) + sum(C)
        pairs = 0
        for t, c, p, st in zip(T, C, pre, starts):
            for i in range(t):
                lo = max(0, c + i - case["window"] + 1 if case["window"] else 0, st[i])
                pairs += max(0, min(max(c + i + 1, p), c + t) - lo)
        return {"bytes": 2 * d * (2 * N * case["Hq"] + 2 * Nk * Hkv) + 4 * N * case["Hq"],
                "flops": 4 * d * case["Hq"] * pairs}
    if case["op"] == "decode":
        L, _, lo = _decode_spans(case)
        keys = sum(max(0, n - a) for n, a in zip(L, lo))
        e = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * keys * Hkv * _row_cost(case) + case["B"] * case["Hq"] * (2 * e * d + 4),
                "flops": 4 * d * case["Hq"] * keys}
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "read":
        return {"bytes": 2 * sum(_lens(case, case["lo"], case["hi"], 0)) * Hkv * (_row_cost(case) + e * d), "flops": 0}
    N = sum(_lens(case, case["new_lo"], case["new_hi"], 0))
    back = 2 * Hkv * e * d if case["cache"] == "q4" else 0
    return {"bytes": N * (2 * case["Hq"] * e * d + 2 * Hkv * (e * d + _row_cost(case)) + back),
            "flops": 6 * N * (case["Hq"] + Hkv) * case["rot"] / 2}


# ------------------------------------------------------------------------------------ 64 bits

def _exact_slot(case, tables, b, p):
    """Rank, page and row of positions p (int64) of sequence b."""
    turn, within = p // (case["I"] * case["cp"]), p % (case["I"] * case["cp"])
    rank = within // case["I"]
    local = turn * case["I"] + within - rank * case["I"]
    return rank, tables[rank, b, local // PAGE].long(), local % PAGE


def _exact_codes(row, d):
    """Row bytes [..., d / 2] -> codes [..., d] by each dim's own place."""
    dim = torch.arange(d, device=row.device)
    word = dim // 8 if d == 64 else 2 * ((dim % 64) // 8) + dim // 64
    nib = word * 8 + dim % 8
    return (row.long()[..., nib // 2] >> (4 * (nib % 2))) & 15


def _exact_rows(case, cache, rank, page, slot):
    if case["cache"] != "q4":
        return cache[rank, page, :, slot].double()
    d = case["d"]
    rec = cache[rank, page]  # [n, Hkv, 9 d]
    take = lambda at, width: torch.gather(  # noqa: E731
        rec, -1, (at[:, None] + torch.arange(width, device=at.device))[:, None].expand(-1, rec.shape[1], -1))
    n = _exact_codes(take(slot * (d // 2), d // 2), d).double()
    pair = take(8 * d + slot * (d // 16), d // 16).contiguous().view(torch.bfloat16).double()
    sc, mn = pair[..., 0::2].repeat_interleave(64, -1), pair[..., 1::2].repeat_interleave(64, -1)
    return mn + sc * n


def _exact_attend(q, k, v, scale, cap, slopes, at, lo, hi):
    """q [i, Hq, d], k / v [j, Hkv, d] in 64 bits; at / lo / hi per query row."""
    G = q.shape[1] // k.shape[1]
    out, lse = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=q.dtype, device=q.device)
    j = torch.arange(k.shape[0], device=q.device)
    for i0 in range(0, q.shape[0], 2048):
        i1 = min(q.shape[0], i0 + 2048)
        a, b = int(lo[i0:i1].min()), int(hi[i0:i1].max())
        if b <= a:
            continue
        seen = (j[a:b] >= lo[i0:i1, None]) & (j[a:b] < hi[i0:i1, None])
        for h in range(q.shape[1]):
            x = (q[i0:i1, h] * scale) @ k[a:b, h // G].T
            if cap:
                x = cap * torch.tanh(x / cap)
            if slopes is not None:
                x = x - slopes[h].double() * (at[i0:i1, None] - j[a:b]).abs().double()
            x = x.masked_fill(~seen, -math.inf)
            z = torch.logsumexp(x, -1)
            lse[i0:i1, h] = z
            w = torch.exp(x - z.clamp(min=-1e300)[:, None])
            out[i0:i1, h] = w @ v[a:b, h // G]
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    dev = _dev()
    if case["op"] == "prefill":
        T, C, pre, starts = _prefill_spans(case)
        outs, lses, r0, k0 = [], [], 0, 0
        for t, c, p, st in zip(T, C, pre, starts):
            at = torch.arange(c, c + t, device=dev)
            lo = torch.tensor(st, device=dev).clamp(min=0)
            if case["window"]:
                lo = torch.maximum(lo, at + 1 - case["window"])
            hi = (at + 1).clamp(min=p)
            x = _exact_attend(s["q"][r0:r0 + t].double(), s["k"][k0:k0 + c + t].double(), s["v"][k0:k0 + c + t].double(),
                              1 / math.sqrt(case["d"]), case["cap"], s["slopes"], at, lo, hi)
            outs.append(x[0])
            lses.append(x[1])
            r0, k0 = r0 + t, k0 + c + t
        return torch.cat(outs), torch.cat(lses)
    if case["op"] == "decode":
        L, _, lo = _decode_spans(case)
        outs, lses = [], []
        for b, (n, a) in enumerate(zip(L, lo)):
            where = _exact_slot(case, s["tables"], b, torch.arange(a, n, device=dev))
            k, v = (_exact_rows(case, s[x], *where) for x in ("k_cache", "v_cache"))
            one = torch.tensor([n - 1 - a], device=dev)
            x = _exact_attend(s["q"][b:b + 1].double(), k, v, 1 / math.sqrt(case["d"]), case["cap"], s["slopes"],
                              one, torch.zeros_like(one), torch.full_like(one, n - a))
            outs.append(x[0])
            lses.append(x[1])
        return torch.cat(outs), torch.cat(lses)
    if case["op"] == "read":
        L = _lens(case, case["lo"], case["hi"], 0)
        rows = [[_exact_rows(case, s[x], *_exact_slot(case, s["tables"], b, torch.arange(n, device=dev)))
                 for b, n in enumerate(L)] for x in ("k_cache", "v_cache")]
        return torch.cat(rows[0]), torch.cat(rows[1])
    new = _lens(case, case["new_lo"], case["new_hi"], 0)
    ctx = _lens(case, case["ctx_lo"], case["ctx_hi"], 1)
    half = case["rot"] // 2
    first = torch.arange(half, device=dev) * (1 if case["style"] == "half" else 2)
    second = first + (half if case["style"] == "half" else 1)
    turn = torch.exp(torch.arange(half, device=dev, dtype=torch.float64) * (-math.log(BASE) / half))
    q, k, v, r0 = s["q"].double(), s["k"].double(), s["v"].double(), 0
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    back_k, back_v = [], []
    for b, (n, c) in enumerate(zip(new, ctx)):
        p = torch.arange(c, c + n, device=dev)
        z = torch.polar(torch.ones(n, half, dtype=torch.float64, device=dev), p[:, None] * turn)[:, None]
        for x in (q, k):
            y = torch.complex(x[r0:r0 + n, :, first], x[r0:r0 + n, :, second]) * z
            x[r0:r0 + n, :, first], x[r0:r0 + n, :, second] = y.real, y.imag
        rank, page, slot = _exact_slot(case, s["tables"], b, p)
        if case["cache"] == "q4":
            back_k.append(_exact_round_trip(k[r0:r0 + n]))
            back_v.append(_exact_round_trip(v[r0:r0 + n]))
        else:
            kc[rank, page, :, slot] = k[r0:r0 + n]
            vc[rank, page, :, slot] = v[r0:r0 + n]
        r0 += n
    if case["cache"] == "q4":
        return q, torch.cat(back_k), torch.cat(back_v)
    return q, kc, vc


def _exact_round_trip(x):
    """What the 4-bit cache holds of rows x [n, Hkv, d] in 64 bits."""
    y = x.unflatten(-1, (-1, 64))
    low = y.min(-1, keepdim=True).values.to(torch.bfloat16).double()
    step = ((y.max(-1, keepdim=True).values - low) / 15).to(torch.bfloat16).double()
    n = torch.round((y - low) / step.clamp(min=1e-300)).clamp(0, 15)
    return (low + step * torch.where(step > 0, n, 0.0)).flatten(-2)
