"""Cases, plain forms and reference results of beam search over an encoder's states: cross attention
to states of another length, the selection of the best continuations over beams and vocabulary, and
the reordering of the beams' paged key-value caches.

Cross attention: query row i of sequence b sees the keys j of the sequence's encoder states in
[lo_i, hi_i): all of them, or the first kv_lens[b] (a padded batch), or those within the row's own range
too (the image that a text token belongs to).  A row without a key gives 0 and LSE -inf.

Selection: continuation (k, v) of a sequence has the score scores[k] + log softmax(logits[k])[v]; the
M best are returned in falling order, ties to the lowest k V + v (a NaN logit counts as -inf), and the
first K of them that do not end the sequence go on as its beams.

Reordering: beam j goes on from parent p.  Of the L cached tokens of a sequence, rank r holds L_r (position
p lies on rank (p // I) % cp at local index (p // (I cp)) I + p % I), 16 to a page.  Pages that are full are
shared: column c < L_r // 16 of beam j's table takes the parent's entry.  The page being filled, column
L_r // 16, becomes beam j's own page of that column, and the L_r % 16 tokens in it are copied there.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 16
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------ the cases

def listed():
    return [
        # one decode step of one user: 4 beams over an encoder's 1500 states, as many kv heads as query heads
        dict(name="cross_step_one", op="cross", B=1, q_lo=4, q_hi=4, kv_lo=1500, kv_hi=1500, Hq=16, Hkv=16, d=64,
             dtype="bf16", pad=False, packed=True, image=0, lens=31),
        # a full decode batch, 4 beams each, grouped heads: the encoder's states are read once for all beams
        dict(name="cross_step_batch", op="cross", B=64, q_lo=4, q_hi=4, kv_lo=512, kv_hi=4096, Hq=32, Hkv=8, d=128,
             dtype="bf16", pad=False, packed=False, image=0, lens=32),
        # a small fp32 batch padded to its longest source
        dict(name="cross_step_f32", op="cross", B=8, q_lo=5, q_hi=5, kv_lo=0, kv_hi=900, Hq=16, Hkv=16, d=64,
             dtype="f32", pad=True, packed=True, image=0, lens=33),
        # ragged prompts over ragged sources, heads of 64
        dict(name="cross_prompt", op="cross", B=9, q_lo=1, q_hi=447, kv_lo=200, kv_hi=1500, Hq=16, Hkv=16, d=64,
             dtype="bf16", pad=False, packed=True, image=0, lens=34),
        # a long prompt over the states of four image tiles
        dict(name="cross_long", op="cross", B=1, q_lo=8192, q_hi=8192, kv_lo=6404, kv_hi=6404, Hq=16, Hkv=2, d=128,
             dtype="bf16", pad=False, packed=False, image=0, lens=35),
        # text with images in between: a token sees the last image before it, the first tokens none
        dict(name="cross_images", op="cross", B=3, q_lo=600, q_hi=2500, kv_lo=3000, kv_hi=8000, Hq=32, Hkv=8, d=128,
             dtype="bf16", pad=False, packed=False, image=1025, lens=36),
        # one user's step: 4 beams, a small vocabulary in fp32
        dict(name="select_one", op="select", B=1, K=4, V=32000, M=8, dtype="f32", eos=True, keep=1.0, pad=0, lens=37),
        # a full batch over a large vocabulary
        dict(name="select_batch", op="select", B=64, K=8, V=128000, M=16, dtype="bf16", eos=True, keep=1.0, pad=0,
             lens=38),
        # constrained decoding: an odd vocabulary padded for the projection, most tokens banned
        dict(name="select_banned", op="select", B=7, K=5, V=50257, M=10, dtype="bf16", eos=True, keep=0.02, pad=47,
             lens=39),
        # one user's step: 4 beams
        dict(name="reorder_one", op="reorder", B=1, K=4, lo=1777, hi=1777, new=150, layers=1, Hkv=2, d=128,
             dtype="bf16", cp=2, I=8, lens=40),
        # a full batch of a model with 8 kv heads, one layer
        dict(name="reorder_batch", op="reorder", B=64, K=8, lo=64, hi=2048, new=128, layers=1, Hkv=8, d=128,
             dtype="bf16", cp=2, I=8, lens=41),
        # all layers of a small model in one call
        dict(name="reorder_layers", op="reorder", B=6, K=5, lo=20, hi=1500, new=64, layers=24, Hkv=16, d=64,
             dtype="bf16", cp=1, I=16, lens=42),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["step", "step", "prompt", "prompt", "select", "select", "reorder", "reorder"])
    c = dict(lens=rng.randrange(1 << 20))
    if op in ("step", "prompt"):
        d, Hkv = rng.choice([64, 128]), rng.choice([1, 2, 4, 8, 16])
        G = rng.choice([1, 1, 2, 3, 4, 6, 8])
        if op == "step":
            dtype = rng.choice(["bf16", "bf16", "f32"])
            B, q_hi, kv = _log(rng, 1, 64), rng.randint(1, 8), _log(rng, 1, 16384)
            # no more encoder states than the full decode batch has; fp32 a quarter of them
            most = 64 * 2000 * 8 * 128 // (1 if dtype == "bf16" else 4)
            kv = max(1, min(kv, most // (B * Hkv * d)))
            if dtype == "f32":
                G = min(G, 4)
            c.update(B=B, q_lo=q_hi, q_hi=q_hi, kv_hi=kv, dtype=dtype, image=0)
        else:
            B, q_hi, kv = _log(rng, 1, 8), _log(rng, 1, 8192), _log(rng, 1, 8192)
            q_hi = max(1, min(q_hi, 8192 * 6404 * 14 // (B * kv * G * Hkv)))
            c.update(B=B, q_lo=max(1, q_hi // 8), q_hi=q_hi, kv_hi=kv, dtype="bf16",
                     image=rng.choice([0, 0, _log(rng, 16, 2000)]))
        c.update(op="cross", Hq=G * Hkv, Hkv=Hkv, d=d, kv_lo=rng.choice([0, c["kv_hi"] // 8, c["kv_hi"]]),
                 pad=rng.random() < 0.3, packed=rng.random() < 0.5)
    elif op == "select":
        B, K, V = _log(rng, 1, 64), rng.choice([1, 2, 3, 4, 5, 8, 12, 16]), _log(rng, 500, 260000)
        B = max(1, min(B, 64 * 8 * 128000 // (K * V)))
        c.update(op="select", B=B, K=K, V=V, M=2 * K, dtype=rng.choice(["bf16", "f32"]), eos=rng.random() < 0.7,
                 keep=rng.choice([1.0, 1.0, 0.3, 0.01]), pad=rng.choice([0, 0, rng.randint(1, 127)]))
        if c["dtype"] == "f32":
            c["B"] = max(1, B // 2)
    else:
        B, K, hi = _log(rng, 1, 64), rng.choice([2, 3, 4, 5, 8, 12, 16]), _log(rng, 1, 4096)
        Hkv, d = rng.choice([1, 2, 4, 8, 16]), rng.choice([64, 128])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        layers = rng.choice([1, 1, 2, 6])
        # no larger than the full batch
        size = Hkv * d * layers * (1 if dtype == "bf16" else 2)
        while B > 1 and B * K * size > 64 * 8 * 8 * 128:
            B //= 2
        hi = max(1, min(hi, 64 * 1024 * 1024 // (B * size)))
        c.update(op="reorder", B=B, K=K, lo=max(1, hi // 8), hi=hi, new=rng.randint(1, 128), layers=layers, Hkv=Hkv,
                 d=d, dtype=dtype, cp=rng.choice([1, 1, 2, 4]), I=rng.choice([1, 5, 8, 16]))
    return c


def _lens(case, lo, hi, salt):
    r = random.Random(case["lens"] * 7 + salt)
    return [r.randint(lo, hi) for _ in range(case["B"])]


def _cross_spans(case):
    """Per sequence: query rows, keys, and with images each row's range of keys."""
    T, S = _lens(case, case["q_lo"], case["q_hi"], 0), _lens(case, case["kv_lo"], case["kv_hi"], 1)
    if not case["image"]:
        return T, S, None
    r, spans = random.Random(case["lens"] * 7 + 2), []
    for t, s in zip(T, S):
        images = -(-s // case["image"])
        starts = sorted(r.randint(0, t) for _ in range(images))  # the row at which each image comes
        seen = np.searchsorted(np.array(starts + [t + 1]), np.arange(t), side="right")  # images before each row
        lo = np.maximum(seen - 1, 0) * case["image"]
        spans.append(np.stack([lo, np.where(seen > 0, np.minimum(lo + case["image"], s), lo)], -1))
    return T, S, np.concatenate(spans).astype(np.int32)


def _beams(case):
    """Per sequence of a reorder case: cached tokens, tokens of its prompt, parents."""
    L = _lens(case, case["lo"], case["hi"], 0)
    r = random.Random(case["lens"] * 7 + 1)
    # now and then a sequence in its first step, whose beams still share the page that the prompt ended in
    P = [n if r.random() < 0.15 else max(0, n - r.randint(1, case["new"])) for n in L]
    # good beams have several children
    parents = [[min(int(r.expovariate(1.0) * case["K"] / 3), case["K"] - 1) for _ in range(case["K"])] for _ in L]
    return L, P, parents


def _held(n, rank, case):
    """Tokens of n that a rank holds."""
    period = case["I"] * case["cp"]
    return n // period * case["I"] + min(max(n % period - rank * case["I"], 0), case["I"])


def _paging(case):
    """Tables before the step and own pages, int32 [cp, B K, columns], the pool's pages, and for each beam
    and rank the column being filled and the tokens in it."""
    L, P, parents = _beams(case)
    K, cp = case["K"], case["cp"]
    wide = max(_held(n, 0, case) for n in L) // PAGE + 1
    r = random.Random(case["lens"] * 7 + 3)
    tables, mine = (np.full((cp, len(L) * K, wide), -1, np.int64) for _ in range(2))
    column, fill = (np.zeros((cp, len(L)), np.int64) for _ in range(2))
    pool = 0
    for k in range(cp):
        n = 0
        for b, (tokens, prompt) in enumerate(zip(L, P)):
            held, start = _held(tokens, k, case), _held(prompt, k, case)
            column[k, b], fill[k, b] = held // PAGE, held % PAGE
            at = slice(b * K, (b + 1) * K)
            fresh = prompt == tokens
            shared = -(-start // PAGE) if fresh else start // PAGE  # columns that every beam has in common
            tables[k, at, :shared] = n + np.arange(shared)
            n += shared
            first = start // PAGE
            count = column[k, b] - first + 1
            mine[k, at, first:first + count] = n + np.arange(K * count).reshape(K, count)
            n += K * count
            for c in range(shared, column[k, b]):  # full pages: any beam's
                tables[k, at, c] = mine[k, [b * K + r.randrange(K) for _ in range(K)], c]
            if not fresh and fill[k, b]:
                tables[k, at, column[k, b]] = mine[k, at, column[k, b]]
        pool = max(pool, n)
    return tables, mine, pool, column, fill


# ------------------------------------------------------------------------------------ the inputs

def _dev():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _gen(seed):
    return torch.Generator(device=_dev()).manual_seed(seed)


def _randn(shape, g, dtype):
    return torch.randn(*shape, generator=g, device=_dev(), dtype=torch.float32).to(dtype)


def _ints(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x), dtype=dtype).to(_dev())


def _cu(lens):
    return _ints(np.cumsum([0] + list(lens)))


def prepare(case, seed):
    g, dev = _gen(seed), _dev()
    s = dict(case=case)
    if case["op"] == "cross":
        T, S, ranges = _cross_spans(case)
        dt, Hkv, d, N = DT[case["dtype"]], case["Hkv"], case["d"], sum(T)
        rows = [max(S)] * len(S) if case["pad"] else S
        if case["packed"]:  # k and v are the columns of one projection of the encoder's states
            k, v = _randn((max(1, sum(rows)), 2 * Hkv, d), g, dt).split([Hkv, Hkv], 1)
        else:
            k, v = (_randn((max(1, sum(rows)), Hkv, d), g, dt) for _ in range(2))
        s.update(q=_randn((N, case["Hq"], d), g, dt), k=k, v=v, cu_q=_cu(T), cu_kv=_cu(rows), max_q=max(T),
                 max_kv=max(S), kv_lens=_ints(S) if case["pad"] else None,
                 ranges=_ints(ranges) if ranges is not None else None)
        return s
    if case["op"] == "select":
        B, K, V = case["B"], case["K"], case["V"]
        logits = 3 * torch.randn(B, K, V + case["pad"], generator=g, device=dev)
        eos = 2
        if case["eos"]:  # the end is likely for some beams
            logits[..., eos] += 8 * torch.rand(B, K, generator=g, device=dev)
        if case["keep"] < 1:
            logits.masked_fill_(torch.rand(B, 1, V + case["pad"], generator=g, device=dev) > case["keep"], -math.inf)
        scores = -10 + 0.7 * torch.randn(B, K, generator=g, device=dev)
        scores = scores.sort(-1, descending=True).values
        if case["keep"] < 1:
            scores[:, -1] = -math.inf  # a beam that nothing could continue
        s.update(logits=logits.to(DT[case["dtype"]])[..., :V], scores=scores, eos=eos if case["eos"] else -1)
        return s
    tables, mine, pool, column, fill = _paging(case)
    perm = np.random.default_rng(seed).permuted(np.tile(np.arange(pool), (case["cp"], 1)), axis=1)
    rank = np.arange(case["cp"])[:, None, None]
    tables, mine = (np.where(t >= 0, perm[rank, np.maximum(t, 0)], -1) for t in (tables, mine))
    L, _, parents = _beams(case)
    shape = (case["layers"], case["cp"], pool, case["Hkv"], PAGE, case["d"])
    dt = DT[case["dtype"]]
    s.update(k_cache=_randn(shape, g, dt), v_cache=_randn(shape, g, dt), tables=_ints(tables), mine=_ints(mine),
             tables_out=_ints(np.full_like(tables, -1)), seq_lens=_ints(L), parents=_ints(parents))
    return s


# ------------------------------------------------------------------------------------ plain forms

def _rows_of(cu, total):
    """(sequence, index within it) of each row."""
    row = torch.arange(total, device=cu.device)
    seq = torch.searchsorted(cu[1:].long(), row, right=True)
    return seq, row - cu.long()[seq]


def _cross(s):
    case, dev = s["case"], s["q"].device
    B, d, Hkv, N = case["B"], case["d"], case["Hkv"], s["q"].shape[0]
    cu_q, cu_kv = s["cu_q"].long(), s["cu_kv"].long()
    most = max(1, s["max_kv"])
    i, j = torch.arange(s["max_q"], device=dev)[None], torch.arange(most, device=dev)[None]
    rows = torch.minimum(cu_q[:-1, None] + i, cu_q[-1:] - 1)
    keys = torch.clamp(torch.minimum(cu_kv[:-1, None] + j, cu_kv[-1:] - 1), min=0)
    lens = s["kv_lens"].long() if s["kv_lens"] is not None else cu_kv[1:] - cu_kv[:-1]
    q = s["q"][rows].float().view(B, s["max_q"], Hkv, -1, d).permute(0, 2, 3, 1, 4)
    k = s["k"][keys].float().permute(0, 2, 3, 1)[:, :, None]
    v = s["v"][keys].float().permute(0, 2, 1, 3)[:, :, None]
    # rows behind a sequence's states are not its values: whatever lies there is left out
    v = v.masked_fill((j >= lens[:, None])[:, None, None, :, None], 0.0)
    mask = (j < lens[:, None])[:, None]
    if s["ranges"] is not None:
        span = s["ranges"].long()[rows]
        mask = mask & (j[:, None] >= span[..., :1]) & (j[:, None] < span[..., 1:])
    score = q @ k
    score *= 1.0 / math.sqrt(d)
    score.masked_fill_(~mask[:, None, None], -math.inf)
    m = score.amax(-1, keepdim=True)
    score -= torch.where(m > -math.inf, m, 0.0)
    p = score.exp_()
    total = p.sum(-1, keepdim=True)
    o = p @ v / torch.where(total > 0, total, 1)
    lse = (m + total.log()).squeeze(-1)
    b, t = _rows_of(s["cu_q"], N)
    o = o.permute(0, 3, 1, 2, 4)[b, t].reshape(N, case["Hq"], d)
    return o.to(s["q"].dtype), lse.permute(0, 3, 1, 2)[b, t].reshape(N, case["Hq"])


def _select(s):
    """In 64 bits: continuations of different beams lie close to one another."""
    case = s["case"]
    K, V, M = case["K"], case["V"], case["M"]
    x = s["logits"].double()
    x = torch.where(x.isnan(), -math.inf, x)
    m = x.amax(-1, keepdim=True)
    x = x - torch.where(m > -math.inf, m, 0.0)
    x = s["scores"].double()[..., None] + (x - x.exp().sum(-1, keepdim=True).log())
    x = torch.where(x.isnan(), -math.inf, x).flatten(1)  # a beam without a token: -inf less -inf
    best, at = x.sort(dim=-1, descending=True, stable=True)
    best, at = best[:, :M], at[:, :M]
    beams, tokens = at // V, at % V
    last = (tokens == s["eos"]).to(torch.int8)
    on = last.sort(dim=-1, stable=True).indices[:, :K]  # the first K that do not end the sequence
    take = [y.gather(1, on) for y in (best, beams, tokens)]
    return [take[0].float(), take[1].int(), take[2].int(), best.float(), beams.int(), tokens.int()]


def _reorder(s):
    case, dev = s["case"], s["tables"].device
    B, K, cp, I = case["B"], case["K"], case["cp"], case["I"]
    L = s["seq_lens"].long()[None]
    rank = torch.arange(cp, device=dev)[:, None]
    held = L // (I * cp) * I + (L % (I * cp) - rank * I).clamp(0, I)  # [cp, B]
    column, fill = held // PAGE, held % PAGE
    old, mine = (t.long().view(cp, B, K, -1) for t in (s["tables"], s["mine"]))
    at = s["parents"].long()[None, :, :, None].expand_as(old)
    new = old.gather(2, at)
    c = torch.arange(old.shape[-1], device=dev)
    here = column[:, :, None, None]
    out = s["tables_out"].view(cp, B, K, -1)
    out.copy_(torch.where(c < here, new, torch.where(c == here, mine, out.long())))
    col = here.clamp(max=old.shape[-1] - 1).expand(-1, -1, K, 1)
    src, dst = (t.gather(3, col).squeeze(-1) for t in (new, mine))
    need = ((fill > 0)[:, :, None] & (src != dst)).nonzero(as_tuple=True)
    r, src, dst, n = need[0], src[need], dst[need], fill[need[0], need[1]]
    live = (torch.arange(PAGE, device=dev) < n[:, None])[None, :, None, :, None]
    for cache in (s["k_cache"], s["v_cache"]):
        cache[:, r, dst] = torch.where(live, cache[:, r, src], cache[:, r, dst])
    return s["tables_out"], s["k_cache"], s["v_cache"]


# ------------------------------------------------------------------------------------ the framework's calls

def _own_cross(s):
    import context_gqa_attention_gb300 as cpa
    return cpa.cp_cross_attention(s["q"], s["cu_q"], s["k"], s["v"], s["cu_kv"], kv_lens=s["kv_lens"],
                                  key_ranges=s["ranges"], max_seqlen_q=s["max_q"], max_seqlen_kv=s["max_kv"])


def _own_select(s):
    import context_gqa_attention_gb300 as cpa
    case = s["case"]
    if "workspace" not in s:  # a program keeps its zero-filled workspace
        size = cpa.cp_beam_select_workspace_size(case["B"], case["K"], case["V"], case["M"])
        s["workspace"] = torch.zeros(size, dtype=torch.uint8, device=s["logits"].device)
    return cpa.cp_beam_select(s["logits"], s["scores"], num_candidates=case["M"], eos_token=s["eos"],
                              workspace=s["workspace"])


def _own_reorder(s):
    import context_gqa_attention_gb300 as cpa
    case = s["case"]
    cpa.cp_beam_reorder(s["parents"], s["seq_lens"], s["tables"], s["mine"], s["k_cache"], s["v_cache"], case["cp"],
                        case["I"], tables_out=s["tables_out"])
    return s["tables_out"], s["k_cache"], s["v_cache"]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"cross": _own_cross, "select": _own_select, "reorder": _own_reorder}[op](state)
    return {"cross": _cross, "select": _select, "reorder": _reorder}[op](state)


# ------------------------------------------------------------------------------------ work

def work(case):
    e = 4 if case.get("dtype") == "f32" else 2
    if case["op"] == "cross":
        T, S, ranges = _cross_spans(case)
        d, Hq, Hkv = case["d"], case["Hq"], case["Hkv"]
        pairs, keys, at = 0, 0, 0
        for t, n in zip(T, S):
            if ranges is None:
                pairs, keys = pairs + t * n, keys + n
            else:
                span = ranges[at:at + t]
                pairs += int((span[:, 1] - span[:, 0]).sum())
                seen = np.zeros(n + 1, np.int64)  # keys that some row sees
                np.add.at(seen, span[:, 0], 1)
                np.add.at(seen, span[:, 1], -1)
                keys += int((seen.cumsum()[:n] > 0).sum())
            at += t
        return {"bytes": e * d * (2 * sum(T) * Hq + 2 * keys * Hkv) + 4 * sum(T) * Hq, "flops": 4 * d * Hq * pairs}
    if case["op"] == "select":
        rows = case["B"] * case["K"]
        return {"bytes": rows * (e * case["V"] + 4) + 12 * (rows + case["B"] * case["M"]), "flops": 4 * rows * case["V"]}
    tables, mine, _, column, fill = _paging(case)
    _, _, parents = _beams(case)
    K, pages = case["K"], 0  # rows that are read and rows that are written
    for k in range(case["cp"]):
        for b, p in enumerate(parents):
            if fill[k, b]:
                src = tables[k, [b * K + x for x in p], column[k, b]]
                dst = mine[k, b * K:(b + 1) * K, column[k, b]]
                moved = src != dst
                pages += int(fill[k, b]) * (len(set(src[moved].tolist())) + int(moved.sum()))
    entries = K * int((column + 1).sum())
    return {"bytes": 2 * case["layers"] * pages * case["Hkv"] * case["d"] * e + 8 * entries + 4 * case["B"] * (K + 1),
            "flops": 0}


# ------------------------------------------------------------------------------------ 64 bits

def _exact_cross(s):
    case, dev = s["case"], s["q"].device
    T, S, ranges = _cross_spans(case)
    G, N = case["Hq"] // case["Hkv"], sum(T)
    out = torch.zeros(N, case["Hq"], case["d"], dtype=torch.float64, device=dev)
    lse = torch.full((N, case["Hq"]), -math.inf, dtype=torch.float64, device=dev)
    starts = np.cumsum([0] + ([max(S)] * len(S) if case["pad"] else S))
    row = 0
    for t, n, k0 in zip(T, S, starts):
        for i0 in range(0, t if n else 0, 4096):
            i1 = min(t, i0 + 4096)
            seen = torch.ones(i1 - i0, n, dtype=torch.bool, device=dev)
            if ranges is not None:
                span = torch.as_tensor(ranges[row + i0:row + i1].astype(np.int64)).to(dev)
                at = torch.arange(n, device=dev)
                seen = ~((at < span[:, :1]) | (at >= span[:, 1:]))
            for h in range(case["Hq"]):
                q = s["q"][row + i0:row + i1, h].double() / math.sqrt(case["d"])
                x = torch.einsum("id,jd->ij", q, s["k"][k0:k0 + n, h // G].double()).masked_fill(~seen, -math.inf)
                z = torch.logsumexp(x, -1)
                w = torch.exp(x - z.clamp(min=-1e300)[:, None])
                out[row + i0:row + i1, h] = w @ s["v"][k0:k0 + n, h // G].double()
                lse[row + i0:row + i1, h] = z
        row += t
    return out, lse


def _exact_select(s):
    case = s["case"]
    V, M, K = case["V"], case["M"], case["K"]
    got = [[] for _ in range(6)]
    for b in range(case["B"]):
        x = s["logits"][b].double().nan_to_num(nan=-math.inf, posinf=math.inf, neginf=-math.inf)
        x = (torch.log_softmax(x, -1) + s["scores"][b].double()[:, None]).nan_to_num(nan=-math.inf, neginf=-math.inf)
        x = x.reshape(-1)
        border = x.kthvalue(x.numel() - M + 1).values
        above, equal = (x > border).nonzero()[:, 0].cpu().numpy(), (x == border).nonzero()[:M, 0].cpu().numpy()
        at = np.concatenate([above, equal])
        value = x[torch.as_tensor(at).to(x.device)].cpu().numpy()
        order = np.lexsort((at, -value))[:M]
        best = [(value[o], at[o] // V, at[o] % V) for o in order]
        on = [c for c in best if c[2] != s["eos"]][:K]
        for i, c in enumerate((on, best)):
            for f in range(3):
                got[3 * i + f].append([y[f] for y in c])
    kinds = (torch.float64, torch.int32, torch.int32) * 2
    return [torch.tensor(np.array(x), dtype=k) for x, k in zip(got, kinds)]


def _exact_reorder(s):
    case = s["case"]
    tables, mine = s["tables"].cpu().numpy(), s["mine"].cpu().numpy()
    L, _, parents = _beams(case)
    K = case["K"]
    out = s["tables_out"].cpu().numpy().copy()
    moves = []
    for k in range(case["cp"]):
        for b, n in enumerate(L):
            held = sum(1 for p in range(n) if p // case["I"] % case["cp"] == k)
            full, rest = divmod(held, PAGE)
            for j, p in enumerate(parents[b]):
                out[k, b * K + j, :full] = tables[k, b * K + p, :full]
                out[k, b * K + j, full] = mine[k, b * K + j, full]
                if rest:
                    moves.append((k, tables[k, b * K + p, full], mine[k, b * K + j, full], rest))
    caches = []
    for cache in (s["k_cache"], s["v_cache"]):
        new = cache.double()
        for k, src, dst, rest in moves:
            new[:, k, int(dst), :, :rest] = cache[:, k, int(src), :, :rest].double()
        caches.append(new)
    return torch.from_numpy(out), caches[0], caches[1]


def exact(case, seed):
    s = prepare(case, seed)
    return {"cross": _exact_cross, "select": _exact_select, "reorder": _exact_reorder}[case["op"]](s)
