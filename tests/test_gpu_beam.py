"""Selection and reordering of beams against the float64 oracle: ties, banned tokens, NaN and infinities, odd sizes and
alignments; tables, pages and 4-bit records bit for bit; and a beam search of all calls together.

Scores: a sum of weights is off by at most 2^-20 (exponentials by 2^-22 of themselves and, their exponents being fp32,
2^-23 of exponents up to 2^4 for what counts; fp32 sums), its logarithm by as much, and the score is rounded once:
2^-19 + 2^-24 |score|.  Beams and tokens are equal to the oracle's; the inputs' scores differ by more than twice that,
or are equal exactly, which is asserted."""
import math

import numpy as np
import pytest
import torch

from oracle import beam_oracle as bo
from oracle import serving_oracle as so

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
I32 = dict(dtype=torch.int32, device=DEV)


def _np(t):
    return t.detach().double().cpu().numpy()


# ------------------------------------------------------------------------------------ selection

def check_select(got, logits, scores, M, eos):
    ns, nb, nt, cs, cb, ct = (x.cpu().numpy() for x in got)
    B, K, _ = logits.shape
    assert ns.shape == nb.shape == nt.shape == (B, K) and cs.shape == cb.shape == ct.shape == (B, M)
    x, s = _np(logits), _np(scores)
    for b in range(B):
        best, on = bo.select(x[b], s[b], M, eos)
        value = np.array([c[0] for c in best])
        gap = value[:-1] - value[1:]
        same = np.array([p[1] == q[1] for p, q in zip(best, best[1:])], dtype=bool)  # compared exactly
        assert (same | (gap > 2.0 ** -18) | (gap == 0) | np.isnan(gap)).all(), "the inputs have a near tie"
        for have, want in (((cs, cb, ct), best), ((ns, nb, nt), on)):
            w = np.array([c[0] for c in want])
            fin = np.isfinite(w)
            assert np.array_equal(have[1][b], [c[1] for c in want]) and np.array_equal(have[2][b], [c[2] for c in want])
            assert np.array_equal(np.isneginf(have[0][b]), ~fin)
            assert (np.abs(have[0][b][fin] - w[fin]) <= 2.0 ** -19 + 2.0 ** -24 * np.abs(w[fin])).all()


SELECT = [
    # B, K, V, M, dtype, eos, row padding
    (1, 1, 1, 1, "f32", -1, 0),
    (1, 1, 7, 4, "bf16", -1, 1),
    (2, 3, 2, 6, "f32", 1, 0),                 # all continuations are candidates
    (1, 4, 32000, 8, "f32", 2, 0),
    (3, 5, 50257, 10, "bf16", 11, 0),          # odd: rows at every alignment
    (3, 5, 50257, 10, "f32", 11, 3),
    (2, 2, 4099, 5, "bf16", 7, 5),
    (70, 2, 1000, 4, "bf16", -1, 0),
    (5, 16, 30011, 32, "bf16", 3, 0),
    (2, 32, 2048, 64, "f32", 0, 0),
    (1, 32, 65, 64, "bf16", 5, 0),
    (40, 8, 128000, 16, "bf16", 2, 0),         # the long slices
    (40, 4, 60001, 8, "f32", 2, 1),
    (1, 1, 260000, 2, "f32", -1, 0),
]


@pytest.mark.parametrize("B,K,V,M,dtype,eos,pad", SELECT)
def test_selection(lib, B, K, V, M, dtype, eos, pad):
    g = torch.Generator(device=DEV).manual_seed(V + K)
    logits = (3 * torch.randn(B, K, V + pad, generator=g, device=DEV)).to(DT[dtype])
    if eos >= 0:
        logits[..., eos] += 9
    if pad:
        logits[..., V:] = math.inf if dtype == "f32" else math.nan
    scores = -10 + torch.randn(B, K, generator=g, device=DEV)
    got = lib.cp_beam_select(logits[..., :V], scores, num_candidates=M, eos_token=eos)
    check_select(got, logits[..., :V], scores, M, eos)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["equal", "two values", "falling", "rising", "banned", "few", "none", "nan", "inf",
                                  "huge", "zeros"])
@pytest.mark.parametrize("V", [300, 5003, 40000])
def test_selection_of_special_rows(lib, kind, dtype, V):
    B, K, M = 3, 4, 8
    g = torch.Generator(device=DEV).manual_seed(V)
    x = torch.randn(B, K, V, generator=g, device=DEV)
    if kind == "equal":
        x.fill_(0.5)
    elif kind == "two values":
        x = (x > 0).float()
    elif kind in ("falling", "rising"):
        x = torch.linspace(20, -20, V, device=DEV).expand(B, K, V) * (1 if kind == "falling" else -1) + \
            torch.arange(K, device=DEV)[:, None] * 0.011
    elif kind == "banned":
        x[torch.rand(B, 1, V, generator=g, device=DEV).expand(B, K, V) < 0.97] = -math.inf
    elif kind == "few":                        # fewer continuations than candidates
        x[:] = -math.inf
        x[:, 1, V // 2], x[:, 3, V - 1], x[:, 3, 0] = 1.5, -2.0, 3.0
    elif kind == "none":
        x[:] = -math.inf
    elif kind == "nan":
        x[torch.rand(B, K, V, generator=g, device=DEV) < 0.5] = math.nan
        x[1, 2] = math.nan
    elif kind == "inf":
        x[0, 1, 3], x[0, 1, V - 7], x[1, 0, 0], x[2] = math.inf, math.inf, math.inf, -math.inf
        x[2, 0, 5] = math.inf
    elif kind == "huge":
        x *= 1e30
    elif kind == "zeros":                      # 0 and -0 are one value
        x = torch.where(x > 0, 0.0, -0.0)
    x = x.to(DT[dtype]).contiguous()
    scores = torch.tensor([[-1.0, -2.5, -3.25, -7.125]] * B, device=DEV)
    scores[1, 0] = -math.inf
    scores[2, 3] = math.nan
    got = lib.cp_beam_select(x, scores, num_candidates=M, eos_token=5)
    scores[2, 3] = -math.inf
    check_select(got, x, scores, M, 5)


def test_the_first_step_expands_one_beam(lib):
    logits = torch.randn(2, 5, 999, device=DEV)
    logits[:] = logits[:, :1]
    scores = torch.full((2, 5), -math.inf, device=DEV)
    scores[:, 0] = 0
    got = lib.cp_beam_select(logits, scores, num_candidates=10, eos_token=0)
    check_select(got, logits, scores, 10, 0)
    assert bool((got[1] == 0).all())


def test_selection_shares_a_workspace_and_is_the_same_each_time(lib):
    """Shapes in turn, the fused decode's workspace, graphs that share one; results do not depend on the order."""
    shapes = [(3, 4, 32000, 8, "f32"), (64, 2, 999, 4, "bf16"), (1, 16, 50257, 32, "bf16")]
    ws = torch.zeros(max(lib.cp_beam_select_workspace_size(*s[:4]) for s in shapes), dtype=torch.uint8, device=DEV)
    data, graphs = [], []
    for B, K, V, M, dtype in shapes:
        logits, scores = (2 * torch.randn(B, K, V, device=DEV)).to(DT[dtype]), torch.randn(B, K, device=DEV)
        first = lib.cp_beam_select(logits, scores, num_candidates=M, eos_token=1)
        check_select(first, logits, scores, M, 1)
        outs = [torch.empty_like(x) for x in first]
        names = ("next_scores", "next_beams", "next_tokens", "cand_scores", "cand_beams", "cand_tokens")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            lib.cp_beam_select(logits, scores, num_candidates=M, eos_token=1, workspace=ws, **dict(zip(names, outs)))
        data.append((first, outs)), graphs.append((graph, logits, scores))     # (what a graph reads stays alive)
    for _ in range(20):
        for (graph, *_), (first, outs) in zip(graphs, data):
            for x in outs:
                x.fill_(-3)
            graph.replay()
            assert all(torch.equal(x, y) for x, y in zip(first, outs))
    torch.cuda.synchronize()
    assert int(ws[:65536 * 4].view(torch.int32).abs().max()) == 0


# ------------------------------------------------------------------------------------ reordering

def paging(lens, K, cp, I, cols, r, fresh=()):
    """Tables whose beams share full pages and own the ones being filled (but for fresh sequences), the own pages."""
    B = len(lens)
    tables, own = (np.full((cp, B * K, cols), -1, np.int32) for _ in range(2))
    pool = 0
    for k in range(cp):
        ids = 0
        for b, n in enumerate(lens):
            full, rest = divmod(bo.held(n, k, cp, I), 16)
            at = slice(b * K, (b + 1) * K)
            for c in range(full + 1):
                if c >= cols:
                    continue
                own[k, at, c] = ids + np.arange(K)
                ids += K
                if c < full:
                    tables[k, at, c] = own[k, b * K + r.integers(0, K, K), c]
                elif rest:
                    tables[k, at, c] = own[k, b * K, c] if b in fresh else own[k, at, c]
            if b in fresh and rest and full < cols:      # the prompt's last page is nobody's own
                tables[k, at, full] = ids
                ids += 1
        pool = max(pool, ids)
    return tables, own, pool


def bits(t):
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


@pytest.mark.parametrize("B,K,cp,I,Hkv,d,kind,layers", [
    (1, 1, 1, 16, 1, 64, "bf16", 1), (1, 4, 2, 8, 2, 128, "bf16", 1), (5, 3, 4, 5, 3, 64, "bf16", 2),
    (3, 5, 1, 1, 8, 128, "f32", 1), (4, 8, 2, 8, 2, 64, "f32", 3), (3, 16, 2, 3, 1, 128, "bf16", 1),
    (2, 32, 1, 16, 2, 64, "bf16", 2), (2, 17, 3, 8, 2, 128, "f32", 1), (4, 4, 2, 8, 2, 128, "q4", 2),
    (3, 6, 1, 16, 5, 64, "q4", 1), (70, 2, 1, 8, 1, 64, "bf16", 1)])
@pytest.mark.parametrize("in_place", [False, True])
def test_reordering(lib, B, K, cp, I, Hkv, d, kind, layers, in_place):
    r = np.random.default_rng(B * 100 + K)
    lens = [int(x) for x in r.choice([0, 1, 15, 16, 17, 31, 32, 33, 64, 100, 159], B)]
    cols = 12
    tables, own, pool = paging(lens, K, cp, I, cols, r, fresh={0})
    parents = r.integers(0, K, (B, K)).astype(np.int32)
    if B > 1:
        parents[1] = r.permutation(K)                    # pages change places
    shape = ((layers,) if layers > 1 else ()) + (cp, pool + 2, Hkv) + ((9 * d,) if kind == "q4" else (16, d))
    g = torch.Generator(device=DEV).manual_seed(3)
    caches = [torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8) if kind == "q4"
              else torch.randn(shape, generator=g, device=DEV).to(DT[kind]) for _ in range(2)]
    # the oracle in the pools' own bits
    old = [x.cpu().numpy() if kind == "q4" else x.float().cpu().numpy() for x in caches]
    want_t, want = bo.reorder(parents.tolist(), lens, tables, own, old, cp, I)
    t = torch.tensor(tables, device=DEV)
    out = t if in_place else torch.full_like(t, -7)
    err = torch.zeros(1, **I32)
    got = lib.cp_beam_reorder(torch.tensor(parents, device=DEV), torch.tensor(lens, **I32), t, torch.tensor(own, device=DEV),
                              *caches, cp, I, tables_out=out, err=err)
    assert got is out and int(err) == 0
    for x, w in zip(caches, want):
        assert np.array_equal(x.cpu().numpy() if kind == "q4" else x.float().cpu().numpy(), w)
    o = out.cpu().numpy()
    for k in range(cp):
        for b, n in enumerate(lens):
            c = min(cols, bo.held(n, k, cp, I) // 16 + 1)
            rows = slice(b * K, (b + 1) * K)
            assert np.array_equal(o[k, rows, :c], want_t[k, rows, :c])
            assert (o[k, rows, c:] == (tables[k, rows, c:] if in_place else -7)).all()


def test_reordering_of_tables_alone_and_of_layers_one_by_one(lib):
    r = np.random.default_rng(5)
    lens, K, cp, I = [40, 77, 5], 4, 2, 8
    tables, own, pool = paging(lens, K, cp, I, 6, r)
    parents = torch.tensor(r.integers(0, K, (3, K)), **I32)
    t, o, n = torch.tensor(tables, device=DEV), torch.tensor(own, device=DEV), torch.tensor(lens, **I32)
    caches = [torch.randn(5, cp, pool, 2, 16, 64, device=DEV).to(torch.bfloat16) for _ in range(2)]
    once = [x.clone() for x in caches]
    a = lib.cp_beam_reorder(parents, n, t, o, *once, cp, I, tables_out=torch.zeros_like(t))
    for layer in range(5):
        b = lib.cp_beam_reorder(parents, n, t, o, caches[0][layer], caches[1][layer], cp, I, tables_out=torch.zeros_like(t))
        assert torch.equal(a, b)
    assert all(torch.equal(bits(x), bits(y)) for x, y in zip(once, caches))
    assert torch.equal(a, lib.cp_beam_reorder(parents, n, t, o, None, None, cp, I, tables_out=torch.zeros_like(t)))


@pytest.mark.parametrize("in_place", [False, True])
def test_reordering_reports_what_is_out_of_range(lib, in_place):
    r = np.random.default_rng(6)
    lens, K, cp, I = [40, 77, 21], 3, 2, 8
    tables, own, pool = paging(lens, K, cp, I, 4, r)
    base = [torch.randn(cp, pool, 1, 16, 64, device=DEV) for _ in range(2)]
    parents = r.integers(0, K, (3, K)).astype(np.int32)

    def run(parents, lens, tables, own):
        caches, err = [x.clone() for x in base], torch.zeros(1, **I32)
        t = torch.tensor(tables, device=DEV)
        out = t if in_place else torch.full_like(t, -7)
        lib.cp_beam_reorder(torch.tensor(parents, device=DEV), torch.tensor(lens, **I32), t, torch.tensor(own, device=DEV),
                            *caches, cp, I, tables_out=out, err=err)
        return int(err), out.cpu().numpy(), [x.cpu().numpy() for x in caches]

    e0, t0, c0 = run(parents, lens, tables, own)
    assert e0 == 0
    untouched = tables if in_place else np.full_like(tables, -7)
    for value in (-1, K, 2 ** 31 - 1, -2 ** 31):             # a parent that is none: that beam stays
        p = parents.copy()
        p[1, 2] = value
        e, t, c = run(p, lens, tables, own)
        assert e == 5
        assert np.array_equal(t[:, K + 2], untouched[:, K + 2])
        keep = np.arange(3 * K) != K + 2
        assert np.array_equal(t[:, keep], t0[:, keep])
    for value in (-1, 65, 10 ** 9):                          # a length that the tables do not hold: the sequence stays
        e, t, c = run(parents, [lens[0], 129 if value == 65 else value, lens[2]], tables, own)
        assert e == 5 and np.array_equal(t[:, K:2 * K], untouched[:, K:2 * K])
        assert np.array_equal(t[:, :K], t0[:, :K]) and np.array_equal(t[:, 2 * K:], t0[:, 2 * K:])
    for bad in (-1, pool, 2 ** 31 - 1):
        col = [bo.held(77, k, cp, I) // 16 for k in range(cp)]
        o = own.copy()
        o[0, K + 1, col[0]] = bad                            # an own page outside the pool: the parent's stays
        e, t, c = run(parents, lens, tables, o)
        assert e == 5 and t[0, K + 1, col[0]] == tables[0, K + parents[1, 1], col[0]]
        x = tables.copy()
        x[0, K + parents[1, 1], col[0]] = bad                # a source outside it: nothing is copied
        e, t, c = run(parents, lens, x, own)
        assert e == 5 and t[0, K + 1, col[0]] == own[0, K + 1, col[0]]
        for k in (0, 1):
            assert np.array_equal(c[k][0, own[0, K + 1, col[0]]], base[k].cpu().numpy()[0, own[0, K + 1, col[0]]])
    # exactly full tables: nothing to fill, nothing to report
    e, t, c = run(parents, [lens[0], 128, lens[2]], np.abs(tables) % pool, own)
    assert e == 0


def test_pools_past_32_bit_offsets(lib):
    """Pages at the end of a pool of 6 GB."""
    K, Hkv, d, pages = 3, 8, 128, 200000
    pool = [torch.empty(1, pages, Hkv, 16, d, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    own = torch.tensor([[[pages - 5], [pages - 1], [7]]], **I32)
    for x in pool:
        for p in (pages - 5, pages - 1, 7):
            x[0, p] = torch.randn(Hkv, 16, d, device=DEV)
    old = [[x[0, p].clone() for p in (pages - 5, pages - 1, 7)] for x in pool]
    out = lib.cp_beam_reorder(torch.tensor([[1, 2, 0]], **I32), torch.tensor([11], **I32), own, own, *pool, 1, 16)
    assert torch.equal(out, own)
    for x, o in zip(pool, old):
        for j, (p, src) in enumerate(((pages - 5, 1), (pages - 1, 2), (7, 0))):
            assert torch.equal(x[0, p, :, :11], o[src][:, :11]) and torch.equal(x[0, p, :, 11:], o[j][:, 11:])


# ------------------------------------------------------------------------------------ together

@pytest.mark.parametrize("kind", ["bf16", "q4"])
@pytest.mark.parametrize("cp,I", [(1, 16), (2, 8)])
def test_a_beam_search(lib, kind, cp, I):
    """Selection, reordering, append, self-attention over each beam's table and cross attention over the shared
    states, step after step, on two sequences; every step's attention is that of the beams' histories."""
    B, K, Hq, Hkv, d, V, steps, cols, prompt = 2, 3, 4, 2, 64, 97, 40, 8, 21
    g = torch.Generator(device=DEV).manual_seed(9)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device=DEV).to(torch.bfloat16)

    states = [50, 133]
    ck, cv = rand(sum(states), Hkv, d), rand(sum(states), Hkv, d)
    emb = rand(V, Hq + 2 * Hkv, d)                       # a token's q, k and v
    head = rand(Hq * d, V).float() * 0.1
    beams, own_cols = B * K, -(-(prompt + steps) // 16) + 1
    assert own_cols <= cols
    own = torch.arange(beams * cols, **I32).view(1, beams, cols).expand(cp, -1, -1).contiguous() + B * cols
    pool = (beams + B) * cols
    shape = (cp, pool, Hkv) + ((9 * d,) if kind == "q4" else (16, d))
    dt = torch.uint8 if kind == "q4" else torch.bfloat16
    kc, vc = (torch.zeros(shape, dtype=dt, device=DEV) for _ in range(2))
    tables = torch.full((cp, beams, cols), -1, **I32)
    shared = -(-prompt // 16)
    for b in range(B):                                   # the prompt's pages, one set for all beams of a sequence
        tables[:, b * K:(b + 1) * K, :shared] = torch.arange(b * cols, b * cols + shared, **I32)
    tokens = torch.randint(0, V, (B, prompt), generator=g, device=DEV)
    x = emb[tokens.view(-1)]
    first = tables[:, ::K].contiguous()
    lib.cp_rope_kv_cache_write(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], torch.tensor([0, prompt, 2 * prompt], **I32),
                               torch.zeros(B, **I32), kc, vc, first, cp, I)
    hist = [[tokens[b].tolist()] * K for b in range(B)]
    logits = (0.3 * torch.randn(B, K, V, generator=g, device=DEV)).contiguous()
    logits[:] = logits[:, :1]
    scores = torch.tensor([[0.0] + [-math.inf] * (K - 1)] * B, device=DEV)
    spare = torch.full_like(tables, -1)
    cu = torch.arange(beams + 1, **I32)
    err = torch.zeros(1, **I32)
    seen_parents = set()
    for step in range(steps):
        n = prompt + step
        want = [bo.select(_np(logits[b]), _np(scores[b]), 2 * K, 0)[1] for b in range(B)]
        scores, parents, tok, *_ = lib.cp_beam_select(logits, scores, eos_token=0)
        assert parents.tolist() == [[c[1] for c in w] for w in want] and tok.tolist() == [[c[2] for c in w] for w in want]
        seen_parents.update(map(tuple, parents.tolist()))
        hist = [[hist[b][p] + [t] for p, t in zip(parents[b].tolist(), tok[b].tolist())] for b in range(B)]
        lib.cp_beam_reorder(parents, torch.full((B,), n, **I32), tables, own, kc, vc, cp, I, tables_out=spare, err=err)
        tables, spare = spare, tables
        x = emb[tok.view(-1).long()]
        q = x[:, :Hq].contiguous()
        lib.cp_rope_kv_cache_write(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], cu, torch.full((beams,), n, **I32), kc, vc, tables,
                                   cp, I, err=err)
        lens = torch.full((beams,), n + 1, **I32)
        call = lib.cp_decode_attention_q4 if kind == "q4" else lib.cp_decode_attention_mod
        mine, _ = call(q, kc, vc, tables, lens, cp, I, max_seq_len=n + 1, err=err)
        theirs, _ = lib.cp_cross_attention(q, torch.tensor([0, K, 2 * K], **I32), ck, cv,
                                           torch.tensor([0, states[0], sum(states)], **I32), max_seqlen_q=K, err=err)
        if step % 7 == 0 or step == steps - 1:
            for b in range(B):
                for j in range(K):
                    y = emb[torch.tensor(hist[b][j], device=DEV)]
                    kk, vv = _np(y[:, Hq:Hq + Hkv]), _np(y[:, Hq + Hkv:])
                    if kind == "q4":
                        for z in (kk, vv):
                            for row in z.reshape(-1, d):
                                row[:] = so.q4_values(*so.q4_codes(row))
                    o, _, a, _ = bo.cross(_np(q[b * K + j][None]), kk, vv, 1 / math.sqrt(d))
                    # P in bf16 (4 bits: against value - minimum, at most twice), the output's rounding, scores
                    tol = 2.0 ** -8 * (3 if kind == "q4" else 1) * (a + 4) + 2.0 ** -8 * np.abs(o) + 2e-3
                    assert (np.abs(_np(mine[b * K + j]) - o[0]) <= tol[0]).all(), (step, b, j)
        s0 = 0
        for b, n_s in enumerate(states):
            o, _, a, _ = bo.cross(_np(q[b * K:(b + 1) * K]), _np(ck[s0:s0 + n_s]), _np(cv[s0:s0 + n_s]), 1 / math.sqrt(d))
            assert (np.abs(_np(theirs[b * K:(b + 1) * K]) - o) <= 2.0 ** -8 * (a + np.abs(o)) + 2e-3).all()
            s0 += n_s
        logits = ((mine + theirs).float().view(beams, -1) @ head).view(B, K, V)
    assert int(err) == 0
    assert len(seen_parents) > 5                         # beams did change places
