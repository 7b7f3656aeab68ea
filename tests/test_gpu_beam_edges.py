"""Cross attention and beam selection at their edges: batches on both sides of the ordered items' 32 sequences, many
heads to a kv head, guard words around outputs and workspace, scores that are not finite, scores replaced in place,
rows of logits past 32-bit offsets."""
import math

import numpy as np
import pytest
import torch

from test_gpu_beam import check_select
from test_gpu_cross import check, exact

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
I32 = dict(dtype=torch.int32, device=DEV)


def _cu(lens):
    return torch.tensor(np.cumsum([0] + list(lens)), **I32)


# B, rows of a sequence up to, keys up to, Hq, Hkv, d, dtype
BATCHES = [(32, 90, 300, 8, 2, 64, "bf16"), (33, 90, 300, 8, 2, 64, "bf16"), (45, 150, 700, 6, 2, 128, "bf16"),
           (2, 40, 900, 100, 1, 128, "bf16"), (3, 2, 4000, 128, 2, 64, "bf16"), (3, 1, 2600, 64, 1, 128, "f32"),
           (40, 6, 900, 12, 4, 64, "f32"), (40, 5, 3000, 12, 4, 128, "bf16")]


@pytest.mark.parametrize("B,T,S,Hq,Hkv,d,dtype", BATCHES)
@pytest.mark.parametrize("ranged", [False, True])
def test_padded_batches_between_guards(lib, B, T, S, Hq, Hkv, d, dtype, ranged):
    r = np.random.default_rng(B + S)
    rows, keys = r.integers(0, T + 1, B), r.integers(0, S + 1, B)
    rows[0], keys[0], rows[-1], keys[-1] = T, S, 1, 0            # the longest; a row without a key
    g = torch.Generator(device=DEV).manual_seed(B)
    n, pad = int(rows.sum()), 64
    q = torch.randn(n, Hq, d, generator=g, device=DEV).to(DT[dtype])
    k, v = (torch.randn(B * S, Hkv, d, generator=g, device=DEV).to(DT[dtype]) for _ in range(2))
    hidden = (torch.arange(S, device=DEV)[None] >= torch.tensor(keys, device=DEV)[:, None]).reshape(-1)
    k[hidden], v[hidden] = math.nan, math.inf
    ranges = None
    if ranged:
        lo = torch.randint(0, S, (n,), generator=g, device=DEV)
        ranges = torch.stack([lo, lo + torch.randint(0, S, (n,), generator=g, device=DEV)], -1).int().contiguous()
    spans = [(int(a), int(t), b * S, int(m)) for b, (a, t, m) in enumerate(zip(np.cumsum([0] + list(rows)), rows, keys))]
    if ranged:
        clipped = ranges.clone()
        for a, t, _, m in spans:
            clipped[a:a + t] = clipped[a:a + t].clamp(max=m)
    want = exact(q, k, v, spans, d ** -0.5, clipped if ranged else None)

    need = lib.cp_cross_attention_workspace_size(B, Hq, Hkv, d, T, S, total_q=n, total_kv=B * S, padded=True, dtype=DT[dtype])
    ws = torch.full((need + 2 * 256,), 0xa5, dtype=torch.uint8, device=DEV)
    out = torch.full((n + 2 * pad, Hq, d), 12345.0, dtype=DT[dtype], device=DEV)
    lse = torch.full((n + 2 * pad, Hq), 12345.0, device=DEV)
    err = torch.zeros(1, **I32)
    lib.cp_cross_attention(q, _cu(rows), k, v, _cu([S] * B), kv_lens=torch.tensor(keys, **I32), key_ranges=ranges,
                           max_seqlen_q=T, max_seqlen_kv=S, workspace=ws[256:256 + need], out=out[pad:pad + n],
                           out_lse=lse[pad:pad + n], err=err)
    assert int(err) == 0
    check(out[pad:pad + n], lse[pad:pad + n], want, dtype == "f32")
    mark = torch.tensor(12345.0, dtype=DT[dtype], device=DEV)
    for x, m in ((out, mark), (lse, 12345.0)):
        assert bool((x[:pad] == m).all()) and bool((x[pad + n:] == m).all())
    assert bool((ws[:256] == 0xa5).all()) and bool((ws[256 + need:] == 0xa5).all())


@pytest.mark.parametrize("T,Hq,d", [(5, 1, 128), (15, 1, 128), (9, 3, 64)])
def test_many_tiles_in_flight_on_every_sm(lib, T, Hq, d):
    """f32 under load: copies of consecutive tiles land in any order, and a warp takes only some of them."""
    B, S = 152, 2000
    g = torch.Generator(device=DEV).manual_seed(T)
    k, v = (torch.randn(B * S, 1, d, generator=g, device=DEV) for _ in range(2))
    q = torch.randn(B * T, Hq, d, generator=g, device=DEV)
    spans = [(b * T, T, b * S, S) for b in range(B)]
    for _ in range(3):
        out, lse = lib.cp_cross_attention(q, _cu([T] * B), k, v, _cu([S] * B), max_seqlen_q=T, max_seqlen_kv=S)
    check(out, lse, exact(q, k, v, spans, d ** -0.5), True)


# B, rows of a sequence up to, keys up to, Hq, Hkv, d: few items of many rows, whose parts meet in clusters
MEETING = [(1, 300, 2000, 2, 2, 64), (1, 1000, 1000, 6, 2, 64), (3, 200, 1500, 2, 2, 64), (2, 700, 2500, 4, 1, 128),
           (1, 2048, 3500, 2, 2, 128), (5, 40, 1200, 16, 2, 64), (4, 90, 260, 3, 1, 64), (1, 129, 700, 65, 1, 64)]


@pytest.mark.parametrize("B,T,S,Hq,Hkv,d", MEETING)
@pytest.mark.parametrize("padded", [False, True])
def test_parts_that_meet_in_clusters(lib, B, T, S, Hq, Hkv, d, padded):
    """Sequences that end inside a part, or hold no key of it; infinities and NaN behind a sequence's keys; twice the same."""
    r = np.random.default_rng(S)
    rows, keys = r.integers(0, T + 1, B), r.integers(0, S + 1, B)
    rows[0], keys[0], keys[-1] = T, S, (S if B == 1 else 3)
    held = np.full(B, S) if padded else keys
    g = torch.Generator(device=DEV).manual_seed(S)
    n = int(rows.sum())
    q = torch.randn(n, Hq, d, generator=g, device=DEV).bfloat16()
    k, v = (torch.randn(int(held.sum()), Hkv, d, generator=g, device=DEV).bfloat16() for _ in range(2))
    starts = np.cumsum([0] + list(held))
    for b in range(B):
        k[starts[b] + keys[b]:starts[b + 1]], v[starts[b] + keys[b]:starts[b + 1]] = math.nan, math.inf
    spans = [(int(a), int(t), int(s), int(m)) for a, t, s, m in zip(np.cumsum([0] + list(rows)), rows, starts, keys)]
    f = lambda: lib.cp_cross_attention(q, _cu(rows), k, v, _cu(held), kv_lens=torch.tensor(keys, **I32) if padded else None,
                                       max_seqlen_q=T, max_seqlen_kv=S)
    out, lse = f()
    check(out, lse, exact(q, k, v, spans, d ** -0.5), False)
    again = f()
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("T", [200, 3])
def test_a_visible_nan_in_one_part(lib, T):
    g = torch.Generator(device=DEV).manual_seed(T)
    q, k, v = (torch.randn(n, 2, 64, generator=g, device=DEV).bfloat16() for n in (T, 2000, 2000))
    v[1700, 0, 5], v[3, 1, 7] = math.nan, math.inf
    out, lse = lib.cp_cross_attention(q, _cu([T]), k, v, _cu([2000]), max_seqlen_q=T)
    assert bool(out[:, 0, 5].isnan().all()) and bool(out[:, 1, 7].isposinf().all()) and bool(lse.isfinite().all())
    v[1700, 0, 5] = v[3, 1, 7] = 0
    clean, _ = lib.cp_cross_attention(q, _cu([T]), k, v, _cu([2000]), max_seqlen_q=T)
    out[:, 0, 5], out[:, 1, 7] = clean[:, 0, 5], clean[:, 1, 7]
    assert torch.equal(out, clean)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scores_that_are_not_finite_and_scores_in_place(lib, dtype):
    g = torch.Generator(device=DEV).manual_seed(5)
    logits = (3 * torch.randn(4, 4, 5000, generator=g, device=DEV)).to(DT[dtype])
    scores = torch.tensor([[math.inf, -1.5, math.nan, -math.inf], [-2.0, -math.inf, -1.0, -1.25],
                           [math.inf, math.inf, math.nan, math.nan], [-3e38, -1.0, -3.4e38, -0.5]], device=DEV)
    got = lib.cp_beam_select(logits, scores, num_candidates=8, eos_token=17)
    for b in (0, 1, 2):
        check_select([x[b:b + 1] for x in got], logits[b:b + 1], scores[b:b + 1], 8, 17)
    assert set(got[4][3].tolist()) <= {1, 3}
    mine = scores.clone()
    again = lib.cp_beam_select(logits, mine, num_candidates=8, eos_token=17, next_scores=mine)
    assert again[0].data_ptr() == mine.data_ptr()
    for x, y in zip(got, again):
        assert torch.equal(x, y)


def test_rows_of_logits_past_32_bit_offsets(lib):
    K, V, stride = 3, 70001, 1_100_000_003                      # the last row starts behind 2^31 elements
    flat = torch.empty(2 * stride + V, dtype=torch.bfloat16, device=DEV)
    logits = flat.as_strided((1, K, V), (K * stride, stride, 1))
    small = (3 * torch.randn(1, K, V, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)).bfloat16()
    logits.copy_(small)
    scores = torch.tensor([[-4.0, -3.0, -1.0]], device=DEV)
    check_select(lib.cp_beam_select(logits, scores, eos_token=2), small, scores, 6, 2)


def test_calls_at_once_on_two_streams(lib):
    """Each kind of call in flight on one stream while the others run on another: the results of one after the other."""
    g = torch.Generator(device=DEV).manual_seed(9)
    normal = lambda *s: torch.randn(*s, generator=g, device=DEV)
    jobs = []
    for T, S, Hq, Hkv, d, dtype in [(300, 2000, 2, 2, 64, "bf16"), (1000, 3000, 8, 2, 128, "bf16"), (4, 1500, 8, 8, 64, "bf16"),
                                    (5, 1200, 4, 2, 128, "f32"), (8, 16384, 4, 1, 128, "bf16")]:
        q, k, v = (normal(n, h, d).to(DT[dtype]) for n, h in ((2 * T, Hq), (2 * S, Hkv), (2 * S, Hkv)))
        a = (q, _cu([T, T]), k, v, _cu([S, S]))
        jobs.append(lambda a=a, T=T, S=S: lib.cp_cross_attention(*a, max_seqlen_q=T, max_seqlen_kv=S))
    logits, scores = (3 * normal(6, 5, 50257)).bfloat16(), normal(6, 5)
    jobs.append(lambda: lib.cp_beam_select(logits, scores, eos_token=3))
    parents = torch.randint(0, 4, (3, 4), generator=g, device=DEV).int()
    tables, lens = torch.arange(12 * 3, **I32).reshape(1, 12, 3), torch.tensor([40, 16, 5], **I32)
    jobs.append(lambda: (lib.cp_beam_reorder(parents, lens, tables, tables, None, None, 1, 16, tables_out=torch.zeros_like(tables)),))
    want = [[x.clone() for x in f()] for f in jobs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for r in range(12):
        for i in range(len(jobs)):
            for n, s in enumerate(streams):
                at = (i + r + n * (1 + r % 5)) % len(jobs)
                with torch.cuda.stream(s):
                    got.append((at, jobs[at]()))
    torch.cuda.synchronize()
    for at, out in got:
        for x, y in zip(out, want[at]):
            assert torch.equal(x, y), at
