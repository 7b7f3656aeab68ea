"""Cross attention against the float64 oracle: few and many query rows, every dtype and head layout, padded batches,
key ranges, empty rows, strides, and everything outside a row's keys poisoned.

Tolerances are test_gpu_serving's, which derives them: a score is off by at most 2^-16 of scale sum |q||k| (sums of
128 products in fp32), the LSE by that, 2^-22 of itself and 1e-6; the output by 2 e |v|_avg, 2^-18 |v|_avg for fp32
sums over the keys and, in bf16, 2^-8 |v|_avg for P's rounding and 2^-8 |O| for the output's."""
import math

import numpy as np
import pytest
import torch

from oracle import beam_oracle as bo

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
I32 = dict(dtype=torch.int32, device=DEV)


def _np(t):
    return t.detach().double().cpu().numpy()


def _cu(lens):
    return torch.tensor(np.cumsum([0] + list(lens)), **I32)


def check(out, lse, want, f32, what=""):
    O, L, A, big = want
    fin = np.isfinite(L)
    if lse is not None:
        l = _np(lse)
        assert np.array_equal(np.isneginf(l), ~fin), f"{what}: rows without keys differ"
        e = 2.0 ** -16 * big + 2.0 ** -22 * np.where(fin, np.abs(L), 0) + 1e-6
        off = np.abs(np.where(fin, l - np.where(fin, L, 0), 0))
        assert (off <= e).all(), f"{what}: lse off by {off.max()}, {(off / e).max()} of its tolerance"
    e = 2.0 ** -16 * big + 1e-6
    tol = (2 * e[..., None] + 2.0 ** -18) * A + 1e-30
    if not f32:
        tol = tol + 2.0 ** -8 * A + 2.0 ** -8 * np.abs(O)
    o = _np(out)
    assert np.isfinite(o).all(), f"{what}: not finite"
    off = np.abs(o - O)
    assert (off <= tol).all(), f"{what}: out off by {off.max()}, {(off / tol).max()} of its tolerance"
    assert (o[~fin] == 0).all()


def exact(q, k, v, spans, scale, ranges=None):
    """Float64 on the GPU, for long sequences.  spans: per sequence (q0, T, k0, S)."""
    N, Hq, d = q.shape
    G = Hq // k.shape[1]
    O, A = (torch.zeros(N, Hq, d, dtype=torch.float64, device=DEV) for _ in range(2))
    L, big = torch.full((N, Hq), -math.inf, dtype=torch.float64, device=DEV), torch.zeros(N, Hq, dtype=torch.float64, device=DEV)
    for q0, T, k0, S in spans:
        if T == 0 or S == 0:
            continue
        for h in range(Hq):
            for a in range(q0, q0 + T, 2048):
                z = min(q0 + T, a + 2048)
                x, kk, vv = q[a:z, h].double(), k[k0:k0 + S, h // G].double(), v[k0:k0 + S, h // G].double()
                s, b = scale * x @ kk.T, scale * x.abs() @ kk.abs().T
                if ranges is not None:
                    j = torch.arange(S, device=DEV)
                    hide = (j < ranges[a:z, :1]) | (j >= ranges[a:z, 1:])
                    s, b = s.masked_fill(hide, -math.inf), b.masked_fill(hide, 0)
                L[a:z, h] = torch.logsumexp(s, -1)
                w = torch.exp(s - L[a:z, h].clamp(min=-1e300)[:, None])
                O[a:z, h], A[a:z, h], big[a:z, h] = w @ vv, w @ vv.abs(), b.amax(-1)
    return tuple(_np(x) for x in (O, L, A, big))


CASES = [
    # query rows, keys, Hq, Hkv, d, dtype
    ([1], [1], 1, 1, 64, "bf16"),
    ([4], [1500], 4, 4, 64, "bf16"),                     # a step of four beams
    ([4, 4, 4], [37, 0, 700], 8, 2, 128, "bf16"),        # 16 rows a kv head
    ([5, 5], [129, 64], 6, 1, 128, "bf16"),              # 30 rows: two row groups, the second in part
    ([3, 8], [65, 300], 16, 2, 64, "bf16"),              # 64 rows
    ([7, 1, 0, 2], [63, 200, 50, 1], 14, 2, 128, "bf16"),
    ([20, 3], [260, 128], 4, 2, 128, "bf16"),            # 40 rows
    ([65], [129], 1, 1, 128, "bf16"),                    # the first that goes to the big tiles
    ([130, 1, 0, 300], [200, 0, 77, 513], 6, 2, 64, "bf16"),   # G = 3: 42 tokens a tile
    ([100, 257], [1, 300], 8, 1, 128, "bf16"),
    ([33, 70], [640, 127], 10, 2, 128, "bf16"),          # G = 5
    ([2, 3], [90, 400], 128, 1, 64, "bf16"),             # 128 heads to a kv head: a token a tile
    ([3], [300], 65, 1, 64, "bf16"),
    ([5], [33], 4, 4, 64, "f32"),
    ([4, 0, 9], [100, 5, 31], 6, 2, 128, "f32"),
    ([40, 3], [65, 0], 8, 2, 64, "f32"),                 # several items of 16 rows
    ([2, 7], [1000, 1], 16, 1, 128, "f32"),              # G = 16
    ([1], [257], 3, 3, 128, "f32"),
]


@pytest.mark.parametrize("T,S,Hq,Hkv,d,dtype", CASES)
@pytest.mark.parametrize("form", ["plain", "padded", "ranges", "padded ranges"])
def test_against_the_oracle(lib, T, S, Hq, Hkv, d, dtype, form):
    r = np.random.default_rng(len(T) * 1000 + Hq + sum(S))
    f32, scale = dtype == "f32", 1 / math.sqrt(d)
    pad = max(S) + 3 if "padded" in form else 0
    rows = [pad or n for n in S]
    q = torch.tensor(r.normal(size=(sum(T), Hq, d)), dtype=DT[dtype])
    k, v = (torch.tensor(r.normal(size=(sum(rows) + 5, Hkv, d)), dtype=DT[dtype]) for _ in range(2))
    starts = np.cumsum([0] + rows)
    key = np.zeros(len(k), bool)
    for a, n in zip(starts, S):
        key[a:a + n] = True
    ranges = None
    if "ranges" in form:
        ranges = np.concatenate([np.sort(r.integers(-2, n + 3, size=(t, 2)), -1) for t, n in zip(T, S)])
        for i in r.integers(0, sum(T), max(1, sum(T) // 4)):     # rows without a key, rows of one, all keys
            ranges[i] = [(5, 5), (9, 2), (0, 1), (0, 10 ** 9), (-2 ** 31, 2 ** 31 - 1)][int(r.integers(5))]
        at = np.cumsum([0] + list(T))
    for x in (k, v):
        x[~torch.tensor(key)] = [math.nan, math.inf][x is v]
    want = [np.concatenate(x) for x in zip(*(
        bo.cross(_np(q[a:a + t]), _np(k[b:b + n]), _np(v[b:b + n]), scale, None if ranges is None else ranges[a:a + t])
        for a, t, b, n in zip(np.cumsum([0] + list(T)), T, starts, S)))]
    err = torch.zeros(1, **I32)
    out, lse = lib.cp_cross_attention(
        q.to(DEV), _cu(T), k.to(DEV), v.to(DEV), _cu(rows), kv_lens=torch.tensor(S, **I32) if pad else None,
        key_ranges=torch.tensor(ranges, **I32) if ranges is not None else None, max_seqlen_q=max(T),
        max_seqlen_kv=max(S), err=err)
    assert int(err) == 0
    check(out, lse, want, f32, form)


LONG = [
    # query rows, keys, Hq, Hkv, d, dtype
    ([4] * 64, [500 + 53 * i for i in range(64)], 32, 8, 128, "bf16"),
    ([8] * 3, [9000, 12345, 1], 16, 2, 128, "bf16"),      # 64 rows, parts through the workspace
    ([5], [16384], 2, 2, 64, "bf16"),
    ([1] * 200, [130] * 200, 4, 4, 64, "bf16"),
    ([2500], [3001], 16, 2, 128, "bf16"),                 # cut tail
    ([700, 2, 1300], [1500, 4000, 900], 12, 12, 64, "bf16"),
    ([64], [20000], 8, 1, 128, "bf16"),                   # four tiles of rows, cut into many parts
    ([5] * 8, [900, 1, 0, 450, 333, 800, 7, 64], 16, 16, 64, "f32"),
    ([3], [20011], 4, 1, 128, "f32"),                     # parts through the workspace
    ([300], [700], 4, 2, 64, "f32"),
]


@pytest.mark.parametrize("T,S,Hq,Hkv,d,dtype", LONG)
@pytest.mark.parametrize("cut", [True, False])
def test_long_and_many(lib, T, S, Hq, Hkv, d, dtype, cut):
    g = torch.Generator(device=DEV).manual_seed(sum(S))
    kv = torch.randn(sum(S), 2 * Hkv, d, generator=g, device=DEV).to(DT[dtype])      # columns of one projection
    k, v = kv.split([Hkv, Hkv], 1)
    q = torch.randn(sum(T), Hq + 2, d, generator=g, device=DEV).to(DT[dtype])[:, 1:Hq + 1]
    ws = None if cut else torch.empty(0, dtype=torch.uint8, device=DEV)
    out, lse = lib.cp_cross_attention(q, _cu(T), k, v, _cu(S), max_seqlen_q=max(T), max_seqlen_kv=max(S), workspace=ws)
    spans = list(zip(np.cumsum([0] + list(T)), T, np.cumsum([0] + list(S)), S))
    check(out, lse, exact(q, k, v, spans, 1 / math.sqrt(d)), dtype == "f32")


@pytest.mark.parametrize("d,Hq,Hkv,T", [(128, 8, 2, 900), (64, 16, 16, 400), (128, 32, 8, 2), (64, 6, 2, 12)])
def test_images_between_text(lib, d, Hq, Hkv, T):
    """Rows that see one image of several, the first rows none; infinities and NaN in images that a row does not see."""
    per, images = 333, 5
    g = torch.Generator(device=DEV).manual_seed(T)
    k, v = (torch.randn(per * images, Hkv, d, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(T, Hq, d, generator=g, device=DEV).to(torch.bfloat16)
    seen = torch.arange(T, device=DEV) * (images + 1) // T - 1          # -1: no image yet
    ranges = torch.stack([seen.clamp(min=0) * per, torch.where(seen < 0, 0, (seen + 1) * per)], -1).int().contiguous()
    want = exact(q, k, v, [(0, T, 0, per * images)], 1 / math.sqrt(d), ranges)
    hidden = [i for i in range(images) if not bool((seen == i).any())]
    for i in hidden:
        k[i * per:(i + 1) * per], v[i * per:(i + 1) * per] = math.nan, math.inf
    cu_q, cu_kv = _cu([T]), _cu([per * images])
    out, lse = lib.cp_cross_attention(q, cu_q, k, v, cu_kv, key_ranges=ranges, max_seqlen_q=T)
    check(out, lse, want, False)
    if not hidden:                                       # every image is seen by some: one of them goes bad
        bad = images // 2
        rows = seen == bad
        v[bad * per + 5, 0, 3] = math.inf
        v[bad * per + 7, Hkv - 1, 5] = math.nan
        o2, l2 = lib.cp_cross_attention(q, cu_q, k, v, cu_kv, key_ranges=ranges, max_seqlen_q=T)
        assert torch.equal(l2, lse)
        assert torch.equal(o2[~rows], out[~rows])
        G = Hq // Hkv
        assert bool(torch.isposinf(o2[rows][:, :G, 3]).all()) and bool(o2[rows][:, -G:, 5].isnan().all())
        o2[rows, :G, 3], o2[rows, -G:, 5] = out[rows, :G, 3], out[rows, -G:, 5]
        assert torch.equal(o2, out)


@pytest.mark.parametrize("T", [3, 200])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_visible_infinity_or_nan_is_not_hidden(lib, T, dtype):
    q = torch.ones(T, 2, 64, device=DEV).to(DT[dtype])
    k = torch.ones(150, 2, 64, device=DEV).to(DT[dtype])
    v = torch.ones(150, 2, 64, device=DEV).to(DT[dtype])
    v[140, 0, 1], v[3, 1, 2] = math.inf, math.nan
    out, lse = lib.cp_cross_attention(q, _cu([T]), k, v, _cu([150]), max_seqlen_q=T)
    assert bool(torch.isposinf(out[:, 0, 1]).all()) and bool(out[:, 1, 2].isnan().all())
    out[:, 0, 1], out[:, 1, 2] = 1, 1
    assert bool(((out.float() - 1).abs() <= 2.0 ** -7).all()) and bool(torch.isfinite(lse).all())
    k[5] = math.nan                                       # a key that is NaN: the rows and their LSEs are
    out, lse = lib.cp_cross_attention(q, _cu([T]), k, v, _cu([150]), max_seqlen_q=T)
    assert bool(out.isnan().all()) and bool(lse.isnan().all())


@pytest.mark.parametrize("T,dtype", [(1, "bf16"), (1, "f32"), (16, "bf16"), (200, "bf16")])
def test_scores_that_climb_and_fall_far(lib, T, dtype):
    """Scores from -400 to 400 nats along the keys, up and down: the reference moves all the way, or stays."""
    d, S = 64, 777
    for sign in (1, -1):
        q = torch.zeros(T, 1, d, device=DEV)
        q[..., 0] = 8
        k = torch.zeros(S, 1, d, device=DEV)
        k[:, 0, 0] = sign * torch.linspace(-400, 400, S, device=DEV).to(torch.bfloat16).float()
        v = torch.randn(S, 1, d, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
        q, k, v = (x.to(DT[dtype]) for x in (q, k, v))
        out, lse = lib.cp_cross_attention(q, _cu([T]), k, v, _cu([S]), max_seqlen_q=T)
        check(out, lse, exact(q, k, v, [(0, T, 0, S)], 1 / math.sqrt(d)), dtype == "f32")


def test_given_scale_and_no_lse(lib):
    q, k, v = (torch.randn(n, 2, 64, device=DEV).to(torch.bfloat16) for n in (70, 300, 300))
    out, lse = lib.cp_cross_attention(q, _cu([70]), k, v, _cu([300]), softmax_scale=0.3, want_lse=False)
    assert lse is None
    check(out, None, exact(q, k, v, [(0, 70, 0, 300)], float(np.float32(0.3))), False)


@pytest.mark.parametrize("T,dtype", [(4, "bf16"), (4, "f32"), (150, "bf16")])
def test_rows_behind_the_last_sequence_and_sequences_that_go_past_the_rows(lib, T, dtype):
    dt = DT[dtype]
    q, k, v = (torch.randn(n, 4, 64, device=DEV).to(dt) for n in (2 * T + 7, 500, 500))
    ref, rl = lib.cp_cross_attention(q[:2 * T].contiguous(), _cu([T, T]), k, v, _cu([300, 200]), max_seqlen_q=T)
    out, lse = torch.full_like(q, 7), torch.full((2 * T + 7, 4), 7.0, device=DEV)
    err = torch.zeros(1, **I32)
    kw = dict(out=out, out_lse=lse, err=err)
    lib.cp_cross_attention(q, _cu([T, T]), k, v, _cu([300, 200]), max_seqlen_q=T, **kw)
    assert int(err) == 0 and torch.equal(out[:2 * T], ref) and torch.equal(lse[:2 * T], rl)
    assert bool((out[2 * T:] == 7).all()) and bool((lse[2 * T:] == 7).all())
    bad = [
        (torch.tensor([0, T, 5 * T + 9], **I32), _cu([300, 200]), None, T, [1, 0]),   # more query rows than there are
        (_cu([T, T]), torch.tensor([0, 300, 501], **I32), None, T, [1, 0]),           # more keys
        (torch.tensor([0, T, T - 1], **I32), _cu([300, 200]), None, T, [1, 0]),       # a negative length
        (_cu([T, T]), torch.tensor([0, 300, 10], **I32), None, T, [1, 0]),
        (torch.tensor([-3, T, 2 * T], **I32), _cu([300, 200]), None, T + 3, [0, 1]),
        (_cu([T, T]), torch.tensor([-1, 300, 500], **I32), None, T, [0, 1]),
        (_cu([T, T]), _cu([300, 200]), [300, 201], T, [1, 1]),                        # kv_lens: the nearest
        (_cu([T, T]), _cu([300, 200]), [300, -5], T, [1, 2]),
        (_cu([T, T]), _cu([300, 200]), None, T - 1, [3, 3]),                          # max_seqlen_q: the rest is left out
    ]
    for cu_q, cu_kv, lens, most, ok in bad:
        out.fill_(7), lse.fill_(7), err.zero_()
        lib.cp_cross_attention(q, cu_q, k, v, cu_kv, kv_lens=None if lens is None else torch.tensor(lens, **I32),
                               max_seqlen_q=most, **kw)
        assert int(err) == 5
        for b, state in enumerate(ok):
            o, l, a, z = out[b * T:(b + 1) * T], lse[b * T:(b + 1) * T], ref[b * T:(b + 1) * T], rl[b * T:(b + 1) * T]
            if state == 1:
                assert torch.allclose(o.float(), a.float(), atol=2.0 ** -6) and torch.allclose(l, z, atol=1e-4)
            elif state == 0:
                assert bool((o == 7).all()) and bool((l == 7).all())
            elif state == 2:
                assert bool((o == 0).all()) and bool(l.isneginf().all())
            else:
                assert torch.allclose(o[:-1].float(), a[:-1].float(), atol=2.0 ** -6) and bool((o[-1:] == 7).all())
        assert bool((out[2 * T:] == 7).all())


def test_no_rows_no_keys_and_empty_tensors(lib):
    q, k = torch.randn(6, 4, 64, device=DEV).to(torch.bfloat16), torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    for x in (q, q.float(), q.repeat(40, 1, 1)):
        out, lse = lib.cp_cross_attention(x, _cu([len(x)]), k.to(x.dtype), k.to(x.dtype), _cu([0]))
        assert bool((out == 0).all()) and bool(lse.isneginf().all())
        out, lse = lib.cp_cross_attention(x[:0], _cu([0]), x[:, :2].contiguous(), x[:, :2].contiguous(), _cu([len(x)]))
        assert out.shape == (0, 4, 64) and lse.shape == (0, 4)


@pytest.mark.parametrize("T,S,Hq,Hkv,d,dtype", [(4, 16384, 4, 1, 128, "bf16"), (1000, 3000, 8, 2, 64, "bf16"),
                                                (3, 9000, 2, 1, 64, "f32"), (8, 500, 16, 2, 128, "bf16")])
def test_in_a_graph_on_another_stream_and_twice_the_same(lib, T, S, Hq, Hkv, d, dtype):
    q, k, v = (torch.randn(n, h, d, device=DEV).to(DT[dtype]) for n, h in ((T, Hq), (S, Hkv), (S, Hkv)))
    cu_q, cu_kv = _cu([T]), _cu([S])
    size = lib.cp_cross_attention_workspace_size(1, Hq, Hkv, d, T, S, dtype=DT[dtype])
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    kw = dict(max_seqlen_q=T, max_seqlen_kv=S, workspace=ws)
    ref, rl = lib.cp_cross_attention(q, cu_q, k, v, cu_kv, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, b = lib.cp_cross_attention(q, cu_q, k, v, cu_kv, stream=side, max_seqlen_q=T, max_seqlen_kv=S)
    side.synchronize()
    assert torch.equal(a, ref) and torch.equal(b, rl)
    out, lse = torch.empty_like(ref), torch.empty_like(rl)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.cp_cross_attention(q, cu_q, k, v, cu_kv, out=out, out_lse=lse, **kw)
    for _ in range(3):
        q.copy_(torch.randn_like(q, dtype=torch.float32))
        graph.replay()
        ref, rl = lib.cp_cross_attention(q, cu_q, k, v, cu_kv, max_seqlen_q=T, max_seqlen_kv=S)
        assert torch.equal(out, ref) and torch.equal(lse, rl)


def test_rows_past_32_bit_offsets(lib):
    """k and v as columns of rows so wide that the last keys lie past 2^32 bytes."""
    S, wide, d = 4100, 1024 * 1024 // 2, 64
    kv = torch.empty(S, wide, dtype=torch.bfloat16, device=DEV)
    k = kv[:, 128:128 + 2 * d].view(S, 2, d)
    v = kv[:, wide - 2 * d:].view(S, 2, d)
    k.copy_(torch.randn(S, 2, d, device=DEV)), v.copy_(torch.randn(S, 2, d, device=DEV))
    for T in (3, 90):
        q = torch.randn(T, 4, d, device=DEV).to(torch.bfloat16)
        out, lse = lib.cp_cross_attention(q, _cu([T]), k, v, _cu([S]), max_seqlen_q=T)
        check(out, lse, exact(q, k, v, [(0, T, 0, S)], 1 / math.sqrt(d)), False)
