"""Memory that one part of a call, or one call, writes and another reads at once: results must not depend on
how the two fall together."""
import numpy as np
import pytest
import torch

from test_gpu_serving_large import DEV, DT, I32, _attend, _check, _cu, _fill, _pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,Hq,Hkv", [(128, 4, 2), (128, 8, 1), (64, 16, 1), (128, 16, 1)])
def test_q4_records_that_land_over_the_query_operands(lib, d, Hq, Hkv):
    """The last stage of a warp's ring first holds the query operands, and the first iteration already fills it
    with records: splits of a few iterations, 200 calls, each bit for bit the first, which is right."""
    lens = [1024, 640, 333]
    k, v, t, K, V = _fill(lib, lens, Hkv, d, 2, 8, torch.bfloat16, True, 11)
    q, sl = torch.randn(3, Hq, d, device=DEV).to(torch.bfloat16), torch.tensor(lens, **I32)
    ws = torch.zeros(lib.cp_decode_workspace_size(3, Hq, Hkv, d, 2, 1), dtype=torch.uint8, device=DEV)
    kw = dict(num_splits=1, split_tokens=768, workspace=ws)
    first = [x.clone() for x in lib.cp_decode_attention_q4(q, k, v, t, sl, 2, 8, **kw)]
    at = 0
    for b, n in enumerate(lens):
        one = torch.tensor([n - 1], device=DEV)
        o, l, a, big = _attend(q[b:b + 1].double(), K[at:at + n], V[at:at + n], 0 * one, one + 1, one, 0.0, None)
        _check(first[0][b:b + 1], first[1][b:b + 1], o, l, a, big, 0.0, None, n, extra=float(V.abs().max()), what=f"sequence {b}")
        at += n
    for _ in range(200):
        assert all(torch.equal(x, y) for x, y in zip(lib.cp_decode_attention_q4(q, k, v, t, sl, 2, 8, **kw), first))


@pytest.mark.parametrize("kind", ["f32", "f32_64", "bf16", "q4"])
def test_steps_that_rewrite_what_the_step_before_read(lib, kind):
    """Append, decode and merge of partials, step after step with nothing between them, over the same buffers: a
    kernel is placed while the ones before it run, some of which read the lines (queries, half-filled pages,
    partials) that the one just before it rewrites.  As with a synchronization after each call, bit for bit."""
    dt = DT["f32"] if kind.startswith("f32") else DT["bf16"]
    B, Hq, Hkv, d, cp, I, L, q4 = 4, 8, 2, 64 if kind == "f32_64" else 128, 2, 8, 60, kind == "q4"
    g = torch.Generator(device=DEV).manual_seed(9)
    x = torch.randn(L, B, Hq + 2 * Hkv, d, generator=g, device=DEV).to(dt)
    freq = torch.tensor(10000.0 ** (-np.arange(d // 2) / (d // 2)), device=DEV)
    cu1 = _cu([1] * B)
    at = [torch.full((B,), i, **I32) for i in range(L + 1)]
    fused, part = ((lib.cp_decode_attention_q4, lib.cp_partial_attn_decode_q4) if q4 else
                   (lib.cp_decode_attention_mod, lib.cp_partial_attn_decode_mod))
    results = []
    for wait in (True, False, False, False):
        k, v, t = _pool([L] * B, Hkv, d, cp, I, dt, q4, 1)
        k.zero_(), v.zero_()
        ws = torch.zeros(lib.cp_decode_workspace_size(B, Hq, Hkv, d, cp, 2), dtype=torch.uint8, device=DEV)
        q, out = (torch.zeros(B, Hq, d, dtype=dt, device=DEV) for _ in range(2))
        lse, po = torch.zeros(B, Hq, device=DEV), torch.zeros(2 * cp, B, Hq, d, device=DEV)
        pl = torch.zeros(2 * cp, B, Hq, device=DEV)
        seen = [[torch.empty(B, Hq, d, dtype=dt, device=DEV) for _ in range(2)] for _ in range(L)]
        torch.cuda.synchronize()

        def done():
            if wait:
                torch.cuda.synchronize()
        for i in range(L):
            qi, kn, vn = x[i].split([Hq, Hkv, Hkv], 1)
            lib.cp_rope_kv_cache_write(kn, vn, cu1, at[i], k, v, t, cp, I, inv_freq=freq, q=qi, q_out=q)
            done()
            kw = dict(num_splits=2, split_tokens=16)
            fused(q, k, v, t, at[i + 1], cp, I, workspace=ws, out=seen[i][0], out_lse=lse, **kw)
            done()
            part(q, k, v, t, at[i + 1], cp, I, out=po, lse=pl, **kw)
            done()
            lib.cp_lse_merge(po, pl, out=seen[i][1], out_dtype=dt)
            done()
        torch.cuda.synchronize()
        results.append(seen)
    for other in results[1:]:
        assert all(torch.equal(a, b) for x, y in zip(results[0], other) for a, b in zip(x, y))


def test_a_call_given_a_stream_allocates_and_reads_lengths_on_it(lib):
    """With stream= and the lengths still being written on that stream, a call that asks for the longest itself
    plans for what they become; a workspace and outputs made for the call are not memory that work still
    pending on the current stream uses."""
    B, L, Hq, Hkv, d, cp, I = 64, 600, 32, 8, 128, 2, 8
    s = torch.cuda.Stream()
    k, v, t, _, _ = _fill(lib, [L] * B, Hkv, d, cp, I, DT["bf16"], False, 2)
    q = torch.randn(B, Hq, d, device=DEV).to(torch.bfloat16)
    qp, kp, vp = (torch.randn(900, h, d, device=DEV).to(torch.bfloat16) for h in (8, 2, 2))
    lens, cu, zero = torch.full((B,), L, **I32), _cu([300, 600]), torch.zeros(B, **I32)
    out0 = _cu([L] * B)
    big = torch.randn(4096, 4096, device=DEV)

    def merged(partials, stream):
        return lib.cp_lse_merge(*partials, stream=stream)

    def attend(call, **plan):
        return lambda lens, cu, out0, kw: call(q, k, v, t, lens, cp, I, **plan, **kw)
    calls = [
        attend(lib.cp_decode_attention),
        attend(lib.cp_decode_attention, num_splits=5, split_tokens=64),        # a workspace's counters
        attend(lib.cp_decode_attention_mod),
        lambda lens, cu, out0, kw: merged(lib.cp_partial_attn_decode(q, k, v, t, lens, cp, I, **kw), kw["stream"]),
        lambda lens, cu, out0, kw: merged(lib.cp_partial_attn_decode_mod(q, k, v, t, lens, cp, I, **kw), kw["stream"]),
        lambda lens, cu, out0, kw: lib.cp_kv_cache_read(k, v, out0, zero, t, cp, I, **kw),
        lambda lens, cu, out0, kw: lib.cp_attn_prefill_mod(qp, cu, kp, vp, softcap=9.0, **kw),
        lambda lens, cu, out0, kw: lib.cp_attn_prefill_fused(qp, cu, 2, kp, vp, stream=kw["stream"]),
        lambda lens, cu, out0, kw: merged(lib.cp_partial_attn_prefill(qp, cu, 2, k=kp, v=vp, **kw), kw["stream"]),
    ]
    err = torch.zeros(1, **I32)
    late = [torch.zeros_like(x) for x in (lens, cu, out0)]
    for i, call in enumerate(calls):
        want = [x.clone() for x in call(lens, cu, out0, dict(err=err, stream=None))]
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            for x in late:
                x.zero_()
            for _ in range(20):
                big @ big
            for x, y in zip(late, (lens, cu, out0)):
                x.copy_(y)
        # blocks of the outputs' and the workspace's sizes, free again, that the busy current stream will still fill
        for _ in range(20):
            big @ big
        for n in {x.numel() * x.element_size() for x in want} | {lib.cp_decode_workspace_size(B, Hq, Hkv, d, cp, 5)}:
            for _ in range(3):
                torch.empty(n, dtype=torch.uint8, device=DEV).fill_(255)
        got = call(*late, dict(err=err, stream=s))
        torch.cuda.synchronize()
        assert int(err) == 0 and all(torch.equal(a, b) for a, b in zip(got, want)), i
