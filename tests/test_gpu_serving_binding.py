"""What the serving calls' Python binding refuses, and how it treats outputs, streams and defaults."""
import pytest
import torch

import context_gqa_attention_gb300 as cpa

pytestmark = pytest.mark.gpu
DEV = "cuda"
B, Hq, Hkv, d, cp, I, POOL, BLOCKS, N = 2, 4, 2, 64, 2, 8, 12, 5, 6


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _bf(*shape):
    return torch.randn(*shape, device=DEV).to(torch.bfloat16)


@pytest.fixture
def t():
    tables = torch.arange(cp * B * BLOCKS, dtype=torch.int32, device=DEV).reshape(cp, B, BLOCKS) % POOL
    return dict(kc=_bf(cp, POOL, Hkv, 16, d), vc=_bf(cp, POOL, Hkv, 16, d), tables=tables, q=_bf(B, Hq, d),
                k4=torch.zeros(cp, POOL, Hkv, 9 * d, dtype=torch.uint8, device=DEV),
                v4=torch.zeros(cp, POOL, Hkv, 9 * d, dtype=torch.uint8, device=DEV),
                sl=_i32(40, 17), cu=_i32(0, 4, 6), start=_i32(3, 9), kn=_bf(N, Hkv, d), vn=_bf(N, Hkv, d), qn=_bf(N, Hq, d),
                freq=torch.ones(d // 2, dtype=torch.float64, device=DEV))


def write(t, **kw):
    a = {**t, **kw}
    rest = {k: v for k, v in kw.items() if k not in t}
    return cpa.cp_rope_kv_cache_write(a["kn"], a["vn"], a["cu"], a["start"], a["kc"], a["vc"], a["tables"],
                                      a.get("cp", cp), I, inv_freq=a["freq"], q=a["qn"],
                                      **{k: v for k, v in rest.items() if k != "cp"})


def read(t, **kw):
    a = {**t, **kw}
    rest = {k: v for k, v in kw.items() if k not in t}
    return cpa.cp_kv_cache_read(a["kc"], a["vc"], a["cu"], a["start"], a["tables"], cp, I, **{"total": N, **rest})


def decode(t, **kw):
    a = {**t, **kw}
    rest = {k: v for k, v in kw.items() if k not in t}
    return cpa.cp_decode_attention_mod(a["q"], a["kc"], a["vc"], a["tables"], a["sl"], cp, I, **rest)


def partial(t, **kw):
    a = {**t, **kw}
    rest = {k: v for k, v in kw.items() if k not in t}
    return cpa.cp_partial_attn_decode_mod(a["q"], a["kc"], a["vc"], a["tables"], a["sl"], cp, I, **rest)


def decode4(t, **kw):
    a = {**t, **kw}
    rest = {k: v for k, v in kw.items() if k not in t}
    return cpa.cp_decode_attention_q4(a["q"], a["k4"], a["v4"], a["tables"], a["sl"], cp, I, **rest)


def prefill(t, **kw):
    a = {**t, **kw}
    rest = {k: v for k, v in kw.items() if k not in t}
    return cpa.cp_attn_prefill_mod(a["qn"], a["cu"], a["kn"], a["vn"], **rest)


F32 = torch.float32
REFUSED = [
    (write, lambda t: dict(kn=t["kn"].cpu())),
    (write, lambda t: dict(vn=t["vn"].cpu())),
    (write, lambda t: dict(vn=t["vn"].float())),
    (write, lambda t: dict(vn=t["vn"][:5])),
    (write, lambda t: dict(kn=t["kn"].transpose(0, 1).contiguous().transpose(0, 1))),     # heads not dense
    (write, lambda t: dict(kn=t["kn"][0])),
    (write, lambda t: dict(kn=t["kn"].half(), vn=t["vn"].half(), qn=t["qn"].half(), kc=t["kc"].half(), vc=t["vc"].half())),
    (write, lambda t: dict(qn=t["qn"].float())),
    (write, lambda t: dict(cu=t["cu"].long())),
    (write, lambda t: dict(start=t["start"][:1])),
    (write, lambda t: dict(tables=t["tables"][:1])),
    (write, lambda t: dict(tables=t["tables"].transpose(0, 1))),
    (write, lambda t: dict(kc=t["kc"].float())),
    (write, lambda t: dict(vc=t["vc"][:, :4])),
    (write, lambda t: dict(vc=t["vc"][:, :4].contiguous())),
    (write, lambda t: dict(cp=3)),
    (write, lambda t: dict(cp=1 << 40)),
    (write, lambda t: dict(freq=t["freq"].float())),
    (write, lambda t: dict(freq=torch.ones(5, dtype=torch.float64, device=DEV))),         # 10 rotated dims
    (write, lambda t: dict(freq=torch.ones(40, dtype=torch.float64, device=DEV))),        # more than the head has
    (write, lambda t: dict(q_out=t["qn"].float())),
    (write, lambda t: dict(q_out=t["qn"][:5])),
    (write, lambda t: dict(qn=None, q_out=t["qn"])),
    (write, lambda t: dict(k_out=t["kn"][:5])),
    (write, lambda t: dict(err=torch.zeros(1, device=DEV))),
    (write, lambda t: dict(err=torch.zeros(0, dtype=torch.int32, device=DEV))),
    (write, lambda t: dict(rope_style=2)),
    (write, lambda t: dict(kn=torch.zeros(N * Hkv * d + 4, dtype=torch.bfloat16, device=DEV)[4:].view(N, Hkv, d))),
    (read, lambda t: dict(out_dtype=F32)),
    (read, lambda t: dict(out_dtype=torch.float16)),
    (read, lambda t: dict(k_out=t["kn"][:5])),
    (read, lambda t: dict(v_out=t["vn"].float())),
    (read, lambda t: dict(kc=t["kc"].cpu(), total=None)),
    (read, lambda t: dict(cu=t["cu"].cpu())),
    (read, lambda t: dict(total=1 << 33)),
    (read, lambda t: dict(kc=t["kc"].reshape(cp, POOL, Hkv * 16, d))),
    (read, lambda t: dict(vc=t["v4"])),
    (decode, lambda t: dict(q=t["q"].float())),
    (decode, lambda t: dict(q=t["q"].half())),
    (decode, lambda t: dict(q=t["q"][0])),
    (decode, lambda t: dict(q=t["q"].transpose(0, 1).contiguous().transpose(0, 1))),
    (decode, lambda t: dict(q=torch.cat([t["q"], t["q"][:, :1]], 1))),                    # 5 heads over 2
    (decode, lambda t: dict(kc=t["k4"], vc=t["v4"])),
    (decode, lambda t: dict(sl=t["sl"][:1])),
    (decode, lambda t: dict(sl=t["sl"].long())),
    (decode, lambda t: dict(alibi_slopes=torch.ones(Hkv, device=DEV))),
    (decode, lambda t: dict(alibi_slopes=torch.ones(Hq))),
    (decode, lambda t: dict(kv_start=_i32(0))),
    (decode, lambda t: dict(softcap=-1.0)),
    (decode, lambda t: dict(softcap=float("nan"))),
    (decode, lambda t: dict(window=-1)),
    (decode, lambda t: dict(num_splits=0, split_tokens=16)),
    (decode, lambda t: dict(num_splits=129, split_tokens=16)),                            # 258 parts
    (decode, lambda t: dict(num_splits=1, split_tokens=15)),
    (decode, lambda t: dict(workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))),
    (decode, lambda t: dict(workspace=torch.zeros(1 << 20, device=DEV))),
    (decode, lambda t: dict(out=t["q"].float())),
    (decode, lambda t: dict(out=t["q"][:1])),
    (decode, lambda t: dict(out_lse=torch.zeros(Hq, B, device=DEV))),
    (partial, lambda t: dict(num_splits=2, split_tokens=16, out=torch.zeros(2, B, Hq, d, device=DEV))),
    (partial, lambda t: dict(num_splits=-1, split_tokens=16)),
    (decode4, lambda t: dict(k4=t["kc"], v4=t["vc"])),
    (decode4, lambda t: dict(q=t["q"].float())),
    (decode4, lambda t: dict(k4=t["k4"][..., :500].contiguous(), v4=t["v4"][..., :500].contiguous())),
    (prefill, lambda t: dict(qn=t["qn"].float())),
    (prefill, lambda t: dict(qn=t["qn"].cpu())),
    (prefill, lambda t: dict(kn=t["kn"][:5], vn=t["vn"][:5])),
    (prefill, lambda t: dict(vn=t["vn"][:5])),
    (prefill, lambda t: dict(kn=t["kn"][..., :32].contiguous(), vn=t["vn"][..., :32].contiguous())),
    (prefill, lambda t: dict(cu_seqlens_kv=_i32(0, 4))),
    (prefill, lambda t: dict(kv_start=_i32(0, 0))),
    (prefill, lambda t: dict(prefix_lens=_i32(0))),
    (prefill, lambda t: dict(out_lse=torch.zeros(N, Hkv, device=DEV))),
    (prefill, lambda t: dict(alibi_slopes=torch.ones(Hq, dtype=torch.bfloat16, device=DEV))),
    (prefill, lambda t: dict(softcap=1e-9)),
]


@pytest.mark.parametrize("i", range(len(REFUSED)))
def test_refusals(lib, t, i):
    call, bad = REFUSED[i]
    call(t)                      # as it is, the call is taken
    kept = {n: x.clone() for n, x in t.items()}
    with pytest.raises(cpa.CPError) as e:
        call(t, **bad(t))
    assert e.value.status in (1, 2) and e.value.detail
    torch.cuda.synchronize()
    assert all(torch.equal(kept[n], t[n]) for n in kept)


def test_wrong_kinds_of_arguments_raise(lib, t):
    for call, bad in ((write, dict(kn=3)), (decode, dict(q="q")), (decode, dict(sl=None)), (decode, dict(softcap="x")),
                      (read, dict(total="x")), (prefill, dict(window=1.5)), (decode4, dict(k4=[1]))):
        with pytest.raises((cpa.CPError, TypeError, AttributeError)):
            call(t, **bad)


def test_outputs_given_are_the_ones_returned(lib, t):
    q_out, k_out = torch.empty_like(t["qn"]), torch.empty_like(t["kn"])
    a, b = write(t, q_out=q_out, k_out=k_out)
    assert a is q_out and b is k_out
    assert write(t)[1] is None and write(t, qn=None) == (None, None)
    assert torch.equal(write(t)[0], q_out)
    ko, vo = torch.empty_like(t["kn"]), torch.empty_like(t["vn"])
    a, b = read(t, k_out=ko, v_out=vo, total=None)
    assert a is ko and b is vo and torch.equal(read(t)[0], ko) and torch.equal(read(t, total=None)[1], vo)
    for call in (decode, decode4):
        out, lse = torch.empty_like(t["q"]), torch.empty(B, Hq, device=DEV)
        a, b = call(t, out=out, out_lse=lse)
        assert a is out and b is lse
        want = call(t)
        assert torch.equal(want[0], out) and torch.equal(want[1], lse)
        a, b = call(t, want_lse=False)
        assert b is None and torch.equal(a, out)
    po, pl = partial(t, num_splits=2, split_tokens=16)
    assert po.shape == (2 * cp, B, Hq, d) and pl.shape == (2 * cp, B, Hq)
    out, lse = torch.empty_like(t["qn"]), torch.empty(N, Hq, device=DEV)
    a, b = prefill(t, out=out, out_lse=lse)
    assert a is out and b is lse and torch.equal(prefill(t)[0], out)


def test_references_are_not_lost_or_kept(lib, t):
    """Returned outputs are owned by the caller alone; refused calls keep nothing."""
    import gc
    import sys
    out = torch.empty_like(t["q"])
    before = [sys.getrefcount(x) for x in (*t.values(), out, None)][:-1]
    for _ in range(5):
        decode(t, out=out)
        write(t)
        with pytest.raises(cpa.CPError):
            decode(t, out=out, window=-1)
    assert [sys.getrefcount(x) for x in (*t.values(), out, None)][:-1] == before
    torch.cuda.synchronize()
    gc.collect()                # (what earlier tests left to the collector is not this one's)
    used = torch.cuda.memory_allocated()
    for _ in range(10):
        decode(t)
        prefill(t)
    assert torch.cuda.memory_allocated() == used


def test_the_stream_given_is_the_one_used(lib, t):
    """A call with stream= waits for that stream's work, and one within a stream context for its."""
    s = torch.cuda.Stream()
    want = decode(t)[0].clone()
    q = torch.zeros_like(t["q"])
    torch.cuda.synchronize()
    out = torch.empty_like(q)
    big = torch.randn(4096, 4096, device=DEV)
    for how in ("argument", "context"):
        q.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            for _ in range(20):
                big @ big
            q.copy_(t["q"])
            if how == "context":
                decode(t, q=q, out=out)
        if how == "argument":
            decode(t, q=q, out=out, stream=s, workspace=torch.zeros(1 << 20, dtype=torch.uint8, device=DEV), num_splits=1,
                   split_tokens=32)
        s.synchronize()
        torch.cuda.synchronize()
        assert float((out.float() - want.float()).abs().max()) <= 2.0 ** -7 * float(want.float().abs().max())


def test_a_workspace_made_for_a_stream_is_filled_on_it(lib):
    """Without a workspace the call zero-fills one on the stream it runs on, whatever the current one does."""
    B, L, s = 64, 600, torch.cuda.Stream()
    pages = -(-L // 32)
    kc, vc = (_bf(cp, B * pages, 8, 16, d) for _ in range(2))
    tables = torch.arange(B * pages, dtype=torch.int32, device=DEV).reshape(1, B, pages).repeat(cp, 1, 1)
    q, sl = _bf(B, 32, d), torch.full((B,), L, dtype=torch.int32, device=DEV)
    kw = dict(num_splits=5, split_tokens=64)        # more CTAs than run at once: merged through the counters
    want = cpa.cp_decode_attention_mod(q, kc, vc, tables, sl, cp, I, **kw)[0].clone()
    need = cpa.cp_decode_workspace_size(B, 32, 8, d, cp, 5)
    big = torch.randn(4096, 4096, device=DEV)
    out, lse = torch.empty_like(want), torch.empty(B, 32, device=DEV)
    torch.cuda.synchronize()
    for how in (None, s):
        dirty = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        del dirty                                   # the next block of this size holds its bytes
        for _ in range(20):
            big @ big                               # the current stream is busy
        cpa.cp_decode_attention_mod(q, kc, vc, tables, sl, cp, I, stream=how, out=out, out_lse=lse, **kw)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        out.zero_()


def test_inference_mode_and_leaves_that_want_gradients(lib, t):
    want = decode(t)[0]
    with torch.inference_mode():
        assert torch.equal(decode(t)[0], want)
    q = t["q"].clone().requires_grad_()
    got = decode(t, q=q)[0]
    assert torch.equal(got, want) and not got.requires_grad


def test_prefill_told_that_no_sequence_has_rows(lib):
    """max_seqlen_q = 0: a sequence longer than what one tile row holds is reported, rows of a padded batch whose
    sequences are all empty are left as they are, and nothing is reported for those."""
    for Hq, Hkv in ((4, 2), (3, 1)):
        i32 = dict(dtype=torch.int32, device="cuda")
        q, k, v = (torch.randn(700, h, 64, device="cuda").to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
        cu = torch.tensor([0, 100, 700], **i32)
        want, want_lse = lib.cp_attn_prefill_mod(q, cu, k, v, max_seqlen_q=600)
        err, out, lse = torch.zeros(1, **i32), torch.full_like(want, 9.0), torch.full_like(want_lse, 9.0)
        lib.cp_attn_prefill_mod(q, cu, k, v, max_seqlen_q=0, out=out, out_lse=lse, err=err)
        assert int(err) == 5 and torch.equal(out[:100], want[:100]) and torch.equal(lse[:100], want_lse[:100])
        out.fill_(9.0), lse.fill_(9.0), err.zero_()
        lib.cp_attn_prefill_mod(q, torch.zeros(3, **i32), k, v, out=out, out_lse=lse, err=err)
        assert int(err) == 0 and bool((out == 9.0).all()) and bool((lse == 9.0).all())
