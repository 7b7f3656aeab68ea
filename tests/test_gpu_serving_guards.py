"""Guard regions around every output of the serving calls: each is a view into a larger buffer whose ends
hold a canary that must survive the call bit for bit; and inputs with nothing behind them but NaN."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
GUARD = 64          # elements on each side; keeps the view 128-byte aligned for 16- and 32-bit types
I32 = dict(dtype=torch.int32, device=DEV)
BITS = {1: torch.uint8, 2: torch.int16, 4: torch.int32}
CANARY = {1: 0xA5, 2: 0x7FAD, 4: 0x7FC0DEAD}    # NaNs, read as floats


class Guarded:
    def __init__(self, like):
        n, self.size = like.numel(), like.element_size()
        guard = GUARD * (4 // self.size)
        self.guard = guard
        self.buf = torch.empty(n + 2 * guard, dtype=like.dtype, device=DEV)
        self.bits = self.buf.view(BITS[self.size])
        self.bits.fill_(CANARY[self.size])
        self.view = self.buf[guard:guard + n].view(like.shape)
        self.view.copy_(like)

    def intact(self, what):
        want = CANARY[self.size]
        for x in (self.bits[:self.guard], self.bits[-self.guard:]):
            assert bool((x == want).all()), f"{what}: guard overwritten"


def _cu(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], **I32)


@pytest.mark.parametrize("d,dt,q4,cp,I", [(128, torch.bfloat16, False, 2, 8), (64, torch.bfloat16, True, 3, 5),
                                          (128, torch.float32, True, 1, 16), (64, torch.float32, False, 4, 8),
                                          (128, torch.bfloat16, True, 2, 8)])
def test_write_read_and_decode_stay_in_bounds(lib, d, dt, q4, cp, I):
    lens, Hq, Hkv = [37, 1, 100], 6, 2
    N, B = sum(lens), len(lens)
    blocks = [max(1, -(-(-(-n // (I * cp)) * I) // 16)) for n in lens]
    tables = torch.full((cp, B, max(blocks)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(blocks):
        tables[:, b, :n] = torch.arange(at, at + n, dtype=torch.int32)
        at += n
    tables = Guarded(tables.to(DEV)).view      # (behind the last entry: ids far outside the pool)
    pool = torch.zeros((cp, at, Hkv) + ((9 * d,) if q4 else (16, d)), dtype=torch.uint8 if q4 else dt, device=DEV)
    g = {n: Guarded(pool) for n in ("k_cache", "v_cache")}
    kn, vn = (Guarded(torch.randn(N, Hkv, d, device=DEV).to(dt)) for _ in range(2))
    q = Guarded(torch.randn(N, Hq, d, device=DEV).to(dt))
    g.update(q_out=Guarded(q.view), k_out=Guarded(kn.view))
    cu, zero = Guarded(_cu(lens)).view, Guarded(torch.zeros(B, **I32)).view
    freq = Guarded(torch.ones(d, **I32)).view.view(torch.float64)   # (any pattern: d / 2 doubles)
    freq.copy_(10000.0 ** (-torch.arange(d // 2, dtype=torch.float64) * 2 / d))
    lib.cp_rope_kv_cache_write(kn.view, vn.view, cu, zero, g["k_cache"].view, g["v_cache"].view, tables, cp, I, inv_freq=freq,
                               q=q.view, q_out=g["q_out"].view, k_out=g["k_out"].view)
    out = torch.bfloat16 if dt == torch.bfloat16 else torch.float32
    g.update(k_read=Guarded(kn.view.to(out)), v_read=Guarded(kn.view.to(out)))
    lib.cp_kv_cache_read(g["k_cache"].view, g["v_cache"].view, cu, zero, tables, cp, I, k_out=g["k_read"].view,
                         v_out=g["v_read"].view)
    qd = torch.bfloat16 if q4 else dt
    one = Guarded(torch.randn(B, Hq, d, device=DEV).to(qd))
    sl = Guarded(torch.tensor(lens, **I32)).view
    lse = torch.zeros(B, Hq, device=DEV)
    fused, part = ((lib.cp_decode_attention_q4, lib.cp_partial_attn_decode_q4) if q4 else
                   (lib.cp_decode_attention_mod, lib.cp_partial_attn_decode_mod))
    for S, tokens in ((1, 112), (2, 64), (5, 32)):
        ws = Guarded(torch.zeros(lib.cp_decode_workspace_size(B, Hq, Hkv, d, cp, S), dtype=torch.uint8, device=DEV))
        o, l = Guarded(one.view), Guarded(lse)
        po, pl = Guarded(torch.zeros(cp * S, B, Hq, d, device=DEV)), Guarded(torch.zeros(cp * S, B, Hq, device=DEV))
        kw = dict(num_splits=S, split_tokens=tokens, softcap=20.0)
        fused(one.view, g["k_cache"].view, g["v_cache"].view, tables, sl, cp, I, workspace=ws.view, out=o.view, out_lse=l.view, **kw)
        part(one.view, g["k_cache"].view, g["v_cache"].view, tables, sl, cp, I, out=po.view, lse=pl.view, **kw)
        torch.cuda.synchronize()
        for x, n in ((ws, "workspace"), (o, "out"), (l, "lse"), (po, "partial out"), (pl, "partial lse")):
            x.intact(f"{n}, {S} splits")
        assert bool(torch.isfinite(o.view.float()).all()) and bool(torch.isfinite(l.view).all())
    for n, x in g.items():
        x.intact(n)
        if n not in ("k_cache", "v_cache"):
            assert bool(torch.isfinite(x.view.float()).all()), n


@pytest.mark.parametrize("new,ctx,Hq,Hkv,d", [([129, 1, 300], [0, 77, 5], 4, 2, 128), ([257], [0], 3, 1, 64),
                                              ([5, 0, 400], [900, 3, 0], 6, 2, 128)])
def test_prefill_stays_in_bounds(lib, new, ctx, Hq, Hkv, d):
    tot = [a + b for a, b in zip(new, ctx)]
    q = Guarded(torch.randn(sum(new), Hq, d, device=DEV).to(torch.bfloat16))
    k, v = (Guarded(torch.randn(sum(tot), Hkv, d, device=DEV).to(torch.bfloat16)) for _ in range(2))
    start = Guarded(torch.tensor([0 if i % 7 else 1 << 20 for i in range(sum(new))], **I32)).view
    slopes = Guarded(torch.rand(Hq, device=DEV)).view
    for kw in ({}, dict(softcap=30.0), dict(softcap=30.0, kv_start=start), dict(alibi_slopes=slopes, window=100)):
        o, l = Guarded(q.view), Guarded(torch.zeros(sum(new), Hq, device=DEV))
        lib.cp_attn_prefill_mod(q.view, Guarded(_cu(new)).view, k.view, v.view, cu_seqlens_kv=Guarded(_cu(tot)).view,
                                max_seqlen_q=max(new), out=o.view, out_lse=l.view, **kw)
        torch.cuda.synchronize()
        o.intact("out"), l.intact("lse")
        assert bool(torch.isfinite(o.view.float()).all())
        assert not bool(torch.isnan(l.view).any()) and math.isfinite(float(l.view.amax()))


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 128), (3, 1, 64)])
def test_prefill_of_sequences_that_go_past_the_rows(lib, Hq, Hkv, d):
    """cu_seqlens that claim more rows than the tensors have: that sequence is reported and skipped, the ones
    before it are computed, and nothing behind the outputs' rows is written."""
    i32 = dict(dtype=torch.int32, device="cuda")
    q, k, v = (torch.randn(500, h, d, device="cuda").to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    cu = torch.tensor([0, 200, 400], **i32)
    want, want_lse = lib.cp_attn_prefill_mod(q[:400], cu, k[:400], v[:400], softcap=9.0)
    for cu_q, cu_kv, rows, err_want in (([0, 200, 400], None, 200, 5), ([0, 200, 400], [0, 200, 500], 200, 5),
                                        ([0, 200, 2 ** 31 - 1], None, 200, 5), ([-5, 200, 400], None, 0, 5)):
        buf, lbuf, err = torch.full((500, Hq, d), 9.0, device="cuda", dtype=torch.bfloat16), torch.full((500, Hq), 9.0, device="cuda"), torch.zeros(1, **i32)
        n = 400 if cu_kv else 300                   # rows given; the buffers behind them go on
        lib.cp_attn_prefill_mod(q[:n], torch.tensor(cu_q, **i32), k[:n], v[:n], softcap=9.0, max_seqlen_q=200, out=buf[:n], out_lse=lbuf[:n],
                                cu_seqlens_kv=torch.tensor(cu_kv, **i32) if cu_kv else None, err=err)
        assert int(err) == err_want
        if rows:
            assert torch.equal(buf[:rows], want[:rows]) and torch.equal(lbuf[:rows], want_lse[:rows])
        if cu_q[0] == 0:
            assert bool((buf[rows:] == 9.0).all()) and bool((lbuf[rows:] == 9.0).all())
        else:                                       # its second sequence ends at 400 of 300 rows: nothing is left
            assert bool((buf == 9.0).all())
