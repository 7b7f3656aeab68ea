"""What the Python entry points of cross attention, beam selection and reordering refuse, return and keep."""
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _bf(*shape):
    return torch.randn(*shape, device=DEV).to(torch.bfloat16)


def cross(lib, **kw):
    a = dict(q=_bf(6, 4, 64), cu_q=_i32(0, 2, 6), k=_bf(9, 2, 64), v=_bf(9, 2, 64), cu_kv=_i32(0, 4, 9))
    a.update({n: kw.pop(n) for n in list(kw) if n in a})
    return lib.cp_cross_attention(a["q"], a["cu_q"], a["k"], a["v"], a["cu_kv"], **kw)


def select(lib, **kw):
    a = dict(logits=torch.randn(2, 3, 50, device=DEV), scores=torch.zeros(2, 3, device=DEV))
    a.update({n: kw.pop(n) for n in list(kw) if n in a})
    return lib.cp_beam_select(a["logits"], a["scores"], **kw)


def reorder(lib, **kw):
    t = torch.arange(2 * 6 * 4, dtype=torch.int32, device=DEV).view(2, 6, 4) % 24
    a = dict(parents=torch.zeros(2, 3, dtype=torch.int32, device=DEV), seq_lens=_i32(5, 9), tables=t, own=t.clone(),
             k=_bf(2, 24, 2, 16, 64), v=_bf(2, 24, 2, 16, 64), cp=2, I=8)
    a.update({n: kw.pop(n) for n in list(kw) if n in a})
    return lib.cp_beam_reorder(a["parents"], a["seq_lens"], a["tables"], a["own"], a["k"], a["v"], a["cp"], a["I"], **kw)


BAD = [
    (cross, lambda: dict(q=torch.randn(6, 4, 64)), 1), (cross, lambda: dict(q=_bf(6, 256)), 1),
    (cross, lambda: dict(k=torch.randn(9, 2, 64, device=DEV)), 1), (cross, lambda: dict(k=_bf(9, 2, 128)), 1),
    (cross, lambda: dict(v=_bf(8, 2, 64)), 1), (cross, lambda: dict(q=_bf(6, 4, 64).half()), 1),
    (cross, lambda: dict(q=_bf(6, 4, 96), k=_bf(9, 2, 96), v=_bf(9, 2, 96)), 2),
    (cross, lambda: dict(q=_bf(6, 3, 64)), 1), (cross, lambda: dict(cu_kv=_i32(0, 9)), 1),
    (cross, lambda: dict(cu_q=torch.tensor([0, 2, 6], device=DEV)), 1), (cross, lambda: dict(kv_lens=_i32(1)), 1),
    (cross, lambda: dict(key_ranges=_i32(1, 2)), 1), (cross, lambda: dict(out=_bf(6, 4, 128)), 1),
    (cross, lambda: dict(out=torch.empty(6, 4, 64, device=DEV)), 1), (cross, lambda: dict(out_lse=_bf(6, 4)), 1),
    (cross, lambda: dict(workspace=_bf(64)), 1), (cross, lambda: dict(err=torch.zeros(1, device=DEV)), 1),
    (cross, lambda: dict(k=_bf(9, 64, 2).transpose(1, 2)), 1), (cross, lambda: dict(k=_bf(9, 2, 65)[..., :64]), 1),
    (cross, lambda: dict(q=_bf(6, 257)[:, 1:].view(6, 4, 64)), 1), (cross, lambda: dict(max_seqlen_q=-1), 1),
    (cross, lambda: dict(kv_lens=torch.tensor([1, 2], dtype=torch.int32)), 1),
    (select, lambda: dict(logits=torch.randn(2, 3, 50)), 1), (select, lambda: dict(logits=torch.randn(6, 50, device=DEV)), 1),
    (select, lambda: dict(logits=torch.randn(2, 3, 50, device=DEV).half()), 2),
    (select, lambda: dict(logits=torch.randn(2, 50, 3, device=DEV).transpose(1, 2)), 1),
    (select, lambda: dict(logits=torch.randn(2, 4, 50, device=DEV)[:, :3]), 1),
    (select, lambda: dict(scores=torch.zeros(2, 4, device=DEV)), 1), (select, lambda: dict(scores=_bf(2, 3)), 1),
    (select, lambda: dict(num_candidates=2), 1), (select, lambda: dict(num_candidates=5, eos_token=1), 1),
    (select, lambda: dict(logits=torch.randn(2, 40, 50, device=DEV), scores=torch.zeros(2, 40, device=DEV)), 1),
    (select, lambda: dict(workspace=torch.zeros(100, dtype=torch.uint8, device=DEV)), 1),
    (select, lambda: dict(next_beams=torch.zeros(2, 3, dtype=torch.int64, device=DEV)), 1),
    (select, lambda: dict(cand_scores=torch.zeros(2, 5, device=DEV)), 1),
    (reorder, lambda: dict(parents=torch.zeros(2, 3, dtype=torch.int64, device=DEV)), 1),
    (reorder, lambda: dict(parents=_i32(0, 0)), 1), (reorder, lambda: dict(seq_lens=_i32(1)), 1),
    (reorder, lambda: dict(cp=1), 1), (reorder, lambda: dict(own=_i32(1).view(1, 1, 1)), 1),
    (reorder, lambda: dict(k=None), 1), (reorder, lambda: dict(v=_bf(2, 24, 2, 16, 128)), 1),
    (reorder, lambda: dict(k=_bf(2, 24, 2, 8, 64), v=_bf(2, 24, 2, 8, 64)), 2),
    (reorder, lambda: dict(k=_bf(24, 2, 16, 64), v=_bf(24, 2, 16, 64)), 1),
    (reorder, lambda: dict(k=torch.zeros(2, 24, 2, 570, dtype=torch.uint8, device=DEV),
                           v=torch.zeros(2, 24, 2, 570, dtype=torch.uint8, device=DEV)), 1),
    (reorder, lambda: dict(tables_out=_i32(1)), 1), (reorder, lambda: dict(I=0), 1),
]


@pytest.mark.parametrize("i", range(len(BAD)))
def test_refusals(lib, i):
    call, kw, status = BAD[i]
    call(lib)                                       # what is right goes through
    with pytest.raises(lib.CPError) as e:
        call(lib, **kw())
    assert e.value.status == status, e.value
    call(lib)


def test_tables_may_not_overlap_in_part(lib):
    buf = torch.zeros(2 * 2 * 6 * 4, dtype=torch.int32, device=DEV)
    t = buf[:48].view(2, 6, 4)
    for at in (4, 44):
        with pytest.raises(lib.CPError):
            reorder(lib, tables=t, tables_out=buf[at:at + 48].view(2, 6, 4))
    reorder(lib, tables=t, tables_out=buf[48:].view(2, 6, 4))
    own = torch.zeros(2, 6, 4, dtype=torch.int32, device=DEV)
    with pytest.raises(lib.CPError):
        reorder(lib, own=own, tables_out=own)


def test_outputs_given_are_returned_and_defaults_made(lib):
    out, lse = _bf(6, 4, 64), torch.empty(6, 4, device=DEV)
    got = cross(lib, out=out, out_lse=lse, want_lse=False)
    assert got[0] is out and got[1] is lse
    o = [torch.empty(2, 3, device=DEV)] + [torch.empty(2, 3, dtype=torch.int32, device=DEV) for _ in range(2)] + \
        [torch.empty(2, 6, device=DEV)] + [torch.empty(2, 6, dtype=torch.int32, device=DEV) for _ in range(2)]
    names = ("next_scores", "next_beams", "next_tokens", "cand_scores", "cand_beams", "cand_tokens")
    assert all(a is b for a, b in zip(select(lib, **dict(zip(names, o))), o))
    assert select(lib)[3].shape == (2, 6)
    assert select(lib, logits=torch.randn(2, 3, 1, device=DEV))[3].shape == (2, 3)      # what there is
    t = reorder(lib)
    assert t.shape == (2, 6, 4) and t.dtype == torch.int32


def test_references_are_not_kept(lib):
    q, logits, parents = _bf(6, 4, 64), torch.randn(2, 3, 50, device=DEV), torch.zeros(2, 3, dtype=torch.int32, device=DEV)
    before = [sys.getrefcount(x) for x in (q, logits, parents)]
    for _ in range(50):
        cross(lib, q=q), select(lib, logits=logits), reorder(lib, parents=parents)
        for call, kw in ((cross, dict(q=q, max_seqlen_q=-1)), (select, dict(logits=logits, num_candidates=1)),
                         (reorder, dict(parents=parents, I=0))):
            with pytest.raises(lib.CPError):
                call(lib, **kw)
    del kw                                          # (holds the last call's)
    assert [sys.getrefcount(x) for x in (q, logits, parents)] == before


def test_calls_on_a_stream_of_their_own(lib):
    """Work queued before on that stream is waited for; the current stream is not used."""
    side = torch.cuda.Stream()
    big = torch.randn(4096, 4096, device=DEV)
    logits, q = torch.zeros(2, 3, 50, device=DEV), torch.zeros(6, 4, 64, dtype=torch.bfloat16, device=DEV)
    new, new_q = torch.randn(2, 3, 50, device=DEV), _bf(6, 4, 64)
    k, v = _bf(9, 2, 64), _bf(9, 2, 64)
    cu, cu_kv, zero = _i32(0, 2, 6), _i32(0, 4, 9), torch.zeros(2, 3, device=DEV)
    want, want_o = select(lib, logits=new), cross(lib, q=new_q, k=k, v=v)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(5):
            big = big @ big * 1e-3
        logits.copy_(new), q.copy_(new_q)
    got = lib.cp_beam_select(logits, zero, stream=side)
    out = lib.cp_cross_attention(q, cu, k, v, cu_kv, max_seqlen_q=4, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(out[0], want_o[0])


def test_leaves_that_want_gradients(lib):
    q = _bf(6, 4, 64).requires_grad_()
    assert not cross(lib, q=q)[0].requires_grad
    assert not select(lib, logits=torch.randn(2, 3, 50, device=DEV, requires_grad=True))[0].requires_grad
    with torch.inference_mode():
        cross(lib), select(lib), reorder(lib)
