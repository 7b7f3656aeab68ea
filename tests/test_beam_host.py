"""Host-side behaviour of cross attention, beam selection and reordering on a machine without a GPU: refusals
before any launch, and sizes of workspaces."""
import ctypes

import pytest

import context_gqa_attention_gb300 as cpa
from context_gqa_attention_gb300 import _build

P = ctypes.c_void_p(4096)      # an aligned address that no refused call reaches
ODD = ctypes.c_void_p(4100)
BYTE = ctypes.c_void_p(4097)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return cpa.load()


def _fill(a, kw):
    for n, v in kw.items():
        setattr(a, n, v)
    return a


def _detail(lib):
    buf = ctypes.create_string_buffer(256)
    lib.cp_last_error(buf, 256)
    return buf.value.decode()


CROSS = dict(dtype=1, num_seqs=2, num_q_heads=8, num_kv_heads=2, head_dim=128, max_seqlen_q=4, max_seqlen_kv=100,
             total_q=8, total_kv=200, q_stride=1024, k_stride=256, v_stride=512, q=P, k=P, v=P, cu_seqlens_q=P,
             cu_seqlens_kv=P)


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=2), 1), (dict(num_seqs=0), 1), (dict(num_kv_heads=0), 1), (dict(num_q_heads=7), 1),
    (dict(num_q_heads=0), 1), (dict(num_q_heads=258), 2), (dict(dtype=0, num_q_heads=130), 2), (dict(head_dim=96), 2),
    (dict(max_seqlen_q=-1), 1), (dict(max_seqlen_kv=-1), 1), (dict(total_q=-1), 1), (dict(total_kv=-1), 1),
    (dict(cu_seqlens_q=None), 1), (dict(cu_seqlens_kv=None), 1), (dict(q=None), 1), (dict(k=ODD), 1), (dict(v=None), 1),
    (dict(q_stride=1020), 1), (dict(q_stride=1016), 1), (dict(k_stride=248), 1), (dict(v_stride=260), 1),
    (dict(dtype=0, v_stride=514), 1), (dict(k_stride=-256), 1),
    (dict(num_seqs=1 << 20, max_seqlen_q=1 << 20), 1), (dict(dtype=0, num_seqs=1 << 24, max_seqlen_q=1 << 20), 1),
])
def test_cross_refusals(lib, bad, status):
    a = _fill(_fill(cpa.CrossArgs(), CROSS), bad)
    assert lib.cp_cross_attention(ctypes.byref(a), None, 0, P, P, None) == status, _detail(lib)
    assert _detail(lib)


def test_cross_refusals_of_the_outputs_and_calls_without_rows(lib):
    a = _fill(cpa.CrossArgs(), CROSS)
    assert lib.cp_cross_attention(None, None, 0, P, P, None) == 1
    assert lib.cp_cross_attention(ctypes.byref(a), None, 0, None, P, None) == 1
    assert lib.cp_cross_attention(ctypes.byref(a), None, 0, ODD, P, None) == 1
    assert lib.cp_cross_attention(ctypes.byref(a), ODD, 1 << 20, P, P, None) == 1 and "256" in _detail(lib)
    a.total_q, a.q = 0, None
    assert lib.cp_cross_attention(ctypes.byref(a), None, 0, None, None, None) == 0
    assert lib.cp_cross_attention_workspace_size(ctypes.byref(a), None) == 1


SELECT = dict(dtype=1, num_seqs=2, num_beams=4, vocab=1000, num_candidates=8, eos_token=3, logits_stride=1000,
              logits=P, scores=P, next_scores=P, next_beams=P, next_tokens=P, cand_scores=P, cand_beams=P, cand_tokens=P)


@pytest.mark.parametrize("bad", [
    dict(dtype=2), dict(num_seqs=0), dict(num_seqs=65537), dict(num_beams=0), dict(num_beams=33), dict(vocab=0),
    dict(vocab=(1 << 30) + 1, logits_stride=1 << 31), dict(num_candidates=3), dict(num_candidates=65),
    dict(num_candidates=7), dict(vocab=1, num_candidates=5, eos_token=-1), dict(logits_stride=999), dict(logits=None),
    dict(logits=BYTE), dict(dtype=0, logits=ctypes.c_void_p(4098)), dict(scores=None), dict(next_scores=None),
    dict(next_beams=None), dict(next_tokens=None), dict(cand_scores=None), dict(cand_beams=None), dict(cand_tokens=None),
    dict(num_seqs=65536, num_beams=32, vocab=1 << 30, logits_stride=1 << 30),
])
def test_select_refusals(lib, bad):
    a = _fill(_fill(cpa.BeamSelectArgs(), SELECT), bad)
    assert lib.cp_beam_select(ctypes.byref(a), P, 1 << 60, None) == 1, _detail(lib)
    assert _detail(lib)


def test_select_workspace(lib):
    a, n = _fill(cpa.BeamSelectArgs(), SELECT), ctypes.c_size_t()
    assert lib.cp_beam_select_workspace_size(2, 4, 1000, 8, ctypes.byref(n)) == 0 and n.value > 65536 * 4
    assert lib.cp_beam_select(ctypes.byref(a), P, n.value - 1, None) == 1 and "too small" in _detail(lib)
    assert lib.cp_beam_select(ctypes.byref(a), None, n.value, None) == 1
    assert lib.cp_beam_select(ctypes.byref(a), ODD, n.value, None) == 1
    assert lib.cp_beam_select(None, P, n.value, None) == 1
    assert lib.cp_beam_select_workspace_size(2, 4, 1000, 8, None) == 1
    assert lib.cp_beam_select_workspace_size(2, 4, 1, 8, ctypes.byref(n)) == 1
    # it does not shrink with the size: one made for the largest of some batches is enough for all
    sizes = []
    for B in (1, 3, 17, 64):
        assert lib.cp_beam_select_workspace_size(B, 4, 50257, 8, ctypes.byref(n)) == 0
        sizes.append(n.value)
    assert sizes == sorted(sizes)


REORDER = dict(dtype=1, cache_q4=0, num_layers=1, num_seqs=2, num_beams=4, num_kv_heads=2, head_dim=128, cp=2,
               interleave=8, block_size=16, max_blocks=4, pool_pages=8, parents=P, seq_lens=P, tables_in=P,
               own_pages=ctypes.c_void_p(8192), tables_out=ctypes.c_void_p(16384), k_cache=P, v_cache=P)


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=2), 1), (dict(cache_q4=2), 1), (dict(num_layers=0), 1), (dict(num_seqs=0), 1), (dict(num_beams=0), 1),
    (dict(num_beams=33), 1), (dict(num_kv_heads=0), 1), (dict(head_dim=96), 2), (dict(cp=0), 1), (dict(cp=65), 1),
    (dict(interleave=0), 1), (dict(block_size=32), 2), (dict(max_blocks=0), 1), (dict(pool_pages=0), 1),
    (dict(reserved=1), 1), (dict(parents=None), 1), (dict(seq_lens=None), 1), (dict(tables_in=None), 1),
    (dict(own_pages=None), 1), (dict(tables_out=None), 1), (dict(k_cache=None), 1), (dict(v_cache=ODD), 1),
    (dict(tables_out=ODD), 1), (dict(tables_out=ctypes.c_void_p(4096 - 4)), 1), (dict(tables_out=ctypes.c_void_p(8200)), 1),
    (dict(own_pages=P, tables_out=P), 1),
])
def test_reorder_refusals(lib, bad, status):
    a = _fill(_fill(cpa.BeamReorderArgs(), REORDER), bad)
    assert lib.cp_beam_reorder(ctypes.byref(a), None) == status, _detail(lib)
    assert _detail(lib)


def test_struct_mirrors(lib):
    for name, struct in (("cross", cpa.CrossArgs), ("beam_select", cpa.BeamSelectArgs),
                         ("beam_reorder", cpa.BeamReorderArgs)):
        assert getattr(lib, f"cp_{name}_args_size")() == ctypes.sizeof(struct)
