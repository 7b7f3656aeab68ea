"""What the calls return when no outputs are given: tensors with memory of their own."""
import pytest
import torch

from test_gpu_beam import DEV, I32

pytestmark = pytest.mark.gpu


def _bf(*shape):
    return torch.randn(*shape, device=DEV).to(torch.bfloat16)


def test_rows_and_lses_have_memory_of_their_own(lib):
    """Each can be kept, freed, saved or resized apart from the other."""
    cu = lambda *x: torch.tensor(x, **I32)
    outs = lib.cp_cross_attention(_bf(6, 4, 64), cu(0, 2, 6), _bf(9, 2, 64), _bf(9, 2, 64), cu(0, 4, 9))
    for t in outs:
        s = t.untyped_storage()
        assert t.storage_offset() == 0 and s.nbytes() == t.numel() * t.element_size() and t.is_contiguous()
    assert outs[0].untyped_storage().data_ptr() != outs[1].untyped_storage().data_ptr()
    lse = outs[1].clone()
    outs[0].resize_(4096).fill_(77)                      # grows: into new memory
    assert torch.equal(outs[1], lse)


def test_outputs_of_a_selection_do_not_overlap(lib):
    """New and given ones, whose values are what they are when all are given."""
    logits, scores = torch.randn(5, 3, 70, device=DEV), torch.randn(5, 3, device=DEV)
    mine = torch.empty(5, 3, dtype=torch.int32, device=DEV)
    got = lib.cp_beam_select(logits, scores, eos_token=3)
    for t, w in zip(lib.cp_beam_select(logits, scores, eos_token=3, next_tokens=mine), got):
        assert torch.equal(t, w) and t.is_contiguous()
    spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in got)
    assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:]))
    assert all(a % 256 == 0 for a, _ in spans)


def test_empty_outputs(lib):
    zero = torch.zeros(3, **I32)
    out, lse = lib.cp_cross_attention(_bf(0, 4, 64), zero, _bf(9, 2, 64), _bf(9, 2, 64), zero)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4) and out.dtype == torch.bfloat16
    assert out.untyped_storage().nbytes() == 0
