"""Reordering that makes its tables anew: a copy of the ones given wherever a beam or a sequence is left as it is."""
import numpy as np
import pytest
import torch

from oracle import beam_oracle as bo
from test_gpu_beam import DEV, I32, paging

pytestmark = pytest.mark.gpu


def _bf(*shape):
    return torch.randn(*shape, device=DEV).to(torch.bfloat16)


@pytest.mark.parametrize("caches", [True, False])
def test_new_tables_where_a_beam_or_a_sequence_is_left_as_it_is(lib, caches):
    r = np.random.default_rng(6)
    lens, K, cp, I, cols = [40, 77, 21], 3, 2, 8, 9
    tables, own, pool = paging(lens, K, cp, I, cols, r)
    parents = r.integers(0, K, (3, K)).astype(np.int32)
    parents[0, 1], lens[2] = K, 16 * cols * cp + 1           # a parent that is none; a length that the tables do not hold
    base = [_bf(cp, pool, 1, 16, 64) for _ in range(2)]
    want = tables.copy()
    for k in range(cp):
        for b in (0, 1):
            n = bo.held(lens[b], k, cp, I) // 16
            for j, p in enumerate(parents[b]):
                if p < K:
                    want[k, b * K + j, :n] = tables[k, b * K + p, :n]
                    want[k, b * K + j, n] = own[k, b * K + j, n]
    t, err = torch.tensor(tables, device=DEV), torch.zeros(1, **I32)
    for _ in range(3):
        old = torch.full_like(t, 123456)                     # (what the memory of a new tensor may hold)
        del old
        got = lib.cp_beam_reorder(torch.tensor(parents, device=DEV), torch.tensor(lens, **I32), t, torch.tensor(own, device=DEV),
                                  *(base if caches else (None, None)), cp, I, err=err)
        assert int(err) == 5 and got.data_ptr() != t.data_ptr()
        assert np.array_equal(got.cpu().numpy(), want) and np.array_equal(t.cpu().numpy(), tables)


def test_new_tables_on_a_stream_of_their_own(lib):
    """The copy, too, follows what that stream holds."""
    side = torch.cuda.Stream()
    t = torch.full((1, 2, 50), -1, **I32)
    new = torch.arange(100, **I32).view(1, 2, 50)
    args = torch.tensor([[1, 5]], **I32), torch.tensor([20], **I32)
    big = torch.randn(4096, 4096, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(5):
            big = big @ big * 1e-3
        t.copy_(new)
    got = lib.cp_beam_reorder(args[0], args[1], t, new, None, None, 1, 16, stream=side)
    side.synchronize()
    want = new.clone()
    want[0, 0, 0] = new[0, 1, 0]
    assert torch.equal(got, want)
