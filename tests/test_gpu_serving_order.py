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
