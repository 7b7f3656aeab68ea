"""Values that are not finite behind a visible key whose score lies far below the row's largest: however the keys are cut,
the row's component is not finite (infinite or NaN), and every other component is what it is without."""
import math

import pytest
import torch

from test_gpu_cross import DEV, DT, I32, _cu

pytestmark = pytest.mark.gpu

# rows, keys, Hq, Hkv, d, dtype
FAR = [(3, 2000, 2, 2, 64, "bf16"), (3, 20000, 2, 2, 64, "bf16"), (1, 100, 2, 2, 128, "bf16"), (20, 9000, 2, 2, 128, "bf16"),
       (200, 2000, 2, 2, 64, "bf16"), (600, 6404, 16, 2, 128, "bf16"), (300, 2000, 2, 2, 128, "bf16"), (150, 120, 2, 2, 64, "bf16"),
       (3, 2000, 2, 2, 64, "f32"), (3, 20000, 2, 2, 64, "f32"), (5, 300, 2, 2, 128, "f32"), (70, 900, 4, 2, 64, "f32")]


@pytest.mark.parametrize("T,S,Hq,Hkv,d,dtype", FAR)
@pytest.mark.parametrize("form", ["plain", "ranges", "whole", "whole ranges"])
@pytest.mark.parametrize("nats", [30, 200, 5000])
def test_what_is_not_finite_stays_so(lib, T, S, Hq, Hkv, d, dtype, form, nats):
    """The last 8 keys hold nearly all of the weight, the others `nats` less; these keys lie in the first and a middle part."""
    g = torch.Generator(device=DEV).manual_seed(S)
    q = torch.zeros(T, Hq, d, device=DEV)
    q[..., 0] = 8
    k = torch.zeros(S, Hkv, d, device=DEV)
    k[:-8, :, 0] = -nats * math.sqrt(d) / 8
    v = torch.randn(S, Hkv, d, generator=g, device=DEV)
    q, k, v = (x.to(DT[dtype]) for x in (q, k, v))
    ranges = torch.tensor([[0, S]] * T, **I32) if "ranges" in form else None
    ws = torch.empty(0, dtype=torch.uint8, device=DEV) if "whole" in form else None
    f = lambda: lib.cp_cross_attention(q, _cu([T]), k, v, _cu([S]), key_ranges=ranges, max_seqlen_q=T, max_seqlen_kv=S,
                                       workspace=ws)
    clean, cl = f()
    assert bool(clean.isfinite().all()) and bool(cl.isfinite().all())
    v[3, 0, 5], v[S // 2, 1, 7], v[S // 2 + 1, 1, 9] = math.inf, math.nan, -math.inf
    out, lse = f()
    G = Hq // Hkv
    assert torch.equal(lse, cl)
    for h, c in ((0, 5), (1, 7), (1, 9)):
        assert not bool(out[:, h * G:(h + 1) * G, c].isfinite().any()), (h, c)
        out[:, h * G:(h + 1) * G, c] = clean[:, h * G:(h + 1) * G, c]
    assert bool((out[:, G:, 7] == clean[:, G:, 7]).all()) and torch.equal(out, clean)
