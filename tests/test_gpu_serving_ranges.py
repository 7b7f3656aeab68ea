"""Values far apart in size, and scores at the ends of their range, in the serving calls."""
import math

import numpy as np
import pytest
import torch

from test_gpu_serving_large import DEV, I32, _attend, _check, _cu, _pool

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------ V's range, 4 bits
def _minima(pool, t, n, cp, I, d):
    """Each value's group minimum of positions 0..n-1 of sequence 0, [n, Hkv, d], in float64."""
    p = np.arange(n)
    turn = p // I
    rank, local = turn % cp, turn // cp * I + p % I
    page = t.cpu().numpy()[rank, 0, local // 16]
    rec = pool[torch.tensor(rank, device=DEV), torch.tensor(page, device=DEV).long()]        # [n, Hkv, 9 d]
    at = torch.tensor(local % 16, device=DEV)
    pairs = rec[..., 8 * d:].reshape(n, rec.shape[1], 16, d // 16).contiguous()
    pairs = pairs[torch.arange(n, device=DEV), :, at].contiguous().view(torch.bfloat16)      # scale, minimum, ..
    return pairs[..., 1::2].double().repeat_interleave(64, -1)


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 1, 128), (8, 1, 128), (16, 1, 128), (6, 2, 64), (14, 1, 64)])
@pytest.mark.parametrize("cap", [0.0, 500.0])
@pytest.mark.parametrize("rise,fall", [(60.0, 16), (60.0, 24), (60.0, 40), (25.0, 30), (12.0, 12), (9.0, 9), (100.0, 50), (30.0, 7), (12.0, 25), (8.5, 20)])
def test_v_scales_that_fall_while_the_scores_rise(lib, Hq, Hkv, d, cap, rise, fall):
    """The tokens of each later part of the sequence score `rise` (in powers of two) more and their V is 2^-fall
    as large: the parts before it count for nothing then, and what they left behind must not cost the later ones
    their bits.  V's smallest value is near 0 in half of the groups, so that the minima do not stand in for it.

    Tolerance: that of the 4-bit decode (see test_gpu_serving), with |value - minimum| <= |value| + |minimum|
    of the tokens that count.  A factor that is 2^k below the largest that counts is off by 2^-25 2^k units: with
    2^-8 allowed and up to a few hundred equal weights, that needs no term of its own."""
    parts, n, cp, I = 3, 3 * 192, 1, 16
    k, v, t = _pool([n], Hkv, d, cp, I, torch.bfloat16, True, 3)
    g = torch.Generator(device=DEV).manual_seed(4)
    part = torch.arange(n, device=DEV) // 192
    # q = c (1, .., 1), k = a (1, .., 1) + little: q.k / sqrt(d) = c a sqrt(d)
    c = 2.0
    level = (part.double() - (parts - 1)) * rise * math.log(2) / (c * math.sqrt(d))
    kn = (level[:, None, None] + 0.02 * torch.randn(n, Hkv, d, generator=g, device=DEV)).to(torch.bfloat16)
    vn = torch.rand(n, Hkv, d, generator=g, device=DEV)
    vn[:, :, :32] = 2 * vn[:, :, :32] - 1
    vn = (vn * (2.0 ** (fall * (parts - 1 - part.double())))[:, None, None]).to(torch.bfloat16)
    lib.cp_rope_kv_cache_write(kn, vn, _cu([n]), torch.zeros(1, **I32), k, v, t, cp, I)
    K, V = (x.double() for x in lib.cp_kv_cache_read(k, v, _cu([n]), torch.zeros(1, **I32), t, cp, I, out_dtype=torch.float32))
    M = _minima(v, t, n, cp, I, d)
    q = torch.full((1, Hq, d), c, dtype=torch.bfloat16, device=DEV)
    one = torch.tensor([n - 1], device=DEV)
    O, L, A, big = _attend(q.double(), K, V, 0 * one, one + 1, one, cap, None)
    extra = _attend(q.double(), K, M.abs(), 0 * one, one + 1, one, cap, None)[0]
    for S, tokens in ((1, 576), (3, 192), (2, 320)):
        out, lse = lib.cp_decode_attention_q4(q, k, v, t, torch.tensor([n], **I32), cp, I, softcap=cap, num_splits=S, split_tokens=tokens)
        _check(out, lse, O, L, A, big, cap, None, n, extra=extra, what=f"{S} x {tokens}")
