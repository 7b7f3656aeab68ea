"""The sizes that cp_cross_attention_workspace_size answers, against what the calls of each form ask for, and ranged calls
with a workspace of that size between guard words."""
import ctypes
import math

import numpy as np
import pytest
import torch

from test_gpu_cross import DEV, DT, I32, _cu, check, exact

pytestmark = pytest.mark.gpu


def wanted(lib, B, Hq, Hkv, d, T, S, dtype, lens, ranges):
    a = lib.CrossArgs()
    a.dtype, a.num_seqs, a.num_q_heads, a.num_kv_heads, a.head_dim = int(dtype == "bf16"), B, Hq, Hkv, d
    a.max_seqlen_q, a.max_seqlen_kv, a.total_q, a.total_kv = T, S, B * T, B * S
    a.kv_lens, a.key_ranges = int(lens), int(ranges)
    need = ctypes.c_size_t()
    assert lib.load().cp_cross_attention_workspace_size(ctypes.byref(a), ctypes.byref(need)) == 0
    return need.value


# B, rows of a sequence, keys, Hq, Hkv, d, dtype
SHAPES = [(1, 900, 4000, 8, 2, 128, "bf16"), (2, 300, 3007, 16, 4, 128, "bf16"), (1, 600, 6404, 16, 2, 128, "bf16"),
          (1, 200, 4096, 32, 8, 128, "bf16"), (1, 300, 2000, 2, 2, 64, "bf16"), (7, 90, 300, 4, 4, 64, "bf16"),
          (64, 4, 2000, 32, 8, 128, "bf16"), (1, 3, 20000, 2, 1, 64, "bf16"), (1, 3, 20000, 2, 1, 64, "f32"),
          (3, 100, 900, 4, 2, 64, "f32"), (1, 1, 1, 1, 1, 64, "bf16")]


@pytest.mark.parametrize("shape", SHAPES)
def test_sizes_of_each_form(lib, shape):
    B, T, S, Hq, Hkv, d, dtype = shape
    forms = {(l, r): wanted(lib, B, Hq, Hkv, d, T, S, dtype, l, r) for l in (False, True) for r in (False, True)}
    size = lambda **kw: lib.cp_cross_attention_workspace_size(B, Hq, Hkv, d, T, S, dtype=DT[dtype], **kw)
    assert size() == forms[False, False]
    assert size(padded=True) == max(forms[True, False], forms[False, True], forms[True, True])


@pytest.mark.parametrize("B,T,S,Hq,Hkv,d", [x[:6] for x in SHAPES[:4]])
@pytest.mark.parametrize("padded", [False, True])
def test_ranged_parts_between_guards(lib, B, T, S, Hq, Hkv, d, padded):
    """Few items of many rows and long keys: cut through the workspace whose size is asked for."""
    r = np.random.default_rng(S)
    keys = r.integers(S // 2, S + 1, B) if padded else np.full(B, S)
    g = torch.Generator(device=DEV).manual_seed(S)
    n, pad = B * T, 64
    q = torch.randn(n, Hq, d, generator=g, device=DEV).bfloat16()
    k, v = (torch.randn(B * S, Hkv, d, generator=g, device=DEV).bfloat16() for _ in range(2))
    lo = torch.randint(0, S, (n,), generator=g, device=DEV)
    ranges = torch.stack([lo, lo + torch.randint(0, S, (n,), generator=g, device=DEV)], -1).int().contiguous()
    ranges[3], ranges[T - 1] = torch.tensor([0, S], **I32), torch.tensor([5, 5], **I32)
    hidden = (torch.arange(S, device=DEV)[None] >= torch.tensor(keys, device=DEV)[:, None]).reshape(-1)
    k[hidden], v[hidden] = math.nan, math.inf
    clipped = torch.minimum(ranges, torch.tensor(keys, **I32).repeat_interleave(T)[:, None])
    want = exact(q, k, v, [(b * T, T, b * S, int(m)) for b, m in enumerate(keys)], d ** -0.5, clipped)
    need = lib.cp_cross_attention_workspace_size(B, Hq, Hkv, d, T, S, padded=True)
    assert need > 0
    ws = torch.full((need + 2 * 256,), 0xa5, dtype=torch.uint8, device=DEV)
    out = torch.full((n + 2 * pad, Hq, d), 12345.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((n + 2 * pad, Hq), 12345.0, device=DEV)
    err = torch.zeros(1, **I32)
    lib.cp_cross_attention(q, _cu([T] * B), k, v, _cu([S] * B), kv_lens=torch.tensor(keys, **I32) if padded else None,
                           key_ranges=ranges, max_seqlen_q=T, max_seqlen_kv=S, workspace=ws[256:256 + need],
                           out=out[pad:pad + n], out_lse=lse[pad:pad + n], err=err)
    assert int(err) == 0
    check(out[pad:pad + n], lse[pad:pad + n], want, False)
    assert bool((ws[256:256 + need] != 0xa5).any())                  # it was cut
    for x, m in ((out, torch.tensor(12345.0).bfloat16().to(DEV)), (lse, 12345.0)):
        assert bool((x[:pad] == m).all()) and bool((x[pad + n:] == m).all())
    assert bool((ws[:256] == 0xa5).all()) and bool((ws[256 + need:] == 0xa5).all())
