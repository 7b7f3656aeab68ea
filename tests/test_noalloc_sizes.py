"""cp_decode_attention_noalloc takes every size whose partials, LSEs and counters fit its 48 MiB."""
import ctypes

import pytest
import torch

import context_gqa_attention_gb300 as cpa
from context_gqa_attention_gb300 import _build

MiB48 = 48 * 1024 * 1024


def _need(B, Hq, Hkv, d, P):
    """Counters, LSEs and partial rows, each region 256-byte aligned."""
    up = lambda n: -(-n // 256) * 256
    return up(4 * B * Hkv) + up(4 * P * B * Hq) + up(4 * P * B * Hq * d)


# 190 sequences, 64/8 heads, 8 partials: 50,202,624 of 50,331,648 bytes; and its neighbours on both sides
FITS = [(190, 64, 8, 128, 8), (47, 64, 8, 128, 32), (3000, 8, 8, 128, 4), (189, 64, 8, 64, 16)]
DOES_NOT = [(191, 64, 8, 128, 8), (3100, 8, 8, 128, 4)]


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are made up: only where no kernel can start")
@pytest.mark.parametrize("B,Hq,Hkv,d,P", FITS + DOES_NOT)
def test_the_limit_is_the_array(B, Hq, Hkv, d, P):
    _build.build()
    lib = cpa.load()
    assert (_need(B, Hq, Hkv, d, P) <= MiB48) == ((B, Hq, Hkv, d, P) in FITS)
    p = ctypes.c_void_p(4096)
    a = cpa.DecodeArgs(dtype=1, num_seqs=B, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=d, cp=2, interleave=8,
                       block_size=16, num_splits=P // 2, split_tokens=64, max_blocks=8, pool_pages=8, q=p, k_cache=p,
                       v_cache=p, block_tables=p, seq_lens=p)
    st = lib.cp_decode_attention_noalloc(ctypes.byref(a), p, None, None)
    # too large: an invalid argument; else the next thing it does, the array's address, needs a GPU
    assert st == (3 if (B, Hq, Hkv, d, P) in FITS else 1)


@pytest.mark.gpu
def test_a_call_that_nearly_fills_the_array(lib):
    B, Hq, Hkv, d, P = FITS[0]
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(B, Hq, d, generator=g, device="cuda").to(torch.bfloat16)
    kc, vc = (torch.randn(2, 40, Hkv, 16, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    t = torch.randint(0, 40, (2, B, 8), generator=g, device="cuda").to(torch.int32)
    lens = torch.randint(1, 257, (B,), generator=g, device="cuda").to(torch.int32)
    want, want_lse = lib.cp_decode_attention(q, kc, vc, t, lens, 2, 8, num_splits=P // 2, split_tokens=32)
    out, lse = torch.empty_like(want), torch.empty_like(want_lse)
    for _ in range(2):
        out.zero_(), lse.zero_()
        lib.cp_decode_attention_noalloc(q, kc, vc, t, lens, 2, 8, out, num_splits=P // 2, split_tokens=32, out_lse=lse)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
