"""Host-side behaviour of the rotate-and-append, read-back, 4-bit and modified-score calls, on a
machine without a GPU: refusals before any launch, and the split plan's coverage."""
import ctypes
import math

import pytest
import torch

import context_gqa_attention_gb300 as cpa
from context_gqa_attention_gb300 import _build
from oracle import cp_oracle as orc

P = ctypes.c_void_p(4096)      # an aligned address that no refused call reaches
ODD = ctypes.c_void_p(4100)


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


WRITE = dict(dtype=1, cache_q4=0, num_seqs=1, total_new=4, num_q_heads=4, num_kv_heads=2, head_dim=128, cp=2,
             interleave=8, block_size=16, max_blocks=4, rope_style=0, rot_dim=128, pool_pages=8, q_stride=512,
             k_stride=256, v_stride=256, q_out_stride=512, q=P, k=P, v=P, cu_new=P, start_pos=P, inv_freq=P,
             block_tables=P, k_cache=P, v_cache=P, q_out=P)


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=2), 1), (dict(cache_q4=2), 1), (dict(num_seqs=0), 1), (dict(total_new=-1), 1),
    (dict(num_kv_heads=0), 1), (dict(head_dim=96), 2), (dict(cp=0), 1), (dict(cp=65), 1), (dict(interleave=0), 1),
    (dict(block_size=32), 2), (dict(max_blocks=0), 1), (dict(pool_pages=0), 1), (dict(rope_style=2), 1),
    (dict(rot_dim=24), 1), (dict(rot_dim=144), 1), (dict(rot_dim=-16), 1), (dict(inv_freq=None), 1),
    (dict(reserved=1), 1), (dict(cu_new=None), 1), (dict(start_pos=None), 1), (dict(block_tables=None), 1),
    (dict(k=None), 1), (dict(v=ODD), 1), (dict(k_cache=ODD), 1), (dict(v_cache=None), 1), (dict(k_out=ODD), 1),
    (dict(k_stride=260), 1), (dict(v_stride=248), 1), (dict(q_stride=504), 1), (dict(q_out=None), 1),
    (dict(q=None), 1), (dict(q_out_stride=1024), 1), (dict(num_q_heads=0), 1),
])
def test_write_refusals(lib, bad, status):
    a = _fill(_fill(cpa.RopeWriteArgs(), WRITE), bad)
    assert lib.cp_rope_kv_cache_write(ctypes.byref(a), None) == status, _detail(lib)
    assert _detail(lib)


def test_write_and_read_of_no_rows_are_accepted(lib):
    a = _fill(_fill(cpa.RopeWriteArgs(), WRITE), dict(total_new=0))
    assert lib.cp_rope_kv_cache_write(ctypes.byref(a), None) == 0
    r = _fill(cpa.KvReadArgs(), dict(READ, total=0, k_out=None, v_out=None))
    assert lib.cp_kv_cache_read(ctypes.byref(r), None) == 0


READ = dict(out_dtype=1, cache_q4=1, num_seqs=1, total=4, num_kv_heads=2, head_dim=128, cp=2, interleave=8,
            block_size=16, max_blocks=4, pool_pages=8, k_cache=P, v_cache=P, block_tables=P, cu_out=P, start_pos=P,
            k_out=P, v_out=P)


@pytest.mark.parametrize("bad,status", [
    (dict(out_dtype=2), 1), (dict(cache_q4=-1), 1), (dict(num_seqs=0), 1), (dict(total=-1), 1),
    (dict(head_dim=32), 2), (dict(block_size=8), 2), (dict(cp=65), 1), (dict(interleave=0), 1),
    (dict(k_cache=ODD), 1), (dict(v_cache=None), 1), (dict(k_out=None), 1), (dict(v_out=ODD), 1),
    (dict(cu_out=None), 1), (dict(start_pos=None), 1), (dict(block_tables=None), 1), (dict(pool_pages=0), 1),
])
def test_read_refusals(lib, bad, status):
    a = _fill(_fill(cpa.KvReadArgs(), READ), bad)
    assert lib.cp_kv_cache_read(ctypes.byref(a), None) == status, _detail(lib)


DECODE = dict(dtype=1, num_seqs=2, num_q_heads=8, num_kv_heads=2, head_dim=128, cp=2, interleave=8, block_size=16,
              num_splits=2, split_tokens=64, max_blocks=8, pool_pages=8, q=P, k_cache=P, v_cache=P, block_tables=P,
              seq_lens=P, out=P, lse=P)


@pytest.mark.parametrize("name", ["mod", "q4"])
@pytest.mark.parametrize("bad,mod,status", [
    (dict(head_dim=96), {}, 2), (dict(block_size=32), {}, 2), (dict(num_q_heads=34), {}, 2),
    (dict(num_q_heads=7), {}, 1), (dict(split_tokens=40), {}, 1), (dict(num_splits=0), {}, 1),
    (dict(q=None), {}, 1), (dict(k_cache=ODD), {}, 1), (dict(seq_lens=None), {}, 1),
    ({}, dict(softcap=-1.0), 1), ({}, dict(softcap=math.inf), 1), ({}, dict(softcap=math.nan), 1),
    ({}, dict(softcap=1e-9), 1), ({}, dict(softcap=1e12), 1),
    ({}, dict(window=-1), 1), ({}, dict(prefix_lens=P), 1),
])
def test_decode_refusals(lib, name, bad, mod, status):
    a = _fill(_fill(cpa.DecodeArgs(), DECODE), bad)
    m = _fill(cpa.ScoreMod(), mod)
    part, fused = getattr(lib, f"cp_partial_attn_decode_{name}"), getattr(lib, f"cp_decode_attention_{name}")
    assert part(ctypes.byref(a), ctypes.byref(m), None) == status, _detail(lib)
    assert fused(ctypes.byref(a), ctypes.byref(m), P, 1 << 30, P, P, None) == status


def test_fused_decode_refuses_its_own(lib):
    a, m = _fill(cpa.DecodeArgs(), DECODE), cpa.ScoreMod()
    for f in (lib.cp_decode_attention_mod, lib.cp_decode_attention_q4):
        assert f(ctypes.byref(a), ctypes.byref(m), None, 1 << 30, P, P, None) == 1        # no workspace
        assert f(ctypes.byref(a), ctypes.byref(m), ctypes.c_void_p(4096 + 64), 1 << 30, P, P, None) == 1
        assert f(ctypes.byref(a), ctypes.byref(m), P, 100, P, P, None) == 1                # too small
        assert "too small" in _detail(lib)
        assert f(ctypes.byref(a), ctypes.byref(m), P, 1 << 30, ODD, P, None) == 1
        b = _fill(_fill(cpa.DecodeArgs(), DECODE), dict(num_splits=200))
        assert f(ctypes.byref(b), ctypes.byref(m), P, 1 << 30, P, P, None) == 2            # > 256 partials
    f32 = _fill(_fill(cpa.DecodeArgs(), DECODE), dict(dtype=0))
    assert lib.cp_decode_attention_q4(ctypes.byref(f32), ctypes.byref(m), P, 1 << 30, P, P, None) == 2
    assert lib.cp_partial_attn_decode_q4(ctypes.byref(f32), None, None) == 2


PREFILL = dict(mode=0, dtype=1, impl=0, num_seqs=1, num_q_heads=8, num_kv_heads=2, head_dim=128, cp=1,
               max_seqlen_q=4, cu_seqlens_q=P, q=P, k=P, v=P, q_shard=-1, kv_shard=-1, total_q=4)


@pytest.mark.parametrize("bad,mod,status", [
    (dict(mode=1), {}, 2), (dict(dtype=0), {}, 2), (dict(impl=2), {}, 2), (dict(impl=3), {}, 2),
    (dict(head_dim=32), {}, 2), (dict(num_q_heads=7), {}, 1), (dict(q_shard=0), {}, 1), (dict(k=None), {}, 1),
    (dict(v=ODD), {}, 1), (dict(cu_seqlens_q=None), {}, 1), (dict(debug=1), {}, 1),
    (dict(cu_seqlens_kv=P, total_kv=0), {}, 1), ({}, dict(softcap=-0.5), 1), ({}, dict(window=-2), 1),
    (dict(num_seqs=70000), {}, 2), (dict(max_seqlen_q=1 << 24), {}, 2),
])
def test_prefill_refusals(lib, bad, mod, status):
    a = _fill(_fill(cpa.PrefillArgs(), PREFILL), bad)
    m = _fill(cpa.ScoreMod(), mod)
    assert lib.cp_attn_prefill_mod(ctypes.byref(a), ctypes.byref(m), P, P, None) == status, _detail(lib)
    ok = _fill(_fill(cpa.PrefillArgs(), PREFILL), dict(total_q=0))
    assert lib.cp_attn_prefill_mod(ctypes.byref(ok), None, P, P, None) == 0
    assert lib.cp_attn_prefill_mod(ctypes.byref(ok), None, None, P, None) == 1
    assert lib.cp_attn_prefill_mod(ctypes.byref(ok), None, P, None, None) == 1


def test_the_binding_refuses_host_tensors():
    x = torch.zeros(2, 2, 64)
    with pytest.raises(cpa.CPError):
        cpa.cp_kv_cache_read(x, x, x, x, x, 1, 8)
    with pytest.raises(cpa.CPError):
        cpa.cp_decode_attention_q4(x, x, x, x, x, 1, 8)
    with pytest.raises(cpa.CPError):
        cpa.cp_attn_prefill_mod(x, x, x, x)
    with pytest.raises(cpa.CPError):
        cpa.cp_rope_kv_cache_write(x, x, x, x, x, x, x, 1, 8)


def _local_len(L, r, cp, I):
    return L // (I * cp) * I + min(max(L % (I * cp) - r * I, 0), I)


def test_local_len_is_the_deal():
    for cp, I in [(1, 8), (2, 8), (3, 5), (8, 1)]:
        for L in (0, 1, 17, 200):
            assert [_local_len(L, r, cp, I) for r in range(cp)] == orc.local_lengths([L], cp, I)[:, 0].tolist()


@pytest.mark.parametrize("B,Hkv", [(1, 1), (1, 8), (7, 2), (64, 8)])
@pytest.mark.parametrize("cp,I", [(1, 8), (2, 8), (3, 5), (8, 1), (64, 16)])
@pytest.mark.parametrize("q4", [False, True])
def test_the_plan_covers_every_rank(lib, B, Hkv, cp, I, q4):
    for L in (1, 15, 16, 17, 333, 1777, 32768, 1 << 20, (1 << 31) - 1):
        for W in (0, 1, 16, 100, 4096):
            S, st = cpa.cp_decode_mod_plan(B, Hkv, cp, I, L, window=W, q4=q4)
            assert S >= 1 and st >= 16 and st % 16 == 0 and cp * S <= 256
            for n in {L, max(1, L - 7), max(1, L // 2)}:        # any sequence up to the longest
                lo = max(0, n - W) if W else 0
                for r in range(cp):
                    end, first = _local_len(n, r, cp, I), _local_len(lo, r, cp, I)
                    assert first >= end or end - first // 16 * 16 <= S * st, (L, W, n, r)


def test_plan_refusals(lib):
    for bad in ((0, 1, 1, 8, 10), (1, 0, 1, 8, 10), (1, 1, 65, 8, 10), (1, 1, 1, 0, 10), (1, 1, 1, 8, 0)):
        with pytest.raises(cpa.CPError):
            cpa.cp_decode_mod_plan(*bad)
    with pytest.raises(cpa.CPError):
        cpa.cp_decode_mod_plan(1, 1, 1, 8, 10, window=-1)
    assert cpa.cp_q4_record_bytes(128) == 1152 and cpa.cp_q4_record_bytes(64) == 576
