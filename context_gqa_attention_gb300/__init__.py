"""Python binding of libcpattn (include/cpattn.h): causal GQA partial attention over logical
context-parallel shards, LSE merge and the CP layout maps, on one GB300 (sm_103a).

Argument marshalling only: every function below checks tensor placement, dtype and shape,
then calls the C entry point of the same name on the current torch CUDA stream (the serving
calls -- rotate-and-append, read-back, 4-bit decode, modified scores, cross attention, beam search -- do
both in the native module built from csrc/binding.cpp).  All the
arithmetic runs in the library's CUDA kernels; there is no fallback.  A missing or unbuilt
library raises ``CPError``.

PyTorch provides device memory and streams.  Output tensors may be passed in (the library
never allocates); when omitted they are allocated here with ``torch.empty``.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import importlib.util
import inspect
import math
import os
import threading

import torch

from . import _build

__all__ = [
    "CPError", "load", "lib_path", "CP_F32", "CP_BF16", "CP_PASS_KV", "CP_PASS_Q",
    "CP_IMPL_AUTO", "CP_IMPL_TCGEN05", "CP_IMPL_SIMT", "CP_IMPL_TCGEN05_SINGLE",
    "cp_partition", "cp_kv_interleave_layout",
    "cp_partial_attn_prefill", "cp_decode_plan", "cp_partial_attn_decode", "cp_lse_merge",
    "cp_decode_workspace_size", "cp_decode_attention", "cp_decode_attention_noalloc",
    "cp_kv_cache_write", "cp_select_prefill_mode", "cp_attn_prefill_fused",
    "cp_prefill_fused_workspace_size", "STATUS",
    "CP_ROPE_HALF", "CP_ROPE_PAIRS", "cp_rope_kv_cache_write", "cp_kv_cache_read",
    "cp_q4_record_bytes", "cp_attn_prefill_mod", "cp_decode_mod_plan",
    "cp_partial_attn_decode_mod", "cp_decode_attention_mod", "cp_partial_attn_decode_q4",
    "cp_decode_attention_q4", "cp_cross_attention", "cp_cross_attention_workspace_size",
    "cp_beam_select", "cp_beam_select_workspace_size", "cp_beam_reorder",
]

CP_F32, CP_BF16 = 0, 1
CP_PASS_KV, CP_PASS_Q = 0, 1
CP_IMPL_AUTO, CP_IMPL_TCGEN05, CP_IMPL_SIMT, CP_IMPL_TCGEN05_SINGLE = 0, 1, 2, 3
CP_ROPE_HALF, CP_ROPE_PAIRS = 0, 1
STATUS = {0: "CP_OK", 1: "CP_ERR_INVALID_ARG", 2: "CP_ERR_UNSUPPORTED", 3: "CP_ERR_CUDA",
          4: "CP_ERR_TIMEOUT", 5: "CP_ERR_DEVICE_BOUNDS"}

_c_int32_p = ctypes.c_void_p
_vp = ctypes.c_void_p


class CPError(RuntimeError):
    def __init__(self, status, detail):
        super().__init__(f"{STATUS.get(status, status)}: {detail}")
        self.status = status
        self.detail = detail


class PrefillArgs(ctypes.Structure):
    _fields_ = [
        ("mode", ctypes.c_int32), ("dtype", ctypes.c_int32), ("impl", ctypes.c_int32),
        ("num_seqs", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("cp", ctypes.c_int32),
        ("max_seqlen_q", ctypes.c_int32), ("softmax_scale", ctypes.c_float),
        ("cu_seqlens_q", _vp), ("seq_lens_kv", _vp), ("q", _vp), ("k", _vp), ("v", _vp),
        ("k_cache", _vp), ("v_cache", _vp), ("pool_pages", ctypes.c_int64),
        ("block_tables", _vp), ("max_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
        ("interleave", ctypes.c_int32), ("q_shard", ctypes.c_int32), ("kv_shard", ctypes.c_int32),
        ("total_q", ctypes.c_int32), ("debug", ctypes.c_int32), ("out", _vp), ("lse", _vp),
        ("err", _vp), ("cu_seqlens_kv", _vp), ("total_kv", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class DecodeArgs(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int32), ("num_seqs", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("cp", ctypes.c_int32),
        ("interleave", ctypes.c_int32), ("block_size", ctypes.c_int32),
        ("num_splits", ctypes.c_int32), ("split_tokens", ctypes.c_int32),
        ("softmax_scale", ctypes.c_float), ("max_blocks", ctypes.c_int32),
        ("pool_pages", ctypes.c_int64), ("q", _vp), ("k_cache", _vp), ("v_cache", _vp),
        ("block_tables", _vp), ("seq_lens", _vp), ("out", _vp), ("lse", _vp), ("err", _vp),
    ]


class ScoreMod(ctypes.Structure):
    _fields_ = [("softcap", ctypes.c_float), ("window", ctypes.c_int32), ("alibi_slopes", _vp),
                ("kv_start", _vp), ("prefix_lens", _vp)]


class RopeWriteArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("dtype", "cache_q4", "num_seqs", "total_new", "num_q_heads", "num_kv_heads", "head_dim",
                 "cp", "interleave", "block_size", "max_blocks", "rope_style", "rot_dim", "reserved")] + \
               [(n, ctypes.c_int64) for n in
                ("pool_pages", "q_stride", "k_stride", "v_stride", "q_out_stride")] + \
               [(n, _vp) for n in ("q", "k", "v", "cu_new", "start_pos", "inv_freq", "block_tables",
                                   "k_cache", "v_cache", "q_out", "k_out", "err")]


class KvReadArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("out_dtype", "cache_q4", "num_seqs", "total", "num_kv_heads", "head_dim", "cp",
                 "interleave", "block_size", "max_blocks")] + \
               [("pool_pages", ctypes.c_int64)] + \
               [(n, _vp) for n in ("k_cache", "v_cache", "block_tables", "cu_out", "start_pos", "k_out",
                                   "v_out", "err")]


class CrossArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("dtype", "num_seqs", "num_q_heads", "num_kv_heads", "head_dim", "max_seqlen_q", "max_seqlen_kv",
                 "total_q", "total_kv")] + \
               [("softmax_scale", ctypes.c_float)] + \
               [(n, ctypes.c_int64) for n in ("q_stride", "k_stride", "v_stride")] + \
               [(n, _vp) for n in ("q", "k", "v", "cu_seqlens_q", "cu_seqlens_kv", "kv_lens", "key_ranges", "err")]


class BeamSelectArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("dtype", "num_seqs", "num_beams", "vocab", "num_candidates", "eos_token")] + \
               [("logits_stride", ctypes.c_int64)] + \
               [(n, _vp) for n in ("logits", "scores", "next_scores", "next_beams", "next_tokens", "cand_scores",
                                   "cand_beams", "cand_tokens")]


class BeamReorderArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("dtype", "cache_q4", "num_layers", "num_seqs", "num_beams", "num_kv_heads", "head_dim", "cp",
                 "interleave", "block_size", "max_blocks", "reserved")] + \
               [("pool_pages", ctypes.c_int64)] + \
               [(n, _vp) for n in ("parents", "seq_lens", "tables_in", "own_pages", "tables_out", "k_cache",
                                   "v_cache", "err")]


_LIB = _BINDING = None

# (name, restype, argtypes)
_SIGS = [
    ("cp_status_string", ctypes.c_char_p, [ctypes.c_int32]),
    ("cp_last_error", ctypes.c_int32, [ctypes.c_char_p, ctypes.c_size_t]),
    ("cp_last_error_detail", ctypes.c_int32, [ctypes.c_char_p, ctypes.c_size_t]),
    ("cp_abi_version", ctypes.c_int32, []),
    ("cp_prefill_args_size", ctypes.c_size_t, []),
    ("cp_decode_args_size", ctypes.c_size_t, []),
    ("cp_partition", ctypes.c_int32, [_vp, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _vp,
                                      _vp, _vp, _vp, _vp]),
    ("cp_kv_interleave_layout", ctypes.c_int32, [_vp, ctypes.c_int32, ctypes.c_int32,
                                                 ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                                 _vp, ctypes.c_int32, _vp, _vp, _vp, _vp, _vp,
                                                 _vp]),
    ("cp_kv_cache_write", ctypes.c_int32, [_vp, _vp, _vp, _vp] + [ctypes.c_int32] * 8 +
     [_vp, ctypes.c_int32, ctypes.c_int64, _vp, _vp, _vp, _vp]),
    ("cp_prefill_fused_workspace_size", ctypes.c_int32, [ctypes.POINTER(PrefillArgs),
                                                         ctypes.POINTER(ctypes.c_size_t)]),
    ("cp_attn_prefill_fused", ctypes.c_int32, [ctypes.POINTER(PrefillArgs), _vp, ctypes.c_size_t,
                                               _vp, _vp, _vp]),
    ("cp_select_prefill_mode", ctypes.c_int32, [ctypes.c_int64, ctypes.c_int64] + [ctypes.c_int32] * 4),
    ("cp_partial_attn_prefill", ctypes.c_int32, [ctypes.POINTER(PrefillArgs), _vp]),
    ("cp_decode_plan", ctypes.c_int32, [ctypes.c_int32] * 6 + [ctypes.POINTER(ctypes.c_int32)] * 2),
    ("cp_partial_attn_decode", ctypes.c_int32, [ctypes.POINTER(DecodeArgs), _vp]),
    ("cp_lse_merge", ctypes.c_int32, [_vp, _vp, ctypes.c_int32, ctypes.c_int64, ctypes.c_int32,
                                      ctypes.c_int32, _vp, ctypes.c_int32, _vp, _vp]),
    ("cp_decode_workspace_size", ctypes.c_int32, [ctypes.c_int32] * 6 + [ctypes.POINTER(ctypes.c_size_t)]),
    ("cp_decode_attention", ctypes.c_int32, [ctypes.POINTER(DecodeArgs), _vp, ctypes.c_size_t, _vp,
                                             _vp, _vp]),
    ("cp_decode_attention_noalloc", ctypes.c_int32, [ctypes.POINTER(DecodeArgs), _vp, _vp, _vp]),
    ("cp_rope_write_args_size", ctypes.c_size_t, []),
    ("cp_kv_read_args_size", ctypes.c_size_t, []),
    ("cp_score_mod_size", ctypes.c_size_t, []),
    ("cp_q4_record_bytes", ctypes.c_int64, [ctypes.c_int32]),
    ("cp_rope_kv_cache_write", ctypes.c_int32, [ctypes.POINTER(RopeWriteArgs), _vp]),
    ("cp_kv_cache_read", ctypes.c_int32, [ctypes.POINTER(KvReadArgs), _vp]),
    ("cp_attn_prefill_mod", ctypes.c_int32, [ctypes.POINTER(PrefillArgs), ctypes.POINTER(ScoreMod), _vp,
                                             _vp, _vp]),
    ("cp_decode_mod_plan", ctypes.c_int32, [ctypes.c_int32] * 7 + [ctypes.POINTER(ctypes.c_int32)] * 2),
    ("cp_cross_args_size", ctypes.c_size_t, []),
    ("cp_beam_select_args_size", ctypes.c_size_t, []),
    ("cp_beam_reorder_args_size", ctypes.c_size_t, []),
    ("cp_cross_attention_workspace_size", ctypes.c_int32, [ctypes.POINTER(CrossArgs), ctypes.POINTER(ctypes.c_size_t)]),
    ("cp_cross_attention", ctypes.c_int32, [ctypes.POINTER(CrossArgs), _vp, ctypes.c_size_t, _vp, _vp, _vp]),
    ("cp_beam_select_workspace_size", ctypes.c_int32, [ctypes.c_int32] * 4 + [ctypes.POINTER(ctypes.c_size_t)]),
    ("cp_beam_select", ctypes.c_int32, [ctypes.POINTER(BeamSelectArgs), _vp, ctypes.c_size_t, _vp]),
    ("cp_beam_reorder", ctypes.c_int32, [ctypes.POINTER(BeamReorderArgs), _vp]),
] + [(f"cp_partial_attn_decode_{n}", ctypes.c_int32,
      [ctypes.POINTER(DecodeArgs), ctypes.POINTER(ScoreMod), _vp]) for n in ("mod", "q4")] + \
    [(f"cp_decode_attention_{n}", ctypes.c_int32,
      [ctypes.POINTER(DecodeArgs), ctypes.POINTER(ScoreMod), _vp, ctypes.c_size_t, _vp, _vp, _vp])
     for n in ("mod", "q4")]

EXPORTED = [s[0] for s in _SIGS]


def lib_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = False):
    """Load libcpattn.so (built in-tree by ``__graft_entry__.build()``)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = lib_path()
    if not os.path.exists(path):
        if not build_if_missing:
            raise CPError(3, f"{path} is missing: build the CUDA library first "
                             "(python -c 'import __graft_entry__ as g; g.build()')")
        _build.build()
    lib = ctypes.CDLL(path)
    for name, res, args in _SIGS:
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if lib.cp_prefill_args_size() != ctypes.sizeof(PrefillArgs):
        raise CPError(1, "cp_prefill_args layout mismatch between binding and library")
    if lib.cp_decode_args_size() != ctypes.sizeof(DecodeArgs):
        raise CPError(1, "cp_decode_args layout mismatch between binding and library")
    for name, struct in (("cp_rope_write_args", RopeWriteArgs), ("cp_kv_read_args", KvReadArgs),
                         ("cp_score_mod", ScoreMod), ("cp_cross_args", CrossArgs),
                         ("cp_beam_select_args", BeamSelectArgs), ("cp_beam_reorder_args", BeamReorderArgs)):
        if getattr(lib, name + "_size")() != ctypes.sizeof(struct):
            raise CPError(1, f"{name} layout mismatch between binding and library")
    _LIB = lib
    return lib


def _load_binding():
    built, here = _build.binding_built_for(), _build.binding_target()
    if built != here:
        raise CPError(3, (f"{_build.BINDING} is missing" if not built else f"{_build.BINDING} was built for {built}, "
                          f"not {here}") + ": build it first (python -c 'import __graft_entry__ as g; g.build()')")
    spec = importlib.util.spec_from_file_location("cpattn_binding", _build.BINDING)
    try:
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
    except ImportError as e:
        raise CPError(3, f"{_build.BINDING} does not load: {e}") from e
    module.set_error(CPError)
    return module


def _binding():
    """The native module of the serving calls, loaded by the first of them (the other calls do without)."""
    global _BINDING
    if _BINDING is None:
        load()
        _BINDING = _load_binding()
    return _BINDING


def _check(st):
    if st != 0:
        buf = ctypes.create_string_buffer(512)
        _LIB.cp_last_error(buf, 512)
        raise CPError(st, buf.value.decode(errors="replace"))


# the current stream's handle and device without the objects around them (torch.cuda's own functions
# cost a few microseconds a call, as much as a small launch)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream=None):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        device = getattr(_CALL, "device", None)
        return _raw_stream(torch.cuda.current_device() if device is None else device.index)
    return torch.cuda.current_stream().cuda_stream


def _on(stream):
    """What a call allocates, fills and reads back belongs to the stream that it runs on: on another one a
    workspace could be cleared, or a block's last user finish, too late, and a length be read too early."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(stream.cuda_stream))


def _largest(t, stream):
    with _on(stream):
        return int(t.max().item())


def _longest(cu, stream):
    """The longest of the sequences that cu delimits."""
    with _on(stream):
        return int(cu.diff().max().item()) if cu.numel() > 1 else 0


def _ptr(t):
    return None if t is None else t.data_ptr()


_CALL = threading.local()


def _on_first_tensors_device(fn):
    """Runs an entry point with its first tensor argument's device, and the stream given, current (so
    the launch, the stream and any tensor allocated here belong to them) and makes every other tensor
    argument check that it lives on the same device."""
    at = list(inspect.signature(fn).parameters).index("stream") - 1  # among *args

    @functools.wraps(fn)
    def wrapper(first, *args, **kwargs):
        if not isinstance(first, torch.Tensor) or not first.is_cuda:
            raise CPError(1, f"{fn.__name__}: the first argument must be a CUDA tensor")
        device = first.device
        prev = getattr(_CALL, "device", None)
        _CALL.device = device
        try:
            stream = args[at] if len(args) > at else kwargs.get("stream")
            if stream is None and device.index == torch.cuda.current_device():
                return fn(first, *args, **kwargs)
            with _on(stream), torch.cuda.device(device):
                return fn(first, *args, **kwargs)
        finally:
            _CALL.device = prev
    return wrapper


def _dev(t, name, dtype=None):
    if t is None:
        return
    want = getattr(_CALL, "device", None)
    if t.device != want:
        if not t.is_cuda:
            raise CPError(1, f"{name} must be a CUDA tensor")
        if want is not None:
            raise CPError(1, f"{name} is on {t.device} but the call runs on {want}: every tensor "
                             "of one call must be on the same device")
    if not t.is_contiguous():
        raise CPError(1, f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise CPError(1, f"{name} must be {dtype} (got {t.dtype})")


def _kv_source(a, k, v, cu_seqlens_kv, dtype):
    """PASS_KV operands: k, v [Nkv, Hkv, d] and, for a cached context, cu_seqlens_kv [B + 1]."""
    _dev(k, "k", dtype)
    _dev(v, "v", dtype)
    if k is None or v is None or k.shape != v.shape:
        raise CPError(1, "PASS_KV needs k and v of the same shape [Nkv, Hkv, d]")
    a.num_kv_heads = k.shape[1]
    a.k, a.v = _ptr(k), _ptr(v)
    if cu_seqlens_kv is not None:
        _dev(cu_seqlens_kv, "cu_seqlens_kv", torch.int32)
        a.cu_seqlens_kv, a.total_kv = _ptr(cu_seqlens_kv), k.shape[0]


def _cp_dtype(t):
    if t.dtype == torch.bfloat16:
        return CP_BF16
    if t.dtype == torch.float32:
        return CP_F32
    raise CPError(2, f"unsupported dtype {t.dtype}")


# ------------------------------------------------------------------------------- entry points

@_on_first_tensors_device
def cp_partition(cu_seqlens, cp, total_tokens, perm=None, inv_perm=None, shard_offsets=None,
                 chunk_bounds=None, stream=None):
    """Load-balanced CP partition (see cpattn.h).  Returns (perm, inv_perm, shard_offsets,
    chunk_bounds) as int32 device tensors."""
    load()
    B = cu_seqlens.numel() - 1
    dev = cu_seqlens.device
    perm = torch.empty(total_tokens, dtype=torch.int32, device=dev) if perm is None else perm
    inv_perm = torch.empty(total_tokens, dtype=torch.int32, device=dev) if inv_perm is None else inv_perm
    shard_offsets = torch.empty(cp + 1, dtype=torch.int32, device=dev) if shard_offsets is None else shard_offsets
    chunk_bounds = torch.empty(B, 2 * cp + 1, dtype=torch.int32, device=dev) if chunk_bounds is None else chunk_bounds
    for n, t in (("cu_seqlens", cu_seqlens), ("perm", perm), ("inv_perm", inv_perm),
                 ("shard_offsets", shard_offsets), ("chunk_bounds", chunk_bounds)):
        _dev(t, n, torch.int32)
    _check(_LIB.cp_partition(_ptr(cu_seqlens), B, total_tokens, cp, _ptr(perm), _ptr(inv_perm),
                             _ptr(shard_offsets), _ptr(chunk_bounds), _stream(stream)))
    return perm, inv_perm, shard_offsets, chunk_bounds


@_on_first_tensors_device
def cp_kv_interleave_layout(cu_seq_lens, cp, interleave, total_tokens, block_size=16,
                            block_tables=None, local_lens=None, rank_of_token=None,
                            local_of_token=None, slot_of_token=None, want_slots=True, err=None,
                            stream=None):
    """Round-robin kv placement (see cpattn.h).  Returns (local_lens [cp, B], rank_of_token,
    local_of_token, slot_of_token-or-None)."""
    load()
    B = cu_seq_lens.numel() - 1
    dev = cu_seq_lens.device
    if local_lens is None:
        local_lens = torch.empty(cp, B, dtype=torch.int32, device=dev)
    if rank_of_token is None:
        rank_of_token = torch.empty(total_tokens, dtype=torch.int32, device=dev)
    if local_of_token is None:
        local_of_token = torch.empty(total_tokens, dtype=torch.int32, device=dev)
    if slot_of_token is None and want_slots and block_tables is not None:
        slot_of_token = torch.empty(total_tokens, dtype=torch.int64, device=dev)
    max_blocks = block_tables.shape[-1] if block_tables is not None else 0
    _dev(cu_seq_lens, "cu_seq_lens", torch.int32)
    _dev(block_tables, "block_tables", torch.int32)
    _check(_LIB.cp_kv_interleave_layout(
        _ptr(cu_seq_lens), B, total_tokens, cp, interleave, block_size, _ptr(block_tables),
        max_blocks, _ptr(local_lens), _ptr(rank_of_token), _ptr(local_of_token),
        _ptr(slot_of_token), _ptr(err), _stream(stream)))
    return local_lens, rank_of_token, local_of_token, slot_of_token


@_on_first_tensors_device
def cp_kv_cache_write(k_new, v_new, cu_new, start_pos, k_cache, v_cache, block_tables, cp,
                      interleave, err=None, stream=None):
    """Store new K/V rows [N, Hkv, d] into the per-rank pools [cp, pool, Hkv, bs, d] at their
    round-robin slots (see cpattn.h)."""
    load()
    N, Hkv, d = k_new.shape
    B = cu_new.numel() - 1
    for n, t, dt in (("k_new", k_new, None), ("v_new", v_new, k_new.dtype),
                     ("cu_new", cu_new, torch.int32), ("start_pos", start_pos, torch.int32),
                     ("k_cache", k_cache, k_new.dtype), ("v_cache", v_cache, k_new.dtype),
                     ("block_tables", block_tables, torch.int32)):
        _dev(t, n, dt)
    _check(_LIB.cp_kv_cache_write(_ptr(k_new), _ptr(v_new), _ptr(cu_new), _ptr(start_pos), B, N,
                                  Hkv, d, _cp_dtype(k_new), cp, interleave, k_cache.shape[3],
                                  _ptr(block_tables), block_tables.shape[-1], k_cache.shape[1],
                                  _ptr(k_cache), _ptr(v_cache), _ptr(err), _stream(stream)))


def cp_select_prefill_mode(q_len, kv_len, num_q_heads, num_kv_heads, head_dim, elem_bytes=2):
    """CP_PASS_KV or CP_PASS_Q: the mode measured faster on one GB300 for the nearest shape of a
    (q_len, kv_len, q heads per kv head) grid (see cpattn.h)."""
    load()
    return _LIB.cp_select_prefill_mode(q_len, kv_len, num_q_heads, num_kv_heads, head_dim,
                                       elem_bytes)


@_on_first_tensors_device
def cp_partial_attn_prefill(q, cu_seqlens_q, cp, *, mode=CP_PASS_KV, k=None, v=None,
                            cu_seqlens_kv=None, k_cache=None, v_cache=None, block_tables=None,
                            seq_lens_kv=None, interleave=8, max_seqlen_q=None, softmax_scale=0.0,
                            impl=CP_IMPL_AUTO, q_shard=-1, kv_shard=-1, out=None, lse=None,
                            err=None, debug=0, stream=None):
    """Partial attention of every (Q shard, KV shard) pair (see cpattn.h).

    q: [Nq, Hq, d].  PASS_KV: k, v [Nkv, Hkv, d]; with cu_seqlens_kv (int32 [B + 1]) each
    sequence's queries are the last of its kv tokens (a cached context before them), else
    Nkv = Nq and q, k, v share cu_seqlens_q.  PASS_Q: k_cache/v_cache [cp, pool, Hkv, 16, d],
    block_tables int32 [cp, B, max_blocks], seq_lens_kv int32 [B].
    Returns (out [cp, Nq, Hq, d] f32, lse [cp, Nq, Hq] f32).
    """
    load()
    Nq, Hq, d = q.shape
    B = cu_seqlens_q.numel() - 1
    dev = q.device
    if out is None:
        out = torch.empty(cp, Nq, Hq, d, dtype=torch.float32, device=dev)
    if lse is None:
        lse = torch.empty(cp, Nq, Hq, dtype=torch.float32, device=dev)
    a = PrefillArgs()
    a.mode, a.dtype, a.impl = mode, _cp_dtype(q), impl
    a.num_seqs, a.num_q_heads, a.head_dim, a.cp = B, Hq, d, cp
    a.softmax_scale = softmax_scale
    a.total_q = Nq
    a.q_shard, a.kv_shard = q_shard, kv_shard
    a.debug = debug
    _dev(q, "q")
    _dev(cu_seqlens_q, "cu_seqlens_q", torch.int32)
    _dev(out, "out", torch.float32)
    _dev(lse, "lse", torch.float32)
    if max_seqlen_q is None:
        max_seqlen_q = int((cu_seqlens_q[1:] - cu_seqlens_q[:-1]).max().item()) if B else 0
    a.max_seqlen_q = max_seqlen_q
    a.cu_seqlens_q, a.q, a.out, a.lse, a.err = _ptr(cu_seqlens_q), _ptr(q), _ptr(out), _ptr(lse), _ptr(err)
    if mode == CP_PASS_KV:
        _kv_source(a, k, v, cu_seqlens_kv, q.dtype)
    else:
        _dev(k_cache, "k_cache", q.dtype)
        _dev(v_cache, "v_cache", q.dtype)
        _dev(block_tables, "block_tables", torch.int32)
        _dev(seq_lens_kv, "seq_lens_kv", torch.int32)
        a.num_kv_heads = k_cache.shape[2]
        a.k_cache, a.v_cache = _ptr(k_cache), _ptr(v_cache)
        a.pool_pages = k_cache.shape[1]
        a.block_tables, a.max_blocks = _ptr(block_tables), block_tables.shape[-1]
        a.block_size, a.interleave = k_cache.shape[3], interleave
        a.seq_lens_kv = _ptr(seq_lens_kv)
    _check(_LIB.cp_partial_attn_prefill(ctypes.byref(a), _stream(stream)))
    return out, lse


@_on_first_tensors_device
def cp_attn_prefill_fused(q, cu_seqlens_q, cp, k=None, v=None, *, mode=CP_PASS_KV,
                          cu_seqlens_kv=None, k_cache=None, v_cache=None, block_tables=None,
                          seq_lens_kv=None, interleave=8, max_seqlen_q=None, softmax_scale=0.0,
                          impl=CP_IMPL_AUTO, workspace=None, out=None, out_lse=None,
                          stream=None):
    """Prefill with the merge folded in (see cpattn.h): exact causal attention out [Nq, Hq, d]
    bf16 and lse [Nq, Hq] f32 without partials.  PASS_KV: k, v [Nkv, Hkv, d] (cu_seqlens_kv as
    in cp_partial_attn_prefill).  PASS_Q: the paged round-robin cache as in
    cp_partial_attn_prefill (every rank's resident tokens in one pass); `workspace` (uint8
    CUDA tensor of cp_prefill_fused_workspace_size() bytes) lets it split the tail wave's
    items by rank range; None allocates it, an empty tensor runs every item whole."""
    load()
    Nq, Hq, d = q.shape
    B = cu_seqlens_q.numel() - 1
    if out is None:
        out = torch.empty(Nq, Hq, d, dtype=torch.bfloat16, device=q.device)
    if out_lse is None:
        out_lse = torch.empty(Nq, Hq, dtype=torch.float32, device=q.device)
    for n, t, dt in (("q", q, torch.bfloat16), ("cu_seqlens_q", cu_seqlens_q, torch.int32),
                     ("out", out, torch.bfloat16), ("out_lse", out_lse, torch.float32)):
        _dev(t, n, dt)
    if max_seqlen_q is None:
        max_seqlen_q = int((cu_seqlens_q[1:] - cu_seqlens_q[:-1]).max().item()) if B else 0
    a = PrefillArgs()
    a.mode, a.dtype, a.impl = mode, CP_BF16, impl
    a.num_seqs, a.num_q_heads, a.head_dim, a.cp = B, Hq, d, cp
    a.softmax_scale, a.total_q, a.max_seqlen_q = softmax_scale, Nq, max_seqlen_q
    a.q_shard = a.kv_shard = -1
    a.cu_seqlens_q, a.q = _ptr(cu_seqlens_q), _ptr(q)
    if mode == CP_PASS_KV:
        _kv_source(a, k, v, cu_seqlens_kv, torch.bfloat16)
    else:
        for n, t, dt in (("k_cache", k_cache, torch.bfloat16), ("v_cache", v_cache, torch.bfloat16),
                         ("block_tables", block_tables, torch.int32),
                         ("seq_lens_kv", seq_lens_kv, torch.int32)):
            _dev(t, n, dt)
        a.num_kv_heads = k_cache.shape[2]
        a.k_cache, a.v_cache = _ptr(k_cache), _ptr(v_cache)
        a.pool_pages = k_cache.shape[1]
        a.block_tables, a.max_blocks = _ptr(block_tables), block_tables.shape[-1]
        a.block_size, a.interleave = k_cache.shape[3], interleave
        a.seq_lens_kv = _ptr(seq_lens_kv)
    if workspace is None:
        need = ctypes.c_size_t()
        _check(_LIB.cp_prefill_fused_workspace_size(ctypes.byref(a), ctypes.byref(need)))
        workspace = torch.empty(need.value, dtype=torch.uint8, device=q.device)
    _dev(workspace, "workspace")
    ws, ws_bytes = (_ptr(workspace), workspace.numel()) if workspace.numel() else (None, 0)
    _check(_LIB.cp_attn_prefill_fused(ctypes.byref(a), ws, ws_bytes, _ptr(out), _ptr(out_lse),
                                      _stream(stream)))
    return out, out_lse


def cp_prefill_fused_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, cp,
                                    max_seqlen_q, *, mode=CP_PASS_Q, impl=CP_IMPL_AUTO):
    """Bytes of workspace cp_attn_prefill_fused splits its tail wave with on the current device
    (0: no split for these shapes)."""
    load()
    a = PrefillArgs()
    a.mode, a.dtype, a.impl = mode, CP_BF16, impl
    a.num_seqs, a.num_q_heads, a.num_kv_heads, a.head_dim, a.cp = (
        num_seqs, num_q_heads, num_kv_heads, head_dim, cp)
    a.max_seqlen_q, a.q_shard, a.kv_shard = max_seqlen_q, -1, -1
    need = ctypes.c_size_t()
    _check(_LIB.cp_prefill_fused_workspace_size(ctypes.byref(a), ctypes.byref(need)))
    return need.value


def cp_decode_plan(num_seqs, num_kv_heads, cp, interleave, block_size, max_seq_len):
    """(num_splits, split_tokens) for cp_partial_attn_decode."""
    load()
    ns, st = ctypes.c_int32(), ctypes.c_int32()
    _check(_LIB.cp_decode_plan(num_seqs, num_kv_heads, cp, interleave, block_size, max_seq_len,
                               ctypes.byref(ns), ctypes.byref(st)))
    return ns.value, st.value


@_on_first_tensors_device
def cp_partial_attn_decode(q, k_cache, v_cache, block_tables, seq_lens, cp, interleave, *,
                           max_seq_len=None, num_splits=None, split_tokens=None, softmax_scale=0.0,
                           out=None, lse=None, err=None, stream=None):
    """Per-(rank, split) decode partials (see cpattn.h).  Returns (out [P, B, Hq, d], lse [P, B, Hq])
    with P = cp * num_splits."""
    load()
    B, Hq, d = q.shape
    Hkv, bs = k_cache.shape[2], k_cache.shape[3]
    if num_splits is None or split_tokens is None:
        if max_seq_len is None:
            max_seq_len = int(seq_lens.max().item())
        num_splits, split_tokens = cp_decode_plan(B, Hkv, cp, interleave, bs, max_seq_len)
    P = cp * num_splits
    if out is None:
        out = torch.empty(P, B, Hq, d, dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty(P, B, Hq, dtype=torch.float32, device=q.device)
    for n, t, dt in (("q", q, None), ("k_cache", k_cache, q.dtype), ("v_cache", v_cache, q.dtype),
                     ("block_tables", block_tables, torch.int32), ("seq_lens", seq_lens, torch.int32),
                     ("out", out, torch.float32), ("lse", lse, torch.float32)):
        _dev(t, n, dt)
    a = DecodeArgs()
    a.dtype, a.num_seqs, a.num_q_heads, a.num_kv_heads, a.head_dim = _cp_dtype(q), B, Hq, Hkv, d
    a.cp, a.interleave, a.block_size = cp, interleave, bs
    a.num_splits, a.split_tokens, a.softmax_scale = num_splits, split_tokens, softmax_scale
    a.max_blocks, a.pool_pages = block_tables.shape[-1], k_cache.shape[1]
    a.q, a.k_cache, a.v_cache = _ptr(q), _ptr(k_cache), _ptr(v_cache)
    a.block_tables, a.seq_lens, a.out, a.lse, a.err = (_ptr(block_tables), _ptr(seq_lens), _ptr(out),
                                                       _ptr(lse), _ptr(err))
    _check(_LIB.cp_partial_attn_decode(ctypes.byref(a), _stream(stream)))
    return out, lse


def _decode_args(q, k_cache, v_cache, block_tables, seq_lens, cp, interleave, num_splits,
                 split_tokens, softmax_scale, out, lse, err):
    B, Hq, d = q.shape
    for n, t, dt in (("q", q, None), ("k_cache", k_cache, q.dtype), ("v_cache", v_cache, q.dtype),
                     ("block_tables", block_tables, torch.int32), ("seq_lens", seq_lens, torch.int32)):
        _dev(t, n, dt)
    a = DecodeArgs()
    a.dtype, a.num_seqs, a.num_q_heads, a.num_kv_heads, a.head_dim = _cp_dtype(q), B, Hq, k_cache.shape[2], d
    a.cp, a.interleave, a.block_size = cp, interleave, k_cache.shape[3]
    a.num_splits, a.split_tokens, a.softmax_scale = num_splits, split_tokens, softmax_scale
    a.max_blocks, a.pool_pages = block_tables.shape[-1], k_cache.shape[1]
    a.q, a.k_cache, a.v_cache = _ptr(q), _ptr(k_cache), _ptr(v_cache)
    a.block_tables, a.seq_lens, a.out, a.lse, a.err = (_ptr(block_tables), _ptr(seq_lens), _ptr(out),
                                                       _ptr(lse), _ptr(err))
    return a


def cp_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, cp, num_splits):
    """Bytes of scratch cp_decode_attention needs."""
    load()
    n = ctypes.c_size_t()
    _check(_LIB.cp_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, cp,
                                         num_splits, ctypes.byref(n)))
    return n.value


@_on_first_tensors_device
def cp_decode_attention(q, k_cache, v_cache, block_tables, seq_lens, cp, interleave, *,
                        max_seq_len=None, num_splits=None, split_tokens=None, softmax_scale=0.0,
                        workspace=None, out=None, out_lse=None, want_lse=True, err=None,
                        stream=None):
    """Decode partials + merge in one launch (see cpattn.h).  `workspace` is a zero-filled
    uint8 CUDA tensor of at least cp_decode_workspace_size() bytes; it is left reusable.
    Returns (out [B, Hq, d] dtype of q, lse [B, Hq] f32 or None)."""
    load()
    B, Hq, d = q.shape
    Hkv, bs = k_cache.shape[2], k_cache.shape[3]
    if num_splits is None or split_tokens is None:
        if max_seq_len is None:
            max_seq_len = int(seq_lens.max().item())
        num_splits, split_tokens = cp_decode_plan(B, Hkv, cp, interleave, bs, max_seq_len)
    need = cp_decode_workspace_size(B, Hq, Hkv, d, cp, num_splits)
    if workspace is None:
        workspace = torch.zeros(need, dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty(B, Hq, d, dtype=q.dtype, device=q.device)
    if out_lse is None and want_lse:
        out_lse = torch.empty(B, Hq, dtype=torch.float32, device=q.device)
    _dev(workspace, "workspace")
    _dev(out, "out", q.dtype)
    _dev(out_lse, "out_lse", torch.float32)
    a = _decode_args(q, k_cache, v_cache, block_tables, seq_lens, cp, interleave, num_splits,
                     split_tokens, softmax_scale, None, None, err)
    _check(_LIB.cp_decode_attention(ctypes.byref(a), _ptr(workspace), workspace.numel(), _ptr(out),
                                    _ptr(out_lse), _stream(stream)))
    return out, out_lse


NOALLOC_SCRATCH_BYTES = 48 * 1024 * 1024


@_on_first_tensors_device
def cp_decode_attention_noalloc(q, k_cache, v_cache, block_tables, seq_lens, cp, interleave,
                                out, *, num_splits, split_tokens, softmax_scale=0.0, out_lse=None,
                                err=None, stream=None):
    """cp_decode_attention for callers that cannot allocate device memory at call time.

    Scratch comes from a 48 MiB array built into the library (one per GPU, kept until the
    process exits), so neither this function nor the library allocates: the caller passes
    `out` ([B, Hq, d], dtype of q) and optionally `out_lse` ([B, Hq] f32), and the split plan
    explicitly (cp_decode_plan gives one).  Sizes that need more scratch than the array holds
    raise CPError (CP_ERR_INVALID_ARG).  Calls share the array, so calls that overlap on the GPU
    race; the first call on a device resolves the array's address and should come before any
    stream capture.
    """
    load()
    _dev(out, "out", q.dtype)
    _dev(out_lse, "out_lse", torch.float32)
    a = _decode_args(q, k_cache, v_cache, block_tables, seq_lens, cp, interleave, num_splits,
                     split_tokens, softmax_scale, None, None, err)
    _check(_LIB.cp_decode_attention_noalloc(ctypes.byref(a), _ptr(out), _ptr(out_lse),
                                            _stream(stream)))
    return out, out_lse


@_on_first_tensors_device
def cp_lse_merge(partial_out, partial_lse, out=None, out_dtype=torch.bfloat16, out_lse=None,
                 want_lse=True, stream=None):
    """Merge partials [P, rows, H, d] / [P, rows, H] into out [rows, H, d] (+ lse [rows, H])."""
    load()
    P, rows, H, d = partial_out.shape
    if out is None:
        out = torch.empty(rows, H, d, dtype=out_dtype, device=partial_out.device)
    if out_lse is None and want_lse:
        out_lse = torch.empty(rows, H, dtype=torch.float32, device=partial_out.device)
    _dev(partial_out, "partial_out", torch.float32)
    _dev(partial_lse, "partial_lse", torch.float32)
    _dev(out, "out")
    _dev(out_lse, "out_lse", torch.float32)
    _check(_LIB.cp_lse_merge(_ptr(partial_out), _ptr(partial_lse), P, rows, H, d, _ptr(out),
                             _cp_dtype(out), _ptr(out_lse), _stream(stream)))
    return out, out_lse


# ---------------------------------------------------------- rotation, 4-bit cache, modified scores

def cp_q4_record_bytes(head_dim):
    """Bytes of one record of the 4-bit cache (one kv head's 16 tokens): 9 * head_dim."""
    load()
    return _LIB.cp_q4_record_bytes(head_dim)


_TYPE = {None: -1, torch.float32: CP_F32, torch.bfloat16: CP_BF16}


def _handle(stream):
    return None if stream is None else stream.cuda_stream


def _on_gpu(name, first):
    if not isinstance(first, torch.Tensor) or not first.is_cuda:
        raise CPError(1, f"{name}: the first argument must be a CUDA tensor")


def cp_rope_kv_cache_write(k_new, v_new, cu_new, start_pos, k_cache, v_cache, block_tables, cp,
                           interleave, *, inv_freq=None, rope_style=CP_ROPE_HALF, q=None, q_out=None,
                           k_out=None, err=None, stream=None):
    """Append new K/V rows [N, Hkv, d] to the per-rank pools at their round-robin slots with the
    rotary embedding applied on the way, and rotate the queries q [N, Hq, d] (see cpattn.h).

    The pools are [cp, pool, Hkv, 16, d] of the rows' dtype, or uint8 [cp, pool, Hkv, 9 d] (4-bit
    records).  inv_freq: float64 CUDA tensor [rot_dim / 2] of radians per position (None: no
    rotation).  k_new, v_new and q may be column slices of a wider tensor (any token stride).
    q_out may be q.  Returns (q_out or None, k_out or None); k_out is written only if given."""
    return _binding().rope_write(k_new, v_new, cu_new, start_pos, k_cache, v_cache, block_tables, cp, interleave,
                                 inv_freq, rope_style, q, q_out, k_out, err, _handle(stream))


def cp_kv_cache_read(k_cache, v_cache, cu_out, start_pos, block_tables, cp, interleave, *, total=None,
                     out_dtype=None, k_out=None, v_out=None, err=None, stream=None):
    """Positions start_pos[b] + i of every sequence from the paged round-robin cache to contiguous
    rows cu_out[b] + i of k_out, v_out [N, Hkv, d] (see cpattn.h): the K/V of a pass-KV prefill over
    a cached context.  4-bit records (uint8 pools) come back as the values they stand for, in
    out_dtype (bf16 or f32; the pools' own dtype otherwise).  total: N, when cu_out[B] is not to be
    fetched from the device.  Returns (k_out, v_out)."""
    binding = _binding()
    if total is None:
        _on_gpu("cp_kv_cache_read", k_cache)
        total = -1 if k_out is not None else _largest(cu_out[-1:], stream)
    if out_dtype not in _TYPE:
        raise CPError(2, f"unsupported dtype {out_dtype}")
    return binding.kv_read(k_cache, v_cache, cu_out, start_pos, block_tables, cp, interleave, total,
                           _TYPE[out_dtype], k_out, v_out, err, _handle(stream))


def cp_attn_prefill_mod(q, cu_seqlens_q, k, v, *, cu_seqlens_kv=None, softcap=0.0, window=0,
                        alibi_slopes=None, kv_start=None, prefix_lens=None, max_seqlen_q=None,
                        softmax_scale=0.0, out=None, out_lse=None, err=None, stream=None):
    """Prefill attention with modified scores over contiguous k, v [Nkv, Hkv, d] (see cpattn.h): a
    tanh cap, a distance bias alibi_slopes f32 [Hq], a sliding window, kv_start int32 [Nq] (first
    visible position of each row: its document) and prefix_lens int32 [B] (keys that every query whose
    window and document reach them sees).
    bf16.  Returns (out [Nq, Hq, d] bf16, lse [Nq, Hq] f32)."""
    binding = _binding()
    if max_seqlen_q is None:
        _on_gpu("cp_attn_prefill_mod", q)
        max_seqlen_q = _longest(cu_seqlens_q, stream)
    return binding.prefill(q, cu_seqlens_q, k, v, cu_seqlens_kv, softcap, window, alibi_slopes, kv_start, prefix_lens,
                           max_seqlen_q, softmax_scale, out, out_lse, err, _handle(stream))


def cp_decode_mod_plan(num_seqs, num_kv_heads, cp, interleave, max_seq_len, *, window=0, q4=False):
    """(num_splits, split_tokens) for the decode calls with modified scores or a 4-bit cache."""
    load()
    ns, st = ctypes.c_int32(), ctypes.c_int32()
    _check(_LIB.cp_decode_mod_plan(num_seqs, num_kv_heads, cp, interleave, max_seq_len, window, q4,
                                   ctypes.byref(ns), ctypes.byref(st)))
    return ns.value, st.value


def _splits(q, seq_lens, max_seq_len, num_splits, split_tokens, stream):
    """(longest sequence to plan for or 0, num_splits, split_tokens) of a decode call's arguments."""
    if num_splits is not None and split_tokens is not None:
        return 0, num_splits, split_tokens
    if max_seq_len is None:
        _on_gpu("decode", q)
        max_seq_len = max(1, _largest(seq_lens, stream))
    return max_seq_len, 0, 0


def cp_partial_attn_decode_mod(q, k_cache, v_cache, block_tables, seq_lens, cp, interleave, *,
                               softcap=0.0, window=0, alibi_slopes=None, kv_start=None,
                               max_seq_len=None, num_splits=None, split_tokens=None,
                               softmax_scale=0.0, out=None, lse=None, err=None, stream=None):
    """cp_partial_attn_decode with modified scores (see cpattn.h): a tanh cap, a sliding window, a
    distance bias alibi_slopes f32 [Hq] and kv_start int32 [B] (first visible position).
    Returns (out [P, B, Hq, d], lse [P, B, Hq]), P = cp * num_splits."""
    binding = _binding()
    longest, num_splits, split_tokens = _splits(q, seq_lens, max_seq_len, num_splits, split_tokens, stream)
    return binding.decode_partial(False, q, k_cache, v_cache, block_tables, seq_lens, cp, interleave, softcap,
                                  window, alibi_slopes, kv_start, longest, num_splits, split_tokens,
                                  softmax_scale, err, _handle(stream), out, lse)


def cp_decode_attention_mod(q, k_cache, v_cache, block_tables, seq_lens, cp, interleave, *,
                            softcap=0.0, window=0, alibi_slopes=None, kv_start=None,
                            max_seq_len=None, num_splits=None, split_tokens=None, softmax_scale=0.0,
                            workspace=None, out=None, out_lse=None, want_lse=True, err=None,
                            stream=None):
    """cp_decode_attention with modified scores (see cp_partial_attn_decode_mod and cpattn.h).
    Returns (out [B, Hq, d] dtype of q, lse [B, Hq] f32 or None)."""
    binding = _binding()
    longest, num_splits, split_tokens = _splits(q, seq_lens, max_seq_len, num_splits, split_tokens, stream)
    return binding.decode_fused(False, q, k_cache, v_cache, block_tables, seq_lens, cp, interleave, softcap,
                                window, alibi_slopes, kv_start, longest, num_splits, split_tokens,
                                softmax_scale, err, _handle(stream), workspace, out, out_lse, want_lse)


def cp_partial_attn_decode_q4(q, k_cache, v_cache, block_tables, seq_lens, cp, interleave, *,
                              softcap=0.0, window=0, alibi_slopes=None, kv_start=None,
                              max_seq_len=None, num_splits=None, split_tokens=None,
                              softmax_scale=0.0, out=None, lse=None, err=None, stream=None):
    """cp_partial_attn_decode over the 4-bit cache, uint8 [cp, pool, Hkv, 9 d] (see cpattn.h), bf16
    queries; scores may be modified as in cp_partial_attn_decode_mod."""
    binding = _binding()
    longest, num_splits, split_tokens = _splits(q, seq_lens, max_seq_len, num_splits, split_tokens, stream)
    return binding.decode_partial(True, q, k_cache, v_cache, block_tables, seq_lens, cp, interleave, softcap,
                                  window, alibi_slopes, kv_start, longest, num_splits, split_tokens,
                                  softmax_scale, err, _handle(stream), out, lse)


def cp_decode_attention_q4(q, k_cache, v_cache, block_tables, seq_lens, cp, interleave, *,
                           softcap=0.0, window=0, alibi_slopes=None, kv_start=None,
                           max_seq_len=None, num_splits=None, split_tokens=None, softmax_scale=0.0,
                           workspace=None, out=None, out_lse=None, want_lse=True, err=None,
                           stream=None):
    """cp_decode_attention over the 4-bit cache, uint8 [cp, pool, Hkv, 9 d] (see cpattn.h), bf16
    queries; scores may be modified as in cp_partial_attn_decode_mod."""
    binding = _binding()
    longest, num_splits, split_tokens = _splits(q, seq_lens, max_seq_len, num_splits, split_tokens, stream)
    return binding.decode_fused(True, q, k_cache, v_cache, block_tables, seq_lens, cp, interleave, softcap,
                                window, alibi_slopes, kv_start, longest, num_splits, split_tokens,
                                softmax_scale, err, _handle(stream), workspace, out, out_lse, want_lse)


# ---------------------------------------------------------- cross attention, beam search

def cp_cross_attention_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, max_seqlen_q, max_seqlen_kv, *,
                                      total_q=None, total_kv=None, padded=False, dtype=torch.bfloat16):
    """Bytes of workspace with which cp_cross_attention cuts the keys of these sizes into parts on the current
    device (0: it needs none).  total_q, total_kv: rows of q and of k (num_seqs of the longest, if not given); padded:
    the call gets kv_lens or key_ranges (the most that calls with either or both take).  Other sizes, smaller ones
    too, may be cut into more."""
    load()
    a = CrossArgs()
    if dtype not in (torch.bfloat16, torch.float32):
        raise CPError(2, f"unsupported dtype {dtype}")
    a.dtype, a.num_seqs, a.head_dim = _TYPE[dtype], num_seqs, head_dim
    a.num_q_heads, a.num_kv_heads = num_q_heads, num_kv_heads
    a.max_seqlen_q, a.max_seqlen_kv = max_seqlen_q, max_seqlen_kv
    a.total_q = num_seqs * max_seqlen_q if total_q is None else total_q
    a.total_kv = num_seqs * max_seqlen_kv if total_kv is None else total_kv
    most, need = 0, ctypes.c_size_t()
    for lens, ranges in ((1, None), (None, 1), (1, 1)) if padded else ((None, None),):
        a.kv_lens, a.key_ranges = lens, ranges       # (whether there are any is all that counts here)
        _check(_LIB.cp_cross_attention_workspace_size(ctypes.byref(a), ctypes.byref(need)))
        most = max(most, need.value)
    return most


def cp_cross_attention(q, cu_seqlens_q, k, v, cu_seqlens_kv, *, kv_lens=None, key_ranges=None, max_seqlen_q=None,
                       max_seqlen_kv=None, softmax_scale=0.0, workspace=None, out=None, out_lse=None,
                       want_lse=True, err=None, stream=None):
    """Attention of q [Nq, Hq, d] over an encoder's states k, v [Nkv, Hkv, d], sequence by sequence (cu_seqlens_q,
    cu_seqlens_kv int32 [B + 1]), without causality (see cpattn.h).  A decode step's query rows are its beams.

    kv_lens int32 [B]: a sequence's keys are its first kv_lens[b] rows (a padded batch).  key_ranges int32
    [Nq, 2]: each row sees the keys [lo, hi) of its sequence.  q, k and v may be column slices of a wider tensor
    (any token stride).  bf16 or f32.  `workspace`: uint8 CUDA tensor of cp_cross_attention_workspace_size()
    bytes, left dirty (not the zero-filled one of other calls); None allocates it, an empty one leaves out the cuts that
    need it.  max_seqlen_q is fetched from the device if it is not given; max_seqlen_kv only guides the cut (the average is
    taken).
    Returns (out [Nq, Hq, d] dtype of q, lse [Nq, Hq] f32 or None)."""
    binding = _binding()
    if max_seqlen_q is None:
        _on_gpu("cp_cross_attention", q)
        max_seqlen_q = _longest(cu_seqlens_q, stream)
    if max_seqlen_kv is None:
        _on_gpu("cp_cross_attention", q)
        max_seqlen_kv = -(-k.shape[0] // max(1, cu_seqlens_kv.numel() - 1))
    return binding.cross(q, cu_seqlens_q, k, v, cu_seqlens_kv, kv_lens, key_ranges, max_seqlen_q, max_seqlen_kv,
                         softmax_scale, workspace, out, out_lse, want_lse, err, _handle(stream))


def cp_beam_select_workspace_size(num_seqs, num_beams, vocab, num_candidates):
    """Bytes of scratch cp_beam_select needs (zero-filled before its first use)."""
    load()
    n = ctypes.c_size_t()
    _check(_LIB.cp_beam_select_workspace_size(num_seqs, num_beams, vocab, num_candidates, ctypes.byref(n)))
    return n.value


def cp_beam_select(logits, scores, *, num_candidates=None, eos_token=-1, workspace=None, next_scores=None,
                   next_beams=None, next_tokens=None, cand_scores=None, cand_beams=None, cand_tokens=None, stream=None):
    """The best continuations of each sequence's beams: logits [B, K, vocab] (bf16 or f32, any row stride), scores
    f32 [B, K] (see cpattn.h).  num_candidates: 2 K (or what there is) if not given.  `workspace`: zero-filled uint8
    CUDA tensor of cp_beam_select_workspace_size() bytes, left reusable, for fused decodes of up to 65536 sequences x kv
    heads too; None allocates it.
    Returns (next_scores f32, next_beams, next_tokens int32 [B, K], cand_scores f32, cand_beams, cand_tokens
    int32 [B, num_candidates]): the candidates in falling order, and the first K that are not eos_token.  The new ones
    among them lie in one allocation, which lives as long as any of them; resize none of them."""
    binding = _binding()
    if num_candidates is None:
        _on_gpu("cp_beam_select", logits)
        K, V = logits.shape[-2:] if logits.dim() == 3 else (1, 1)
        num_candidates = min(2 * K, K * V)
    return binding.beam_select(logits, scores, num_candidates, eos_token, workspace, next_scores, next_beams,
                               next_tokens, cand_scores, cand_beams, cand_tokens, _handle(stream))


def cp_beam_reorder(parents, seq_lens, block_tables, own_pages, k_cache, v_cache, cp, interleave, *, tables_out=None,
                    err=None, stream=None):
    """Beam j of sequence b goes on from beam parents[b][j] (int32 [B, K]): its row of block_tables int32 [cp, B K,
    max_blocks] becomes the parent's, and the page being filled is copied to the beam's own (own_pages, shaped as
    block_tables; see cpattn.h).  seq_lens int32 [B]: tokens in the cache.  The pools are [cp, pool, Hkv, 16, d], uint8
    [cp, pool, Hkv, 9 d] (4-bit records) or several layers of either [layers, ..]; None and None: tables only.
    tables_out may be block_tables (in place).  Returns it, or new tables: a copy of block_tables where they are left as
    they are."""
    return _binding().beam_reorder(parents, seq_lens, block_tables, own_pages, k_cache, v_cache, cp, interleave,
                                   tables_out, err, _handle(stream))


def default_scale(head_dim):
    return 1.0 / math.sqrt(head_dim)
