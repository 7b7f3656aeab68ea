// The Python binding of the serving calls (rotate-and-append, cache read-back, 4-bit decode, attention
// with modified scores): checks the tensors, makes the outputs, fills the C structs and calls
// libcpattn.so.  A decode step's kernels run for 5 to 10 us; the same checks and structs in Python
// (ctypes) took the host 24 us a call, here 5 to 6.5.
//
// Every tensor of one call must be on the first one's device, which the call makes current meanwhile; the
// kernels go to the stream given, else to that device's current stream.  A refusal raises
// CPError(status, detail) as the rest of the package does.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <initializer_list>
#include <limits>
#include <sstream>
#include <string>

#include "cpattn.h"

namespace {

using at::Tensor;

PyObject* g_cp_error = nullptr;  // the package's CPError

struct Refused {
  int status;
  std::string detail;
};
[[noreturn]] void refuse(const std::string& detail, int status = CP_ERR_INVALID_ARG) { throw Refused{status, detail}; }

void check(cp_status st) {
  if (st == CP_OK) return;
  char buf[512] = {0};
  cp_last_error(buf, sizeof(buf));
  refuse(buf, st);
}

std::string text(at::IntArrayRef s) {
  std::ostringstream o;
  o << s;
  return o.str();
}

// Positional arguments, taken in order.
struct Args {
  PyObject* const* a;
  Py_ssize_t n, i = 0;
  PyObject* next() {
    if (i >= n) refuse("too few arguments");
    return a[i++];
  }
  const Tensor* opt(const char* name) {
    PyObject* x = next();
    if (x == Py_None) return nullptr;
    if (!THPVariable_Check(x)) refuse(std::string(name) + " must be a tensor");
    return &THPVariable_Unpack(x);
  }
  const Tensor& tensor(const char* name) {
    const Tensor* t = opt(name);
    if (t == nullptr) refuse(std::string(name) + " must be a tensor");
    return *t;
  }
  long long integer(const char* name, long long least, long long most) {
    const long long v = PyLong_AsLongLong(next());
    if (v == -1 && PyErr_Occurred()) throw python_error();
    if (v < least || v > most) refuse(std::string(name) + " = " + std::to_string(v) + " does not fit its type");
    return v;
  }
  int32_t i32(const char* name) {
    return (int32_t)integer(name, std::numeric_limits<int32_t>::min(), std::numeric_limits<int32_t>::max());
  }
  bool flag(const char* name) { return integer(name, 0, 1) != 0; }
  float real() {
    const double v = PyFloat_AsDouble(next());
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return (float)v;
  }
};

// A call's device and stream, and the checks of its tensors.
struct Call {
  at::Device device;
  c10::cuda::CUDAGuard guard;
  mutable c10::cuda::OptionalCUDAStreamGuard on_stream;
  static const Tensor& on_gpu(const Tensor& first, const char* name) {
    if (!first.is_cuda()) refuse(std::string(name) + ": the first argument must be a CUDA tensor");
    return first;
  }
  Call(const Tensor& first, const char* name) : device(on_gpu(first, name).device()), guard(device) {}

  // The handle of the stream argument, None for the device's current stream.  One that is given is current
  // for the rest of the call: what is allocated and filled here belongs to it.
  void* stream(Args& x) const {
    PyObject* o = x.next();
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(device.index()).stream();
    void* s = PyLong_AsVoidPtr(o);
    if (s == nullptr && PyErr_Occurred()) throw python_error();
    on_stream.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(s), device.index()));
    return s;
  }

  void placed(const Tensor& t, const char* name) const {
    if (t.device() == device) return;
    if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
    refuse(std::string(name) + " is on " + t.device().str() + " but the call runs on " + device.str() +
           ": every tensor of one call must be on the same device");
  }
  void typed(const Tensor& t, const char* name, at::ScalarType dtype) const {
    if (t.scalar_type() != dtype)
      refuse(std::string(name) + " must be " + c10::toString(dtype) + " (got " + c10::toString(t.scalar_type()) + ")");
  }
  void dense(const Tensor& t, const char* name, at::ScalarType dtype) const {
    placed(t, name);
    if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
    typed(t, name, dtype);
  }
  void shaped(const Tensor& t, const char* name, std::initializer_list<int64_t> shape) const {
    const at::IntArrayRef want(shape);
    if (t.sizes() != want) refuse(std::string(name) + " must be " + text(want) + " (got " + text(t.sizes()) + ")");
  }
  // n int32
  const int32_t* index(const Tensor* t, const char* name, int64_t n) const {
    if (t == nullptr) return nullptr;
    dense(*t, name, at::kInt);
    if (t->numel() != n)
      refuse(std::string(name) + " must have " + std::to_string(n) + " entries (got " + std::to_string(t->numel()) + ")");
    return static_cast<const int32_t*>(t->const_data_ptr());
  }
  int32_t* error_word(const Tensor* t) const {
    if (t == nullptr) return nullptr;
    dense(*t, "err", at::kInt);
    if (t->numel() < 1) refuse("err must have an entry");
    return static_cast<int32_t*>(t->mutable_data_ptr());
  }
  // a [N, H, d] tensor whose heads are dense within a token; its token stride
  int64_t token_rows(const Tensor& t, const char* name, at::ScalarType dtype) const {
    placed(t, name);
    if (t.dim() != 3) refuse(std::string(name) + " must be [N, H, d]");
    typed(t, name, dtype);
    if (t.numel() != 0 && (t.stride(2) != 1 || (t.size(1) > 1 && t.stride(1) != t.size(2))))
      refuse(std::string("the heads of a token of ") + name + " must be contiguous (only the token stride is free)");
    return t.size(0) > 1 ? t.stride(0) : t.size(1) * t.size(2);
  }
  // The output given, checked, or a new one.
  Tensor output(const Tensor* given, const char* name, std::initializer_list<int64_t> shape, at::ScalarType dtype) const {
    if (given == nullptr) return at::empty(at::IntArrayRef(shape), at::TensorOptions().device(device).dtype(dtype));
    dense(*given, name, dtype);
    shaped(*given, name, shape);
    return *given;
  }
};

cp_dtype dtype_of(const Tensor& t) {
  if (t.scalar_type() == at::kBFloat16) return CP_BF16;
  if (t.scalar_type() == at::kFloat) return CP_F32;
  refuse(std::string("unsupported dtype ") + c10::toString(t.scalar_type()), CP_ERR_UNSUPPORTED);
}
int32_t i32(int64_t v, const char* what) {
  if (v > std::numeric_limits<int32_t>::max()) refuse(std::string(what) + " does not fit 32 bits");
  return (int32_t)v;
}
const void* in(const Tensor& t) { return t.const_data_ptr(); }
void* out_of(const Tensor& t) { return t.mutable_data_ptr(); }

PyObject* pair(const Tensor& a, const Tensor& b) {  // an undefined tensor is None
  THPObjectPtr x(a.defined() ? THPVariable_Wrap(a) : (Py_INCREF(Py_None), Py_None));
  THPObjectPtr y(b.defined() ? THPVariable_Wrap(b) : (Py_INCREF(Py_None), Py_None));
  if (!x || !y) throw python_error();
  PyObject* r = PyTuple_New(2);
  if (r == nullptr) throw python_error();
  PyTuple_SET_ITEM(r, 0, x.release());
  PyTuple_SET_ITEM(r, 1, y.release());
  return r;
}

// The paged pools and their tables.
struct Pool {
  bool q4;
  int32_t Hkv, block_size, max_blocks;
  int64_t pages;
};
// Hkv < 0: any number of heads; B < 0: of sequences
Pool paged(const Call& c, const Tensor& kc, const Tensor& vc, const Tensor& tables, int32_t cp, int64_t B, int64_t d,
           int64_t Hkv, at::ScalarType dtype) {
  Pool p;
  p.q4 = kc.scalar_type() == at::kByte;
  if (kc.dim() != (p.q4 ? 4 : 5))
    refuse("k_cache must be [cp, pool, Hkv, 16, d], or uint8 [cp, pool, Hkv, 9 d] (4-bit)");
  c.dense(kc, "k_cache", p.q4 ? at::kByte : dtype);
  c.dense(vc, "v_cache", kc.scalar_type());
  c.dense(tables, "block_tables", at::kInt);
  if (kc.size(0) != cp || kc.size(-1) != (p.q4 ? 9 * d : d) || (Hkv >= 0 && kc.size(2) != Hkv))
    refuse("k_cache is " + text(kc.sizes()) + ": cp = " + std::to_string(cp) + ", head_dim = " + std::to_string(d) +
           " and " + (Hkv >= 0 ? std::to_string(Hkv) : std::string("any number of")) + " kv heads want another shape");
  if (vc.sizes() != kc.sizes()) refuse("v_cache must be " + text(kc.sizes()) + " (got " + text(vc.sizes()) + ")");
  if (tables.dim() != 3 || tables.size(0) != cp || tables.size(1) != B)
    refuse("block_tables must be [cp, B, max_blocks] = [" + std::to_string(cp) + ", " + std::to_string(B) +
           ", ..] (got " + text(tables.sizes()) + ")");
  p.Hkv = i32(kc.size(2), "the number of kv heads");
  p.block_size = p.q4 ? 16 : i32(kc.size(3), "block_size");
  p.max_blocks = i32(tables.size(2), "max_blocks");
  p.pages = kc.size(1);
  return p;
}
void dims(const Tensor& t, const char* name, int64_t n, const char* want) {
  if (t.dim() != n) refuse(std::string(name) + " must be " + want);
}

// k, v, cu, start, k_cache, v_cache, tables, cp, interleave, inv_freq, style, q, q_out, k_out, err, stream
PyObject* rope_write(Args& x) {
  const Tensor &k = x.tensor("k_new"), &v = x.tensor("v_new");
  const Call c(k, "cp_rope_kv_cache_write");
  const Tensor &cu = x.tensor("cu_new"), &start = x.tensor("start_pos"), &kc = x.tensor("k_cache"),
               &vc = x.tensor("v_cache"), &tables = x.tensor("block_tables");
  cp_rope_write_args a{};
  a.cp = x.i32("cp");
  a.interleave = x.i32("interleave");
  const Tensor* inv_freq = x.opt("inv_freq");
  a.rope_style = x.i32("rope_style");
  const Tensor *q = x.opt("q"), *q_out = x.opt("q_out"), *k_out = x.opt("k_out"), *err = x.opt("err");
  void* stream = c.stream(x);

  const at::ScalarType T = k.scalar_type();
  a.k_stride = c.token_rows(k, "k_new", T);
  a.v_stride = c.token_rows(v, "v_new", T);
  const int64_t N = k.size(0), Hkv = k.size(1), d = k.size(2), B = cu.numel() - 1;
  c.shaped(v, "v_new", {N, Hkv, d});
  a.cu_new = c.index(&cu, "cu_new", B + 1);
  a.start_pos = c.index(&start, "start_pos", B);
  const Pool p = paged(c, kc, vc, tables, a.cp, B, d, Hkv, T);
  a.dtype = dtype_of(k);
  a.cache_q4 = p.q4;
  a.num_seqs = i32(B, "the number of sequences");
  a.total_new = i32(N, "the number of rows");
  a.num_kv_heads = p.Hkv;
  a.head_dim = i32(d, "head_dim");
  a.block_size = p.block_size;
  a.max_blocks = p.max_blocks;
  a.pool_pages = p.pages;
  a.k = in(k);
  a.v = in(v);
  a.block_tables = static_cast<const int32_t*>(in(tables));
  a.k_cache = out_of(kc);
  a.v_cache = out_of(vc);
  if (inv_freq != nullptr) {
    c.dense(*inv_freq, "inv_freq", at::kDouble);
    a.rot_dim = i32(2 * inv_freq->numel(), "rot_dim");
    a.inv_freq = static_cast<const double*>(in(*inv_freq));
  }
  Tensor qo, ko;
  if (q != nullptr) {
    a.q_stride = c.token_rows(*q, "q", T);
    const int64_t Hq = q->size(1);
    c.shaped(*q, "q", {N, Hq, d});
    a.num_q_heads = i32(Hq, "the number of query heads");
    if (q_out != nullptr) {
      a.q_out_stride = c.token_rows(*q_out, "q_out", T);
      c.shaped(*q_out, "q_out", {N, Hq, d});
      qo = *q_out;
    } else {
      qo = c.output(nullptr, "q_out", {N, Hq, d}, T);
      a.q_out_stride = Hq * d;
    }
    a.q = in(*q);
    a.q_out = out_of(qo);
  } else if (q_out != nullptr) {
    refuse("q_out without q");
  }
  if (k_out != nullptr) {
    ko = c.output(k_out, "k_out", {N, Hkv, d}, T);
    a.k_out = out_of(ko);
  }
  a.err = c.error_word(err);
  if (N > 0) check(cp_rope_kv_cache_write(&a, stream));
  return pair(qo, ko);
}

// k_cache, v_cache, cu, start, tables, cp, interleave, total (-1: k_out's), type (-1: k_out's or the
// cache's), k_out, v_out, err, stream
PyObject* kv_read(Args& x) {
  const Tensor& kc = x.tensor("k_cache");
  const Call c(kc, "cp_kv_cache_read");
  const Tensor &vc = x.tensor("v_cache"), &cu = x.tensor("cu_out"), &start = x.tensor("start_pos"),
               &tables = x.tensor("block_tables");
  cp_kv_read_args a{};
  a.cp = x.i32("cp");
  a.interleave = x.i32("interleave");
  int64_t total = x.integer("total", -1, std::numeric_limits<int32_t>::max());
  const int32_t type = x.i32("out_dtype");
  const Tensor *k_out = x.opt("k_out"), *v_out = x.opt("v_out"), *err = x.opt("err");
  void* stream = c.stream(x);

  const bool q4 = kc.scalar_type() == at::kByte;
  const at::ScalarType T = type >= 0           ? (type == CP_BF16 ? at::kBFloat16 : at::kFloat)
                           : k_out != nullptr ? k_out->scalar_type()
                           : q4               ? at::kBFloat16
                                              : kc.scalar_type();
  if (!q4) c.typed(kc, "the cache", T);
  if (kc.dim() < 1) refuse("k_cache must be [cp, pool, Hkv, 16, d], or uint8 [cp, pool, Hkv, 9 d] (4-bit)");
  const int64_t B = cu.numel() - 1, d = q4 ? kc.size(-1) / 9 : kc.size(-1);
  const Pool p = paged(c, kc, vc, tables, a.cp, B, d, -1, kc.scalar_type());
  a.cu_out = c.index(&cu, "cu_out", B + 1);
  a.start_pos = c.index(&start, "start_pos", B);
  if (total < 0) {
    if (k_out == nullptr) refuse("total or k_out must be given");
    dims(*k_out, "k_out", 3, "[N, Hkv, d]");
    total = k_out->size(0);
  }
  const Tensor ko = c.output(k_out, "k_out", {total, p.Hkv, d}, T), vo = c.output(v_out, "v_out", {total, p.Hkv, d}, T);
  a.out_dtype = dtype_of(ko);
  a.cache_q4 = q4;
  a.num_seqs = i32(B, "the number of sequences");
  a.total = i32(total, "total");
  a.num_kv_heads = p.Hkv;
  a.head_dim = i32(d, "head_dim");
  a.block_size = p.block_size;
  a.max_blocks = p.max_blocks;
  a.pool_pages = p.pages;
  a.k_cache = in(kc);
  a.v_cache = in(vc);
  a.block_tables = static_cast<const int32_t*>(in(tables));
  a.k_out = out_of(ko);
  a.v_out = out_of(vo);
  a.err = c.error_word(err);
  if (total > 0) check(cp_kv_cache_read(&a, stream));
  return pair(ko, vo);
}

// softcap, window, alibi_slopes, kv_start [, prefix_lens]
struct ModTensors {
  float softcap;
  int32_t window;
  const Tensor *slopes, *kv_start, *prefix;
};
ModTensors take_mod(Args& x, bool prefill) {
  ModTensors m;
  m.softcap = x.real();
  m.window = x.i32("window");
  m.slopes = x.opt("alibi_slopes");
  m.kv_start = x.opt("kv_start");
  m.prefix = prefill ? x.opt("prefix_lens") : nullptr;
  return m;
}
cp_score_mod score_mod(const Call& c, const ModTensors& m, int64_t Hq, int64_t rows, int64_t B) {
  cp_score_mod r{};
  r.softcap = m.softcap;
  r.window = m.window;
  if (m.slopes != nullptr) {
    c.dense(*m.slopes, "alibi_slopes", at::kFloat);
    c.shaped(*m.slopes, "alibi_slopes", {Hq});
    r.alibi_slopes = static_cast<const float*>(in(*m.slopes));
  }
  r.kv_start = c.index(m.kv_start, "kv_start", rows);
  r.prefix_lens = c.index(m.prefix, "prefix_lens", B);
  return r;
}

// q, cu_q, k, v, cu_kv, mod.., max_seqlen_q, scale, out, out_lse, err, stream
PyObject* prefill(Args& x) {
  const Tensor& q = x.tensor("q");
  const Call c(q, "cp_attn_prefill_mod");
  const Tensor &cu = x.tensor("cu_seqlens_q"), &k = x.tensor("k"), &v = x.tensor("v");
  const Tensor* cu_kv = x.opt("cu_seqlens_kv");
  const ModTensors mt = take_mod(x, true);
  cp_prefill_args a{};
  a.max_seqlen_q = x.i32("max_seqlen_q");
  a.softmax_scale = x.real();
  const Tensor *out = x.opt("out"), *out_lse = x.opt("out_lse"), *err = x.opt("err");
  void* stream = c.stream(x);

  dims(q, "q", 3, "[Nq, Hq, d]");
  c.dense(q, "q", at::kBFloat16);
  c.dense(k, "k", at::kBFloat16);
  c.dense(v, "v", at::kBFloat16);
  const int64_t N = q.size(0), Hq = q.size(1), d = q.size(2), B = cu.numel() - 1;
  if (k.dim() != 3 || k.sizes() != v.sizes() || k.size(2) != d || (cu_kv == nullptr && k.size(0) != N))
    refuse("k and v must be [Nkv, Hkv, " + std::to_string(d) + "] (Nkv = " + std::to_string(N) + " without cu_seqlens_kv)");
  a.mode = CP_PASS_KV;
  a.dtype = CP_BF16;
  a.impl = CP_IMPL_AUTO;
  a.num_seqs = i32(B, "the number of sequences");
  a.num_q_heads = i32(Hq, "the number of query heads");
  a.num_kv_heads = i32(k.size(1), "the number of kv heads");
  a.head_dim = i32(d, "head_dim");
  a.cp = 1;
  a.q_shard = a.kv_shard = -1;
  a.total_q = i32(N, "the number of rows");
  a.cu_seqlens_q = c.index(&cu, "cu_seqlens_q", B + 1);
  a.q = in(q);
  a.k = in(k);
  a.v = in(v);
  if (cu_kv != nullptr) {
    a.cu_seqlens_kv = c.index(cu_kv, "cu_seqlens_kv", B + 1);
    a.total_kv = i32(k.size(0), "the number of kv rows");
  }
  const cp_score_mod m = score_mod(c, mt, Hq, N, B);
  a.err = c.error_word(err);
  const Tensor o = c.output(out, "out", {N, Hq, d}, at::kBFloat16), l = c.output(out_lse, "out_lse", {N, Hq}, at::kFloat);
  check(cp_attn_prefill_mod(&a, &m, out_of(o), static_cast<float*>(out_of(l)), stream));
  return pair(o, l);
}

// What the decode calls share: q4, q, k_cache, v_cache, tables, seq_lens, cp, interleave, mod.., longest
// (0: the splits are given), splits, split_tokens, scale, err, stream
struct Decode {
  bool q4;
  const Tensor &q, &kc, &vc, &tables, &seq_lens;
  const Call c;
  cp_decode_args a{};
  ModTensors mt;
  const Tensor* err;
  void* stream;
  cp_score_mod m;
  int64_t B, Hq, d;
  Decode(Args& x, const char* name)
      : q4(x.flag("q4")), q(x.tensor("q")), kc(x.tensor("k_cache")), vc(x.tensor("v_cache")),
        tables(x.tensor("block_tables")), seq_lens(x.tensor("seq_lens")), c(q, name) {
    a.cp = x.i32("cp");
    a.interleave = x.i32("interleave");
    mt = take_mod(x, false);
    const int32_t longest = x.i32("max_seq_len");
    a.num_splits = x.i32("num_splits");
    a.split_tokens = x.i32("split_tokens");
    a.softmax_scale = x.real();
    err = x.opt("err");
    stream = c.stream(x);

    dims(q, "q", 3, "[B, Hq, d]");
    a.dtype = dtype_of(q);
    c.dense(q, "q", q.scalar_type());
    B = q.size(0), Hq = q.size(1), d = q.size(2);
    const Pool p = paged(c, kc, vc, tables, a.cp, B, d, -1, q.scalar_type());
    if (p.q4 != q4)
      refuse("uint8 pools hold 4-bit records (the *_q4 calls); the *_mod calls take pools of q's dtype");
    a.num_seqs = i32(B, "the number of sequences");
    a.num_q_heads = i32(Hq, "the number of query heads");
    a.num_kv_heads = p.Hkv;
    a.head_dim = i32(d, "head_dim");
    a.block_size = p.block_size;
    a.max_blocks = p.max_blocks;
    a.pool_pages = p.pages;
    a.q = in(q);
    a.k_cache = in(kc);
    a.v_cache = in(vc);
    a.block_tables = static_cast<const int32_t*>(in(tables));
    a.seq_lens = c.index(&seq_lens, "seq_lens", B);
    a.err = c.error_word(err);
    m = score_mod(c, mt, Hq, B, B);
    if (longest > 0)
      check(cp_decode_mod_plan(a.num_seqs, a.num_kv_heads, a.cp, a.interleave, longest, mt.window, q4, &a.num_splits,
                               &a.split_tokens));
  }
};

// Decode.., out, lse
PyObject* decode_partial(Args& x) {
  Decode t(x, "cp_partial_attn_decode");
  const Tensor *out = x.opt("out"), *lse = x.opt("lse");
  const int64_t P = (int64_t)t.a.cp * t.a.num_splits;
  if (P < 1) refuse("cp and num_splits must be at least 1");
  const Tensor o = t.c.output(out, "out", {P, t.B, t.Hq, t.d}, at::kFloat), l = t.c.output(lse, "lse", {P, t.B, t.Hq}, at::kFloat);
  t.a.out = static_cast<float*>(out_of(o));
  t.a.lse = static_cast<float*>(out_of(l));
  check((t.q4 ? cp_partial_attn_decode_q4 : cp_partial_attn_decode_mod)(&t.a, &t.m, t.stream));
  return pair(o, l);
}

// Decode.., workspace, out, out_lse, want_lse
PyObject* decode_fused(Args& x) {
  Decode t(x, "cp_decode_attention");
  const Tensor *given = x.opt("workspace"), *out = x.opt("out"), *out_lse = x.opt("out_lse");
  const bool want_lse = x.flag("want_lse");
  Tensor workspace;
  if (given != nullptr) {
    t.c.dense(*given, "workspace", at::kByte);
    workspace = *given;
  } else {
    size_t need = 0;
    check(cp_decode_workspace_size(t.a.num_seqs, t.a.num_q_heads, t.a.num_kv_heads, t.a.head_dim, t.a.cp, t.a.num_splits,
                                   &need));
    workspace = at::zeros({(int64_t)need}, at::TensorOptions().device(t.c.device).dtype(at::kByte));
  }
  const Tensor o = t.c.output(out, "out", {t.B, t.Hq, t.d}, t.q.scalar_type());
  Tensor l;
  if (out_lse != nullptr || want_lse) l = t.c.output(out_lse, "out_lse", {t.B, t.Hq}, at::kFloat);
  check((t.q4 ? cp_decode_attention_q4 : cp_decode_attention_mod)(
      &t.a, &t.m, out_of(workspace), (size_t)workspace.numel(), out_of(o),
      l.defined() ? static_cast<float*>(out_of(l)) : nullptr, t.stream));
  return pair(o, l);
}

template <PyObject* (*F)(Args&), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    Args x{args, n};
    if (n != N) refuse("expected " + std::to_string(N) + " arguments (got " + std::to_string(n) + ")");
    return F(x);
  } catch (const Refused& e) {
    THPObjectPtr a(Py_BuildValue("(is)", e.status, e.detail.c_str()));
    if (a) PyErr_SetObject(g_cp_error, a.get());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XSETREF(g_cp_error, cls);
  Py_RETURN_NONE;
}

#define ENTRY(name, f, n) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"set_error", set_error, METH_O, nullptr},
    ENTRY("rope_write", rope_write, 16),
    ENTRY("kv_read", kv_read, 13),
    ENTRY("prefill", prefill, 16),
    ENTRY("decode_partial", decode_partial, 20),
    ENTRY("decode_fused", decode_fused, 22),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "cpattn_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_cpattn_binding(void) { return PyModule_Create(&module); }
