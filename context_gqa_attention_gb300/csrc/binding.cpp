// The Python binding of the serving calls (rotate-and-append, cache read-back, 4-bit decode, attention
// with modified scores, cross attention, beam search): checks the tensors, makes the outputs, fills the C structs and calls
// libcpattn.so.  A decode step's kernels run for 5 to 10 us; the same checks and structs in Python
// (ctypes) took the host 24 us a call, here 5 to 6.5.
//
// Every tensor of one call must be on the first one's device, which the call makes current meanwhile; the
// kernels go to the stream given, else to that device's current stream.  A refusal raises
// CPError(status, detail) as the rest of the package does.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/DimVector.h>
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <cuda_runtime_api.h>
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

// The outputs of a call: those given, checked, and new ones, straight from the caching allocator (an allocation through the
// dispatcher costs the host about a microsecond, a quarter of a small call).  New ones are apart, so that who keeps the
// LSEs does not keep the rows; or `together` in one allocation, where they are small and many (the selection's six: 4.7 us
// of the host a call, 7.0 apart).
struct Outputs {
  struct One {
    const Tensor* given;
    const char* name;
    at::DimVector shape;
    at::ScalarType dtype;
    Tensor* to;
  };
  const Call& c;
  c10::SmallVector<One, 6> all;
  explicit Outputs(const Call& call) : c(call) {}
  void add(Tensor& to, const Tensor* given, const char* name, std::initializer_list<int64_t> shape, at::ScalarType dtype) {
    all.push_back({given, name, at::DimVector(shape), dtype, &to});
  }
  static size_t bytes_of(const One& o) {
    size_t n = c10::elementSize(o.dtype);
    for (const int64_t d : o.shape) n *= (size_t)d;
    return n;
  }
  // of the call's device and stream, both current
  static c10::Storage memory(size_t bytes) {
    c10::Allocator* from = c10::cuda::CUDACachingAllocator::get();
    return c10::Storage(c10::make_intrusive<c10::StorageImpl>(c10::StorageImpl::use_byte_size_t(), bytes, from->allocate(bytes), from, true));
  }
  void make(bool together) {
    size_t sum = 0;
    for (const One& o : all) {
      if (o.given == nullptr) {
        sum += (bytes_of(o) + 255) / 256 * 256;
        continue;
      }
      c.dense(*o.given, o.name, o.dtype);
      if (o.given->sizes() != at::IntArrayRef(o.shape))
        refuse(std::string(o.name) + " must be " + text(o.shape) + " (got " + text(o.given->sizes()) + ")");
      *o.to = *o.given;
    }
    c10::Storage shared;
    size_t at = 0;
    for (const One& o : all) {
      if (o.given != nullptr) continue;
      if (together && !shared) shared = memory(sum);
      Tensor t = at::detail::make_tensor<c10::TensorImpl>(together ? c10::Storage(shared) : memory(bytes_of(o)),
                                                          c10::DispatchKeySet(c10::DispatchKey::CUDA), c10::scalarTypeToTypeMeta(o.dtype));
      t.unsafeGetTensorImpl()->set_sizes_contiguous(o.shape);
      if (together) t.unsafeGetTensorImpl()->set_storage_offset((int64_t)(at / c10::elementSize(o.dtype)));
      at += (bytes_of(o) + 255) / 256 * 256;
      *o.to = std::move(t);
    }
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

// q, cu_q, k, v, cu_kv, kv_lens, key_ranges, max_seqlen_q, max_seqlen_kv, scale, workspace, out, out_lse, want_lse,
// err, stream
PyObject* cross(Args& x) {
  const Tensor& q = x.tensor("q");
  const Call c(q, "cp_cross_attention");
  const Tensor &cu = x.tensor("cu_seqlens_q"), &k = x.tensor("k"), &v = x.tensor("v"), &cu_kv = x.tensor("cu_seqlens_kv");
  const Tensor *kv_lens = x.opt("kv_lens"), *ranges = x.opt("key_ranges");
  cp_cross_args a{};
  a.max_seqlen_q = x.i32("max_seqlen_q");
  a.max_seqlen_kv = x.i32("max_seqlen_kv");
  a.softmax_scale = x.real();
  const Tensor *given = x.opt("workspace"), *out = x.opt("out"), *out_lse = x.opt("out_lse");
  const bool want_lse = x.flag("want_lse");
  const Tensor* err = x.opt("err");
  void* stream = c.stream(x);

  const at::ScalarType T = q.scalar_type();
  a.q_stride = c.token_rows(q, "q", T);
  a.k_stride = c.token_rows(k, "k", T);
  a.v_stride = c.token_rows(v, "v", T);
  const int64_t N = q.size(0), Hq = q.size(1), d = q.size(2), B = cu.numel() - 1;
  if (k.size(2) != d) refuse("k must be [Nkv, Hkv, " + std::to_string(d) + "] (got " + text(k.sizes()) + ")");
  c.shaped(v, "v", {k.size(0), k.size(1), d});
  a.dtype = dtype_of(q);
  a.num_seqs = i32(B, "the number of sequences");
  a.num_q_heads = i32(Hq, "the number of query heads");
  a.num_kv_heads = i32(k.size(1), "the number of kv heads");
  a.head_dim = i32(d, "head_dim");
  a.total_q = i32(N, "the number of rows");
  a.total_kv = i32(k.size(0), "the number of kv rows");
  a.cu_seqlens_q = c.index(&cu, "cu_seqlens_q", B + 1);
  a.cu_seqlens_kv = c.index(&cu_kv, "cu_seqlens_kv", B + 1);
  a.kv_lens = c.index(kv_lens, "kv_lens", B);
  a.key_ranges = c.index(ranges, "key_ranges", 2 * N);
  a.q = in(q);
  a.k = in(k);
  a.v = in(v);
  a.err = c.error_word(err);
  Tensor o, l;
  Outputs made(c);
  made.add(o, out, "out", {N, Hq, d}, T);
  if (out_lse != nullptr || want_lse) made.add(l, out_lse, "out_lse", {N, Hq}, at::kFloat);
  made.make(false);
  Tensor workspace;
  if (given != nullptr) {
    c.dense(*given, "workspace", at::kByte);
    workspace = *given;
  } else {
    size_t need = 0;
    check(cp_cross_attention_workspace_size(&a, &need));
    if (need > 0) workspace = at::empty({(int64_t)need}, at::TensorOptions().device(c.device).dtype(at::kByte));
  }
  const size_t bytes = workspace.defined() ? (size_t)workspace.numel() : 0;
  check(cp_cross_attention(&a, bytes ? out_of(workspace) : nullptr, bytes, out_of(o),
                           l.defined() ? static_cast<float*>(out_of(l)) : nullptr, stream));
  return pair(o, l);
}

PyObject* tuple_of(std::initializer_list<Tensor> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (r == nullptr) throw python_error();
  THPObjectPtr hold(r);
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) {
    PyObject* w = THPVariable_Wrap(t);
    if (w == nullptr) throw python_error();
    PyTuple_SET_ITEM(r, i++, w);
  }
  return hold.release();
}

// logits, scores, num_candidates, eos, workspace, the six outputs, stream
PyObject* beam_select(Args& x) {
  const Tensor& logits = x.tensor("logits");
  const Call c(logits, "cp_beam_select");
  const Tensor& scores = x.tensor("scores");
  cp_beam_select_args a{};
  a.num_candidates = x.i32("num_candidates");
  a.eos_token = x.i32("eos_token");
  const Tensor* given = x.opt("workspace");
  const Tensor *ns = x.opt("next_scores"), *nb = x.opt("next_beams"), *nt = x.opt("next_tokens"),
               *cs = x.opt("cand_scores"), *cb = x.opt("cand_beams"), *ct = x.opt("cand_tokens");
  void* stream = c.stream(x);

  dims(logits, "logits", 3, "[B, K, vocab]");
  const int64_t B = logits.size(0), K = logits.size(1), V = logits.size(2);
  // rows of one stride: beams of a sequence, and the sequences behind one another
  const int64_t stride = K > 1 ? logits.stride(1) : B > 1 ? logits.stride(0) : V;
  if (logits.numel() != 0 && ((V > 1 && logits.stride(2) != 1) || (K > 1 && B > 1 && logits.stride(0) != K * stride)))
    refuse("the rows of logits must be contiguous and equally spaced (only the row stride is free)");
  a.dtype = dtype_of(logits);
  c.dense(scores, "scores", at::kFloat);
  c.shaped(scores, "scores", {B, K});
  a.num_seqs = i32(B, "the number of sequences");
  a.num_beams = i32(K, "the number of beams");
  a.vocab = i32(V, "vocab");
  a.logits_stride = stride;
  size_t need = 0;
  check(cp_beam_select_workspace_size(a.num_seqs, a.num_beams, a.vocab, a.num_candidates, &need));
  Tensor workspace;
  if (given != nullptr) {
    c.dense(*given, "workspace", at::kByte);
    workspace = *given;
  } else {
    workspace = at::zeros({(int64_t)need}, at::TensorOptions().device(c.device).dtype(at::kByte));
  }
  const int64_t M = a.num_candidates;
  Tensor o0, o1, o2, o3, o4, o5;
  Outputs made(c);
  made.add(o0, ns, "next_scores", {B, K}, at::kFloat);
  made.add(o1, nb, "next_beams", {B, K}, at::kInt);
  made.add(o2, nt, "next_tokens", {B, K}, at::kInt);
  made.add(o3, cs, "cand_scores", {B, M}, at::kFloat);
  made.add(o4, cb, "cand_beams", {B, M}, at::kInt);
  made.add(o5, ct, "cand_tokens", {B, M}, at::kInt);
  made.make(true);
  a.logits = in(logits);
  a.scores = static_cast<const float*>(in(scores));
  a.next_scores = static_cast<float*>(out_of(o0));
  a.next_beams = static_cast<int32_t*>(out_of(o1));
  a.next_tokens = static_cast<int32_t*>(out_of(o2));
  a.cand_scores = static_cast<float*>(out_of(o3));
  a.cand_beams = static_cast<int32_t*>(out_of(o4));
  a.cand_tokens = static_cast<int32_t*>(out_of(o5));
  check(cp_beam_select(&a, out_of(workspace), (size_t)workspace.numel(), stream));
  return tuple_of({o0, o1, o2, o3, o4, o5});
}

// parents, seq_lens, tables, own_pages, k_cache, v_cache, cp, interleave, tables_out, err, stream
PyObject* beam_reorder(Args& x) {
  const Tensor& parents = x.tensor("parents");
  const Call c(parents, "cp_beam_reorder");
  const Tensor &lens = x.tensor("seq_lens"), &tables = x.tensor("block_tables"), &own = x.tensor("own_pages");
  const Tensor *kc = x.opt("k_cache"), *vc = x.opt("v_cache");
  cp_beam_reorder_args a{};
  a.cp = x.i32("cp");
  a.interleave = x.i32("interleave");
  const Tensor *out = x.opt("tables_out"), *err = x.opt("err");
  void* stream = c.stream(x);

  dims(parents, "parents", 2, "[B, K]");
  const int64_t B = parents.size(0), K = parents.size(1);
  a.parents = c.index(&parents, "parents", B * K);
  a.seq_lens = c.index(&lens, "seq_lens", B);
  c.dense(tables, "block_tables", at::kInt);
  if (tables.dim() != 3 || tables.size(0) != a.cp || tables.size(1) != B * K)
    refuse("block_tables must be [cp, B K, max_blocks] = [" + std::to_string(a.cp) + ", " + std::to_string(B * K) +
           ", ..] (got " + text(tables.sizes()) + ")");
  c.dense(own, "own_pages", at::kInt);
  if (own.sizes() != tables.sizes()) refuse("own_pages must be " + text(tables.sizes()) + " (got " + text(own.sizes()) + ")");
  const Tensor o = c.output(out, "tables_out", {tables.size(0), tables.size(1), tables.size(2)}, at::kInt);
  a.num_seqs = i32(B, "the number of sequences");
  a.num_beams = i32(K, "the number of beams");
  a.max_blocks = i32(tables.size(2), "max_blocks");
  a.num_layers = 1;
  a.block_size = 16;
  if ((kc == nullptr) != (vc == nullptr)) refuse("k_cache and v_cache go together");
  if (kc != nullptr) {
    a.cache_q4 = kc->scalar_type() == at::kByte;
    const int64_t nd = a.cache_q4 ? 4 : 5;
    if (kc->dim() != nd && kc->dim() != nd + 1)
      refuse("k_cache must be [cp, pool, Hkv, 16, d], or uint8 [cp, pool, Hkv, 9 d] (4-bit), or several layers of them "
             "[layers, ..]");
    c.dense(*kc, "k_cache", kc->scalar_type());
    c.dense(*vc, "v_cache", kc->scalar_type());
    if (vc->sizes() != kc->sizes()) refuse("v_cache must be " + text(kc->sizes()) + " (got " + text(vc->sizes()) + ")");
    const int64_t at0 = kc->dim() - nd;
    if (kc->size(at0) != a.cp || (a.cache_q4 && kc->size(-1) % 9 != 0))
      refuse("k_cache is " + text(kc->sizes()) + ": cp = " + std::to_string(a.cp) + " wants another shape");
    if (!a.cache_q4) a.dtype = dtype_of(*kc);
    a.num_layers = i32(at0 ? kc->size(0) : 1, "the number of layers");
    a.pool_pages = kc->size(at0 + 1);
    a.num_kv_heads = i32(kc->size(at0 + 2), "the number of kv heads");
    a.block_size = a.cache_q4 ? 16 : i32(kc->size(at0 + 3), "block_size");
    a.head_dim = i32(a.cache_q4 ? kc->size(-1) / 9 : kc->size(-1), "head_dim");
    a.k_cache = out_of(*kc);
    a.v_cache = out_of(*vc);
  } else {  // tables alone: any page number goes
    a.pool_pages = std::numeric_limits<int32_t>::max();
    a.num_kv_heads = 1;
    a.head_dim = 128;
  }
  a.tables_in = static_cast<const int32_t*>(in(tables));
  a.own_pages = static_cast<const int32_t*>(in(own));
  a.tables_out = static_cast<int32_t*>(out_of(o));
  a.err = c.error_word(err);
  if (out == nullptr) {  // what is left as it is (bad parents, bad lengths, further columns) holds the pages it had
    const cudaError_t e = cudaMemcpyAsync(a.tables_out, a.tables_in, (size_t)o.nbytes(), cudaMemcpyDeviceToDevice,
                                          static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) refuse(std::string("cp_beam_reorder: ") + cudaGetErrorString(e), CP_ERR_CUDA);
  }
  check(cp_beam_reorder(&a, stream));
  PyObject* r = THPVariable_Wrap(o);
  if (r == nullptr) throw python_error();
  return r;
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
    ENTRY("cross", cross, 16),
    ENTRY("beam_select", beam_select, 12),
    ENTRY("beam_reorder", beam_reorder, 11),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "cpattn_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_cpattn_binding(void) { return PyModule_Create(&module); }
