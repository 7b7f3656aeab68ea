// The paged round-robin K/V cache's own traffic: cp_rope_kv_cache_write (rotate q and k by their
// positions and append k and v, as rows of the cache's type or as 4-bit records) and
// cp_kv_cache_read (positions of a sequence back to contiguous rows).
//
// "Add utility functions to enable pass-kv prefill and allgather decode" (vLLM PR 26059),
// Purpose: KV kept round-robin on the CP ranks; "[Feature] Prefill Context Parallel (PCP) basic
// support" (PR 28718), Purpose: per-rank block tables.
//
// Both are bound by HBM: every input row is read once, every output row written once, 16 bytes a
// thread.  A CTA owns a few consecutive tokens: it finds their sequences, positions and page slots
// once (and, when rotating, the cosines and sines of all their angles, shared by every head) in
// shared memory, and its threads then stream the tokens' rows.
#include <math.h>

#include "common.cuh"
#include "q4.cuh"

namespace cpattn {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 64;  // tokens a CTA may own

// Where a token's K and V rows live: the record index of kv head 0 (page (rank, id) of the pool
// times the kv heads) and the row within the page; head < 0: no row to touch.
struct Slot {
  long long head;
  int row;
};

// Number of sequences that end at or before `row` (the sequence of `row`, or B behind the last):
// the CTA's threads compare all ends at once, so the search costs one load latency.
CP_DEV int cta_seq_of_row(const int32_t* __restrict__ cu, int B, int row) {
  int n = 0;
  for (int b0 = 0; b0 < B; b0 += kThreads) {
    const int b = b0 + (int)threadIdx.x;
    n += __syncthreads_count(b < B && __ldg(cu + b + 1) <= row);
  }
  return n;
}

// Position and slot of token row `row` (first candidate sequence s0).  false: behind the last
// sequence.  A position without a page (negative, past the table, an id outside the pool) is
// reported and its slot left empty.
CP_DEV bool locate(const int32_t* __restrict__ cu, const int32_t* __restrict__ start, int B, int s0,
                   int row, int cp, int I, const int32_t* __restrict__ tables, int max_blocks,
                   long long pool, int Hkv, int32_t* err, long long& pos, Slot& slot) {
  slot.head = -1;
  slot.row = 0;
  int s = s0;
  while (s < B && __ldg(cu + s + 1) <= row) ++s;
  if (s >= B || row < __ldg(cu + s)) return false;
  pos = (long long)__ldg(start + s) + (row - __ldg(cu + s));
  if (pos >= 0) {
    const long long turn = pos / I, l = (turn / cp) * I + pos % I, col = l / kQ4Page;
    const int r = (int)(turn % cp);
    const int id = col < max_blocks ? __ldg(tables + ((long long)r * B + s) * max_blocks + col) : -1;
    if (id >= 0 && id < pool) {
      slot.head = (r * pool + id) * Hkv;
      slot.row = (int)(l % kQ4Page);
    }
  }
  if (slot.head < 0) report(err, CP_ERR_DEVICE_BOUNDS);
  return true;
}

// ------------------------------------------------------------------------------ 8-value pieces
template <typename T>
CP_DEV void load8(const T* p, float (&x)[8]);
template <>
CP_DEV void load8(const float* p, float (&x)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
template <>
CP_DEV void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  x[0] = bf16_lo(a.x), x[1] = bf16_hi(a.x), x[2] = bf16_lo(a.y), x[3] = bf16_hi(a.y);
  x[4] = bf16_lo(a.z), x[5] = bf16_hi(a.z), x[6] = bf16_lo(a.w), x[7] = bf16_hi(a.w);
}
CP_DEV void store8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
CP_DEV uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
CP_DEV void store8(__nv_bfloat16* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}

// ------------------------------------------------------------------------------ write
struct WriteParams {
  int B, N, T, Hq, Hkv, cp, I, max_blocks, half, rot;
  long long pool, q_stride, k_stride, v_stride, qo_stride;
  const void *q, *k, *v;
  void *q_out, *k_out;
  uint8_t *k_cache, *v_cache;
  const int32_t *cu, *start, *tables;
  const double* inv_freq;
  int32_t* err;
};

// Rotation.  The angle pos * inv_freq of a far position needs more bits than fp32 has, so it is
// kept in turns: inv_freq / 2 pi as a 64-bit fraction of a turn (one fp64 multiply per frequency),
// times the integer position modulo 2^64, which drops whole turns exactly.  The top 32 bits are
// the angle in [-1/2, 1/2) turns, off by 2^-26 turns at most after the conversion to fp32.
CP_DEV unsigned long long turns_of(double inv_freq) {
  double t = inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
  t -= floor(t);
  return __double2ull_rz(t * 18446744073709551616.0);
}

// The pieces (of 8 dims) a head's thread j handles, and whether they are rotated.  Half style: a
// piece of the first half with its partner in the second; pairs style: two neighbours.
struct Pieces {
  int c0, c1;
  bool rot;
};
CP_DEV Pieces pieces_of(int j, int rot, int half) {
  const int rp = rot >> 4;  // threads of a head whose pieces are rotated
  Pieces s;
  s.rot = j < rp;
  if (half && s.rot) {
    s.c0 = j;
    s.c1 = j + rp;
  } else {
    s.c0 = 2 * j;  // half style: 2 rp + 2 (j - rp), the pieces behind the rotated ones
    s.c1 = 2 * j + 1;
  }
  return s;
}

// Codes of one head's row by the D / 16 neighbouring threads that hold it (pieces c0, c1 each):
// per group of 64 dims the minimum rounded to bf16, the range above it / 15 rounded to bf16, and
// code = nearest integer to (x - minimum) / scale, ties to even, within 0..15.  A group with an
// infinity or a NaN (or a range beyond bf16) is stored as NaN.
template <int D>
CP_DEV void quantise(const float (&a)[8], const float (&b)[8], const Pieces& s, uint8_t* rec, int row,
                     int j, bool live) {
  constexpr int GR = D / kQ4Group, LPH = D / 16;
  float mna = a[0], mxa = a[0], mnb = b[0], mxb = b[0];
  bool bad_a = false, bad_b = false;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    mna = fminf(mna, a[e]), mxa = fmaxf(mxa, a[e]), bad_a |= !isfinite(a[e]);
    mnb = fminf(mnb, b[e]), mxb = fmaxf(mxb, b[e]), bad_b |= !isfinite(b[e]);
  }
  if (bad_a) mxa = INFINITY;  // an infinite range marks the group
  if (bad_b) mxb = INFINITY;
  float sc[GR], mn[GR];
#pragma unroll
  for (int g = 0; g < GR; ++g) {
    const bool ia = GR == 1 || (s.c0 >> 3) == g, ib = GR == 1 || (s.c1 >> 3) == g;
    float lo = fminf(ia ? mna : INFINITY, ib ? mnb : INFINITY);
    float hi = fmaxf(ia ? mxa : -INFINITY, ib ? mxb : -INFINITY);
#pragma unroll
    for (int o = 1; o < LPH; o <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    mn[g] = __bfloat162float(__float2bfloat16_rn(lo));
    sc[g] = __bfloat162float(__float2bfloat16_rn((hi - mn[g]) / 15.f));
    if (!(isfinite(mn[g]) && isfinite(sc[g]))) {
      mn[g] = NAN;
      sc[g] = 0.f;
    }
  }
  if (!live) return;
  auto word = [&](const float (&x)[8], int c) {
    const int g = GR == 1 ? 0 : c >> 3;
    const float m = g == 0 ? mn[0] : mn[GR - 1], d = g == 0 ? sc[0] : sc[GR - 1];
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // (IEEE division: the code is the same wherever the same row is quantised)
      const float n = d > 0.f ? fminf(fmaxf(rintf((x[e] - m) / d), 0.f), 15.f) : 0.f;
      w |= (uint32_t)n << (4 * e);
    }
    reinterpret_cast<uint32_t*>(rec + row * (D / 2))[q4_word<D>(c)] = w;
  };
  word(a, s.c0);
  word(b, s.c1);
  if (j < GR) {
    const float m = j == 0 ? mn[0] : mn[GR - 1], d = j == 0 ? sc[0] : sc[GR - 1];
    reinterpret_cast<uint32_t*>(rec + 8 * D)[row * GR + j] = pack2(d, m);
  }
}

template <typename T, int D, bool Q4>
__global__ void __launch_bounds__(kThreads) rope_write_kernel(const WriteParams p) {
  constexpr int LPH = D / 16;  // threads per head, 16 dims each
  constexpr int U = 2;         // rows in flight per thread
  extern __shared__ float2 cs[];  // [T][rot / 2] cosine, sine
  __shared__ unsigned long long freq[D / 2];
  __shared__ Slot slots[kMaxTokens];
  __shared__ long long posn[kMaxTokens];  // position, or -1: no row (behind the last sequence)
  const int row0 = blockIdx.x * p.T, nt = min(p.T, p.N - row0), h = p.rot >> 1;
  const int nh = p.Hq + 2 * p.Hkv;
  if ((int)threadIdx.x < h) freq[threadIdx.x] = turns_of(p.inv_freq[threadIdx.x]);
  const int s0 = cta_seq_of_row(p.cu, p.B, row0);
  if ((int)threadIdx.x < nt) {
    const int t = threadIdx.x;
    long long pos = 0;
    const bool in = locate(p.cu, p.start, p.B, s0, row0 + t, p.cp, p.I, p.tables, p.max_blocks, p.pool,
                           p.Hkv, p.err, pos, slots[t]);
    posn[t] = in && pos >= 0 ? pos : -1ll;  // a negative position (reported): the row is skipped
  }
  __syncthreads();
  for (int i = threadIdx.x; i < nt * h; i += kThreads) {
    const int t = i / h;
    const unsigned long long f = freq[i - t * h] * (unsigned long long)posn[t];
    const float turn = (float)(int)(uint32_t)(f >> 32) * 2.3283064365386963e-10f;  // 2^-32
    float sn, c;
    sincospif(2.f * turn, &sn, &c);
    cs[i] = make_float2(c, sn);
  }
  __syncthreads();

  const int items = nt * nh * LPH;
  for (int i0 = 0; i0 < items; i0 += U * kThreads) {  // uniform: whole warps stay in the loop
    float a[U][8], b[U][8];
    int tok[U], hd[U];
    Pieces ps[U];
    const int j = threadIdx.x % LPH;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kThreads + (int)threadIdx.x;
      const unsigned unit = (unsigned)i / LPH;
      tok[u] = i < items ? (int)(unit / (unsigned)nh) : -1;
      hd[u] = (int)(unit % (unsigned)nh);
      if (tok[u] >= 0 && posn[tok[u]] < 0) tok[u] = -1;
      ps[u] = pieces_of(j, p.rot, p.half);
      if (tok[u] >= 0) {
        const long long row = row0 + tok[u];
        const T* src = hd[u] < p.Hq ? static_cast<const T*>(p.q) + row * p.q_stride + hd[u] * D
                       : hd[u] < p.Hq + p.Hkv
                           ? static_cast<const T*>(p.k) + row * p.k_stride + (hd[u] - p.Hq) * D
                           : static_cast<const T*>(p.v) + row * p.v_stride + (hd[u] - p.Hq - p.Hkv) * D;
        load8(src + 8 * ps[u].c0, a[u]);
        load8(src + 8 * ps[u].c1, b[u]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) a[u][e] = b[u][e] = 0.f;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool live = tok[u] >= 0;
      const bool is_v = hd[u] >= p.Hq + p.Hkv;
      if (live && ps[u].rot && !is_v) {
        const float2* c = cs + tok[u] * h;
        if (p.half) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 w = c[8 * ps[u].c0 + e];
            const float x = a[u][e], y = b[u][e];
            a[u][e] = x * w.x - y * w.y;
            b[u][e] = y * w.x + x * w.y;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float2 w = c[4 * ps[u].c0 + e / 2], z = c[4 * ps[u].c1 + e / 2];
            const float x = a[u][e], y = a[u][e + 1], s = b[u][e], t = b[u][e + 1];
            a[u][e] = x * w.x - y * w.y;
            a[u][e + 1] = y * w.x + x * w.y;
            b[u][e] = s * z.x - t * z.y;
            b[u][e + 1] = t * z.x + s * z.y;
          }
        }
      }
      const long long row = row0 + tok[u];
      if (live && hd[u] < p.Hq) {
        T* dst = static_cast<T*>(p.q_out) + row * p.qo_stride + hd[u] * D;
        store8(dst + 8 * ps[u].c0, a[u]);
        store8(dst + 8 * ps[u].c1, b[u]);
      }
      const int g = hd[u] - p.Hq - (is_v ? p.Hkv : 0);
      if (live && g >= 0 && !is_v && p.k_out != nullptr) {
        T* dst = static_cast<T*>(p.k_out) + (row * p.Hkv + g) * D;
        store8(dst + 8 * ps[u].c0, a[u]);
        store8(dst + 8 * ps[u].c1, b[u]);
      }
      const Slot sl = live ? slots[tok[u]] : Slot{-1, 0};
      const bool put = live && g >= 0 && sl.head >= 0;
      uint8_t* cache = is_v ? p.v_cache : p.k_cache;
      if constexpr (Q4) {
        uint8_t* rec = put ? cache + (sl.head + g) * q4_record_bytes(D) : nullptr;
        quantise<D>(a[u], b[u], ps[u], rec, sl.row, j, put);
      } else if (put) {
        T* dst = reinterpret_cast<T*>(cache) + ((sl.head + g) * kQ4Page + sl.row) * D;
        store8(dst + 8 * ps[u].c0, a[u]);
        store8(dst + 8 * ps[u].c1, b[u]);
      }
    }
  }
}

// ------------------------------------------------------------------------------ read
struct ReadParams {
  int B, N, T, Hkv, cp, I, max_blocks;
  long long pool;
  const uint8_t *k_cache, *v_cache;
  void *k_out, *v_out;
  const int32_t *cu, *start, *tables;
  int32_t* err;
};

// Rows of the cache's own type (E 16-byte vectors each) copied; U vectors in flight per thread.
template <int E>
__global__ void __launch_bounds__(kThreads) read_rows_kernel(const ReadParams p) {
  constexpr int U = 4;
  __shared__ Slot slots[kMaxTokens];
  const int row0 = blockIdx.x * p.T, nt = min(p.T, p.N - row0);
  const int s0 = cta_seq_of_row(p.cu, p.B, row0);
  if ((int)threadIdx.x < nt) {
    long long pos;
    locate(p.cu, p.start, p.B, s0, row0 + threadIdx.x, p.cp, p.I, p.tables, p.max_blocks, p.pool, p.Hkv,
           p.err, pos, slots[threadIdx.x]);
  }
  __syncthreads();
  const int items = nt * p.Hkv * 2 * E;  // token, K or V, kv head, vector
  for (int i0 = threadIdx.x; i0 < items; i0 += U * kThreads) {
    uint4 x[U];
    uint4* dst[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kThreads;
      dst[u] = nullptr;
      if (i < items) {
        const unsigned unit = (unsigned)i / E, v = (unsigned)i % E;
        const unsigned t = unit / (2u * p.Hkv), m = unit % (2u * p.Hkv);
        const int g = (int)(m >= (unsigned)p.Hkv ? m - p.Hkv : m);
        const Slot sl = slots[t];
        if (sl.head >= 0) {
          const uint8_t* cache = m >= (unsigned)p.Hkv ? p.v_cache : p.k_cache;
          x[u] = __ldg(reinterpret_cast<const uint4*>(cache) + ((sl.head + g) * kQ4Page + sl.row) * E + v);
          dst[u] = static_cast<uint4*>(m >= (unsigned)p.Hkv ? p.v_out : p.k_out) +
                   ((long long)(row0 + t) * p.Hkv + g) * E + v;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (dst[u] != nullptr) *dst[u] = x[u];
  }
}

// 4-bit rows to the values they stand for: a thread turns one word (8 codes) into 8 values.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) read_q4_kernel(const ReadParams p) {
  constexpr int U = 4, W = D / 8, GR = D / kQ4Group;
  __shared__ Slot slots[kMaxTokens];
  const int row0 = blockIdx.x * p.T, nt = min(p.T, p.N - row0);
  const int s0 = cta_seq_of_row(p.cu, p.B, row0);
  if ((int)threadIdx.x < nt) {
    long long pos;
    locate(p.cu, p.start, p.B, s0, row0 + threadIdx.x, p.cp, p.I, p.tables, p.max_blocks, p.pool, p.Hkv,
           p.err, pos, slots[threadIdx.x]);
  }
  __syncthreads();
  const int items = nt * p.Hkv * 2 * W;
  for (int i0 = threadIdx.x; i0 < items; i0 += U * kThreads) {
    uint32_t w[U], sm[U];
    T* dst[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kThreads;
      dst[u] = nullptr;
      if (i < items) {
        const unsigned unit = (unsigned)i / W;
        const int c = (int)((unsigned)i % W);  // dims 8 c ..
        const unsigned t = unit / (2u * p.Hkv), m = unit % (2u * p.Hkv);
        const int g = (int)(m >= (unsigned)p.Hkv ? m - p.Hkv : m);
        const Slot sl = slots[t];
        if (sl.head >= 0) {
          const uint8_t* rec =
              (m >= (unsigned)p.Hkv ? p.v_cache : p.k_cache) + (sl.head + g) * q4_record_bytes(D);
          w[u] = __ldg(reinterpret_cast<const uint32_t*>(rec + sl.row * (D / 2)) + q4_word<D>(c));
          sm[u] = __ldg(reinterpret_cast<const uint32_t*>(rec + 8 * D) + sl.row * GR + (GR == 1 ? 0 : c >> 3));
          dst[u] = static_cast<T*>(m >= (unsigned)p.Hkv ? p.v_out : p.k_out) +
                   ((long long)(row0 + t) * p.Hkv + g) * D + 8 * c;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (dst[u] != nullptr) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = q4_value(sm[u], (w[u] >> (4 * e)) & 15u);
        store8(dst[u], x);
      }
  }
}

// Tokens per CTA: about `want` items of work for its threads, fewer when that would leave SMs
// without a CTA (a step of 64 single tokens runs 64 CTAs of one token each).
int tokens_per_cta(long long N, long long items_per_token, long long want) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
    sms = 152;
  long long t = want / (items_per_token > 0 ? items_per_token : 1);
  const long long spread = N / (4ll * sms);  // at least ~4 CTAs per SM
  t = t < spread ? t : spread;
  return (int)(t < 1 ? 1 : (t > kMaxTokens ? kMaxTokens : t));
}

}  // namespace
}  // namespace cpattn

cudaError_t cp_launch_rope_write(const cp_rope_write_args& a, cudaStream_t s) {
  using namespace cpattn;
  WriteParams p;
  p.B = a.num_seqs;
  p.N = a.total_new;
  p.Hq = a.q != nullptr ? a.num_q_heads : 0;
  p.Hkv = a.num_kv_heads;
  p.cp = a.cp;
  p.I = a.interleave;
  p.max_blocks = a.max_blocks;
  p.half = a.rope_style == CP_ROPE_HALF;
  p.rot = a.rot_dim;
  p.pool = a.pool_pages;
  p.q_stride = a.q_stride;
  p.k_stride = a.k_stride;
  p.v_stride = a.v_stride;
  p.qo_stride = a.q_out_stride;
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  p.q_out = a.q_out;
  p.k_out = a.k_out;
  p.k_cache = static_cast<uint8_t*>(a.k_cache);
  p.v_cache = static_cast<uint8_t*>(a.v_cache);
  p.cu = a.cu_new;
  p.start = a.start_pos;
  p.tables = a.block_tables;
  p.inv_freq = a.inv_freq;
  p.err = a.err;
  p.T = tokens_per_cta(p.N, (long long)(p.Hq + 2 * p.Hkv) * (a.head_dim / 16), 1280);
  if (p.T > 16) p.T = 16;  // the angles of 16 tokens: 8 KB of shared memory
  const unsigned grid = (unsigned)((p.N + p.T - 1) / p.T);
  const size_t smem = (size_t)p.T * (p.rot / 2) * sizeof(float2);
  auto go = [&](auto kern) -> cudaError_t {
    kern<<<grid, kThreads, smem, s>>>(p);
    return cudaGetLastError();
  };
  const bool q4 = a.cache_q4 != 0, bf = a.dtype == CP_BF16;
  if (a.head_dim == 128) {
    if (bf) return q4 ? go(rope_write_kernel<__nv_bfloat16, 128, true>)
                      : go(rope_write_kernel<__nv_bfloat16, 128, false>);
    return q4 ? go(rope_write_kernel<float, 128, true>) : go(rope_write_kernel<float, 128, false>);
  }
  if (bf) return q4 ? go(rope_write_kernel<__nv_bfloat16, 64, true>)
                    : go(rope_write_kernel<__nv_bfloat16, 64, false>);
  return q4 ? go(rope_write_kernel<float, 64, true>) : go(rope_write_kernel<float, 64, false>);
}

cudaError_t cp_launch_kv_read(const cp_kv_read_args& a, cudaStream_t s) {
  using namespace cpattn;
  ReadParams p;
  p.B = a.num_seqs;
  p.N = a.total;
  p.Hkv = a.num_kv_heads;
  p.cp = a.cp;
  p.I = a.interleave;
  p.max_blocks = a.max_blocks;
  p.pool = a.pool_pages;
  p.k_cache = static_cast<const uint8_t*>(a.k_cache);
  p.v_cache = static_cast<const uint8_t*>(a.v_cache);
  p.k_out = a.k_out;
  p.v_out = a.v_out;
  p.cu = a.cu_out;
  p.start = a.start_pos;
  p.tables = a.block_tables;
  p.err = a.err;
  const int d = a.head_dim;
  const int row_bytes = d * (a.out_dtype == CP_BF16 ? 2 : 4);
  p.T = tokens_per_cta(p.N, 2ll * p.Hkv * (a.cache_q4 ? d / 8 : row_bytes / 16), 4 * kThreads);
  const unsigned grid = (unsigned)((p.N + p.T - 1) / p.T);
  if (a.cache_q4) {
    if (d == 128) {
      if (a.out_dtype == CP_BF16) read_q4_kernel<__nv_bfloat16, 128><<<grid, kThreads, 0, s>>>(p);
      else read_q4_kernel<float, 128><<<grid, kThreads, 0, s>>>(p);
    } else {
      if (a.out_dtype == CP_BF16) read_q4_kernel<__nv_bfloat16, 64><<<grid, kThreads, 0, s>>>(p);
      else read_q4_kernel<float, 64><<<grid, kThreads, 0, s>>>(p);
    }
  } else if (row_bytes == 128) {
    read_rows_kernel<8><<<grid, kThreads, 0, s>>>(p);
  } else if (row_bytes == 256) {
    read_rows_kernel<16><<<grid, kThreads, 0, s>>>(p);
  } else {
    read_rows_kernel<32><<<grid, kThreads, 0, s>>>(p);
  }
  return cudaGetLastError();
}
