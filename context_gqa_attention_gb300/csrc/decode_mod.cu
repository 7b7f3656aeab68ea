// Decode over the round-robin paged cache with modified scores (cp_decode_attention_mod) and over
// a cache held in 4 bits (cp_decode_attention_q4), one query token per sequence.
//
// "Add utility functions to enable pass-kv prefill and allgather decode" (vLLM PR 26059),
// Purpose: decode KV stays on the CP ranks round-robin, each rank attends the new query over its
// own tokens and the partials are combined.
//
//   s_j = scale q.k_j;  s_j = cap tanh(s_j / cap);  s_j -= slope |i - j|     (each optional)
//   over the keys j in [lo, L), lo = max(0, L - window, kv_start);  out = softmax(s) V
//
// Work unit (one CTA of 4 warps): split s of rank r's visible tokens of sequence b, kv head g, all
// query heads of the group; a warp takes every fourth page (16 tokens).  Both products run on the
// tensor cores with the *tokens* as the M dimension of S^T = K Q^T (16 tokens x 8 heads per MMA)
// and the head's dims as the M dimension of O^T = V^T P^T, so a page costs D / 16 + D / 16 MMAs
// for up to 8 query heads, and K and V go from global memory straight into the A fragments: the
// contraction order of K's dims and the row order of V's dims are free, so each thread's 16-byte
// (8-byte) piece of a row is a set of whole fragments, and no shared memory or ldmatrix is needed.
// P^T (tokens x heads -> heads x tokens) is transposed between the products by movmatrix.
#include <math.h>

#include "common.cuh"
#include "q4.cuh"
#include "sm100.cuh"

namespace cpattn {
namespace {

constexpr int kWarps = 4;
constexpr int kPage = 16;
constexpr int kMaxPartials = 256;  // cp * splits of one fused call
constexpr float kMaxGrowth = 8.f;  // log2: how far a score may exceed the running reference

enum Format { kBf16 = 0, kQ4 = 1 };

struct ModParams {
  int B, Hq, Hkv, G, cp, I, S, ST, max_blocks, window;
  long long pool;
  float scale, softcap;
  const void* q;
  const uint8_t* kc;
  const uint8_t* vc;
  const int32_t* tables;
  const int32_t* seq_lens;
  const float* slopes;
  const int32_t* kv_start;
  float* out;  // partials [cp*S][B][Hq][D] (the workspace when fused)
  float* lse;
  int32_t* err;
  int fused;
  int32_t* counters;
  void* final_out;
  float* final_lse;
};

// ------------------------------------------------------------------------------ ranges
// Visible positions [lo, L) of a sequence, and a rank's share of them: local tokens [a, n), its
// splits counted from the page that holds a.
struct Span {
  int a, a0, n;
};
CP_DEV int first_visible(const ModParams& p, int b, int L) {
  int lo = 0;
  if (p.window > 0 && L > p.window) lo = L - p.window;
  if (p.kv_start != nullptr) lo = max(lo, __ldg(p.kv_start + b));
  return min(lo, max(L, 0));
}
CP_DEV Span rank_span(const ModParams& p, int L, int lo, int r) {
  Span s;
  s.n = L > 0 ? rank_local_len(L, r, p.cp, p.I) : 0;
  s.a = lo > 0 ? rank_local_len(lo, r, p.cp, p.I) : 0;
  s.a0 = s.a & ~(kPage - 1);
  return s;
}
CP_DEV int live_splits(const ModParams& p, const Span& s) {
  return s.a < s.n ? min(p.S, (s.n - s.a0 + p.ST - 1) / p.ST) : 0;
}
// Splits of all ranks that hold visible tokens (a rank per lane; every lane gets the sum).
CP_DEV int live_total(const ModParams& p, int L, int lo) {
  int c = 0;
  for (int r = threadIdx.x & 31; r < p.cp; r += 32) c += live_splits(p, rank_span(p, L, lo, r));
  return __reduce_add_sync(0xffffffffu, c);
}

// ------------------------------------------------------------------------------ results
template <typename T>
CP_DEV void put4(void* out, long long at, float4 v) {
  if constexpr (sizeof(T) == 2) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + at) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = v;
  }
}

// What the four warps hold of the CTA's split, in shared memory: per warp and head the reference
// m (log2), the sum l and the unnormalised output row.
template <int D, int HR>
struct WarpParts {
  float o[kWarps][HR][D];
  float m[kWarps][HR], l[kWarps][HR];
};

// Warps -> the CTA's partial, and in a fused call partials -> result.  A split publishes its
// partial with one acquire-release count per (sequence, kv head) after a CTA barrier; the CTA that
// counts last reads the others' partials through L2 and merges (weights 2^(lse - max)), then
// returns the counter to zero.  No CTA waits for another.  A (sequence, kv head) with one live
// split writes its result at once.  Sums of weights that are zero mean no visible key; NaN stays.
template <typename T, int D, int HR>
CP_DEV void finish(const ModParams& p, WarpParts<D, HR>& w, int b, int g, int part, int live) {
  constexpr int V = D / 4;  // threads (of 4 dims) per head
  const long long unit0 = (long long)b * p.Hq + (long long)g * p.G;
  const long long stride = (long long)p.B * p.Hq;
  const bool direct = p.fused && live == 1;
  __shared__ int s_last;
  __syncthreads();
  for (int i = threadIdx.x; i < p.G * V; i += blockDim.x) {
    const int hh = i / V, dd = (i % V) * 4;
    float M = -INFINITY;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) M = fmaxf(M, w.m[k][hh]);
    float L = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      const float mk = w.m[k][hh];
      // (a warp whose reference is -inf saw no finite score: its sums are 0, or NaN)
      const float e = mk == M || mk == -INFINITY ? 1.f : exp2f(mk - M);
      const float4 x = *reinterpret_cast<const float4*>(&w.o[k][hh][dd]);
      L += e * w.l[k][hh];
      o.x += e * x.x, o.y += e * x.y, o.z += e * x.z, o.w += e * x.w;
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    o.x *= inv, o.y *= inv, o.z *= inv, o.w *= inv;
    const float lse = L == 0.f ? -INFINITY : ((M == -INFINITY ? 0.f : M) + log2f(L)) * kLn2;
    if (direct) {
      put4<T>(p.final_out, (unit0 + hh) * D + dd, o);
      if (dd == 0 && p.final_lse) p.final_lse[unit0 + hh] = lse;
    } else {
      const long long at = part * stride + unit0 + hh;
      if (L != 0.f || p.fused) *reinterpret_cast<float4*>(p.out + at * D + dd) = o;
      if (dd == 0) p.lse[at] = lse;
    }
  }
  if (!p.fused || direct) return;

  __syncthreads();
  if (threadIdx.x == 0) {
    int prev;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;"
                 : "=r"(prev)
                 : "l"(p.counters + (long long)b * p.Hkv + g)
                 : "memory");
    s_last = prev == live - 1;
  }
  __syncthreads();
  if (!s_last) return;
  // per (partial, head) weights over the warp parts (free now), then the weighted rows
  float* wt = &w.o[0][0][0];
  static_assert(sizeof(w.o) >= kMaxPartials * HR * sizeof(float), "merge weights");
  float* s_M = &w.m[0][0];
  float* s_L = &w.l[0][0];
  const int P = p.cp * p.S, L = __ldg(p.seq_lens + b), lo = first_visible(p, b, L);
  for (int i = threadIdx.x; i < P * p.G; i += blockDim.x) {
    const int k = i / p.G, hh = i % p.G, r = k / p.S;
    const bool on = k % p.S < live_splits(p, rank_span(p, L, lo, r));
    wt[i] = on ? __ldcg(p.lse + k * stride + unit0 + hh) * kLog2e : -INFINITY;
  }
  __syncthreads();
  if (threadIdx.x < p.G) {
    float M = -INFINITY;
    bool nan = false;
    for (int k = 0; k < P; ++k) {
      const float x = wt[k * p.G + threadIdx.x];
      M = fmaxf(M, x);
      nan |= x != x;
    }
    float sum = 0.f;
    for (int k = 0; k < P; ++k) {
      const float x = wt[k * p.G + threadIdx.x];
      const float e = x == -INFINITY ? 0.f : exp2f(x - M);
      wt[k * p.G + threadIdx.x] = e;
      sum += e;
    }
    s_M[threadIdx.x] = M;
    s_L[threadIdx.x] = nan ? NAN : sum;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.G * V; i += blockDim.x) {
    const int hh = i / V, dd = (i % V) * 4;
    const float* src = p.out + (unit0 + hh) * D + dd;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int U = 8;  // partial rows in flight
    for (int k0 = 0; k0 < P; k0 += U) {
      float4 x[U];
      float e[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = k0 + u;
        e[u] = k < P ? wt[k * p.G + hh] : 0.f;
        if (e[u] != 0.f) x[u] = __ldcg(reinterpret_cast<const float4*>(src + k * stride * D));
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (e[u] != 0.f)
          acc.x += e[u] * x[u].x, acc.y += e[u] * x[u].y, acc.z += e[u] * x[u].z, acc.w += e[u] * x[u].w;
    }
    const float sum = s_L[hh], inv = sum == 0.f ? 0.f : 1.f / sum;
    acc.x *= inv, acc.y *= inv, acc.z *= inv, acc.w *= inv;
    put4<T>(p.final_out, (unit0 + hh) * D + dd, acc);
    if (dd == 0 && p.final_lse) p.final_lse[unit0 + hh] = sum == 0.f ? -INFINITY : (s_M[hh] + log2f(sum)) * kLn2;
  }
  if (threadIdx.x == 0) p.counters[(long long)b * p.Hkv + g] = 0;
}

// A split without a visible token: its partial is empty; in a fused call the first CTA of a
// sequence that has no visible key at all writes the result of no keys (0, LSE -inf).
template <typename T, int D>
CP_DEV void finish_empty(const ModParams& p, int b, int g, int r, int split, int part, int live) {
  const long long unit0 = (long long)b * p.Hq + (long long)g * p.G;
  if (!p.fused) {
    for (int i = threadIdx.x; i < p.G; i += blockDim.x)
      p.lse[(long long)part * p.B * p.Hq + unit0 + i] = -INFINITY;
  } else if (live == 0 && r == 0 && split == 0) {
    for (int i = threadIdx.x; i < p.G * D / 4; i += blockDim.x)
      put4<T>(p.final_out, unit0 * D + 4 * i, make_float4(0.f, 0.f, 0.f, 0.f));
    if (p.final_lse != nullptr)
      for (int i = threadIdx.x; i < p.G; i += blockDim.x) p.final_lse[unit0 + i] = -INFINITY;
  }
}

// The CTA's unit of work; false: no visible token falls in it (its empty result is written).
struct Unit {
  int split, g, r, b, part, live, L;
  int l0, l1, a;  // local tokens [max(l0, a), l1); l0 is the first one of a page
};
template <typename T, int D>
CP_DEV bool take_unit(const ModParams& p, Unit& u) {
  u.split = blockIdx.x;
  u.g = blockIdx.y;
  u.r = (int)(blockIdx.z % (unsigned)p.cp);
  u.b = (int)(blockIdx.z / (unsigned)p.cp);
  u.part = u.r * p.S + u.split;
  u.L = __ldg(p.seq_lens + u.b);
  const int lo = first_visible(p, u.b, u.L);
  u.live = p.fused ? live_total(p, u.L, lo) : 0;
  const Span s = rank_span(p, u.L, lo, u.r);
  if (s.a < s.n && (long long)p.S * p.ST < s.n - s.a0 && u.split == 0 && threadIdx.x == 0)
    report(p.err, CP_ERR_DEVICE_BOUNDS);  // the plan does not cover this sequence
  u.a = s.a;
  u.l0 = s.a0 + u.split * p.ST;
  u.l1 = min(s.n, u.l0 + p.ST);
  if (s.a < s.n && u.l0 < u.l1) return true;
  finish_empty<T, D>(p, u.b, u.g, u.r, u.split, u.part, u.live);
  return false;
}

// ------------------------------------------------------------------------------ scores
// cap tanh(x / cap) for x = scale q.k as cap (1 - 2 / (1 + e^(2 x / cap))): absolute error about
// cap 2^-22, which is what matters for exp(x), also where tanh itself is small.
struct Cap {
  float in, out;  // 2 scale log2(e) / cap;  cap log2(e): the result is in log2 units
};
CP_DEV float capped(float qk, const Cap& c) {
  return c.out - __fdividef(2.f * c.out, 1.f + sm100::ex2(qk * c.in));
}

// ------------------------------------------------------------------------------ tensor cores
CP_DEV void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                     uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
CP_DEV uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
CP_DEV uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Pairs (x's half, y's half) of two words: the low halves, or the high ones.
CP_DEV uint32_t low_halves(uint32_t x, uint32_t y) { return __byte_perm(x, y, 0x5410); }
CP_DEV uint32_t high_halves(uint32_t x, uint32_t y) { return __byte_perm(x, y, 0x7632); }

// Codes i and i + 4 of a word (i = 0..3) as the bf16 pair 1 + n / 16: the code becomes the top
// mantissa bits of 1.0, one shift and one three-input logic operation for two values.
template <int I>
CP_DEV uint32_t codes(uint32_t w) {
  return ((I == 0 ? w << 3 : w >> (4 * I - 3)) & 0x00780078u) | 0x3f803f80u;
}

template <int BYTES>
struct Piece {  // BYTES of a row in 32-bit words
  uint32_t w[BYTES / 4];
};
template <int BYTES>
CP_DEV void ldg_piece(Piece<BYTES>& x, const uint8_t* p) {
  if constexpr (BYTES == 16)
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(x.w[0]), "=r"(x.w[1]), "=r"(x.w[2]), "=r"(x.w[3]) : "l"(p));
  else if constexpr (BYTES == 8)
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(x.w[0]), "=r"(x.w[1]) : "l"(p));
  else
    asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(x.w[0]) : "l"(p));
}

// What one thread (row id gid = lane / 4, column id tid = lane % 4) holds of a page of one head.
//   K of tokens gid and gid + 8;  V of tokens 2 tid, 2 tid + 1, 2 tid + 8, 2 tid + 9.
template <int F, int D>
struct Page;
template <int D>
struct Page<kQ4, D> {
  Piece<D / 8> k[2];    // a quarter of the row's D / 2 bytes
  Piece<D / 16> v[4];   // an eighth
  Piece<D / 16> ks[2];  // (scale, minimum) of each group
  Piece<D / 16> vs[2];  // of tokens gid and gid + 8
  CP_DEV void load(const uint8_t* kr, const uint8_t* vr, int gid, int tid) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      ldg_piece(k[i], kr + (gid + 8 * i) * (D / 2) + tid * (D / 8));
      ldg_piece(ks[i], kr + 8 * D + (gid + 8 * i) * (D / 16));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      ldg_piece(v[i], vr + (2 * tid + (i & 1) + 8 * (i >> 1)) * (D / 2) + gid * (D / 16));
#pragma unroll
    for (int i = 0; i < 2; ++i) ldg_piece(vs[i], vr + 8 * D + (gid + 8 * i) * (D / 16));
  }
};
template <int D>
struct Page<kBf16, D> {
  Piece<16> k[2][D / 32];  // 16-byte pieces tid, tid + 4, ..
  Piece<16> v[4][D / 64];  // pieces gid, gid + 8
  CP_DEV void load(const uint8_t* kr, const uint8_t* vr, int gid, int tid) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int c = 0; c < D / 32; ++c) ldg_piece(k[i][c], kr + (gid + 8 * i) * (2 * D) + (4 * c + tid) * 16);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
        ldg_piece(v[i][c], vr + (2 * tid + (i & 1) + 8 * (i >> 1)) * (2 * D) + (8 * c + gid) * 16);
  }
};

template <int F, int D, int NT, bool MOD>
__global__ void __launch_bounds__(kWarps * 32, F == kQ4 ? (NT == 1 ? 4 : 2) : (NT == 1 ? 3 : 2))
    decode_mod_kernel(const ModParams p) {
  using T = __nv_bfloat16;
  constexpr int HR = 8 * NT;         // head rows (query heads of the group, padded)
  constexpr int GR = F == kQ4 ? D / kQ4Group : 1;
  constexpr int KS = D / 16;         // MMAs of each product
  constexpr long long kRec = F == kQ4 ? 9ll * D : 2ll * kPage * D;  // bytes of a head's page
  __shared__ __align__(16) WarpParts<D, HR> parts;
  Unit u;
  if (!take_unit<T, D>(p, u)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tid = lane & 3;

  // Q^T as the B operand of S^T = K Q^T: the dims of MMA ks as K's pieces bring them.  For the
  // 4-bit format also the sums of q over each group, for the heads of this thread's columns.
  uint32_t qb[NT][KS][2];
  float qsum[NT][GR][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int head = gid + 8 * nt;
    const T* row = static_cast<const T*>(p.q) + ((long long)u.b * p.Hq + (long long)u.g * p.G + head) * D;
    float sum[GR];
#pragma unroll
    for (int gr = 0; gr < GR; ++gr) sum[gr] = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        int d0, d1;
        if constexpr (F == kQ4) {  // group-major: 4 MMAs a group, two per word of 8 codes
          const int gr = ks / 4, wi = (ks % 4) / 2, i = (ks % 2) * 2 + e;
          const int base = D == 64 ? 8 * (2 * tid + wi) : 64 * gr + 8 * (2 * tid + wi);
          d0 = base + i;
          d1 = base + i + 4;
        } else {  // two MMAs a 16-byte piece
          d0 = 32 * (ks / 2) + 8 * tid + 4 * (ks % 2) + 2 * e;
          d1 = d0 + 1;
        }
        uint32_t x = 0u;
        if (head < p.G) {
          const uint16_t* rb = reinterpret_cast<const uint16_t*>(row);
          x = (uint32_t)__ldg(rb + d0) | ((uint32_t)__ldg(rb + d1) << 16);
        }
        qb[nt][ks][e] = x;
        if constexpr (F == kQ4) sum[ks / 4] += bf16_lo(x) + bf16_hi(x);
      }
    }
#pragma unroll
    for (int gr = 0; gr < GR; ++gr) {
      qsum[nt][gr][0] = qsum[nt][gr][1] = 0.f;
      if constexpr (F == kQ4) {
        sum[gr] += __shfl_xor_sync(0xffffffffu, sum[gr], 1);
        sum[gr] += __shfl_xor_sync(0xffffffffu, sum[gr], 2);
        qsum[nt][gr][0] = __shfl_sync(0xffffffffu, sum[gr], 8 * tid);      // head 2 tid
        qsum[nt][gr][1] = __shfl_sync(0xffffffffu, sum[gr], 8 * tid + 4);  // head 2 tid + 1
      }
    }
  }

  const float scale_log2 = p.scale * kLog2e;
  const Cap cap{MOD && p.softcap > 0.f ? 2.f * scale_log2 / p.softcap : 0.f, p.softcap * kLog2e};
  float slope[NT][2];
  if constexpr (MOD) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int head = 8 * nt + 2 * tid + c;
        slope[nt][c] = p.slopes != nullptr && head < p.G ? __ldg(p.slopes + u.g * p.G + head) * kLog2e : 0.f;
      }
  }

  // per head of this thread's columns (2 tid, 2 tid + 1): reference, sum of this thread's tokens;
  // 4-bit: the part of the output that does not go through the MMA, per group
  float m[NT][2], l[NT][2], corr[NT][GR][2], o[NT][KS][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      m[nt][c] = -INFINITY;
      l[nt][c] = 0.f;
#pragma unroll
      for (int gr = 0; gr < GR; ++gr) corr[nt][gr][c] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
  }

  const int32_t* trow = p.tables + ((long long)u.r * p.B + u.b) * p.max_blocks;
  const int pg0 = u.l0 / kPage, pg1 = (u.l1 + kPage - 1) / kPage;
  const int mine = pg1 - pg0 > warp ? (pg1 - pg0 - warp + kWarps - 1) / kWarps : 0;
  const long long pool0 = (long long)u.r * p.pool;
  // table entries of this warp's pages, 32 at a time (lane j holds the j-th), a batch ahead
  auto fetch_ids = [&](int j0) -> int {
    const int j = j0 + lane, pg = pg0 + warp + j * kWarps;
    int id = -1;
    if (j < mine && pg < p.max_blocks) id = __ldg(trow + pg);
    return id >= 0 && id < p.pool ? id : -1;
  };
  int ids = fetch_ids(0), ids_next = fetch_ids(32);

  Page<F, D> cur, nxt;
  auto load = [&](int j, Page<F, D>& x) -> bool {  // this warp's page j; false: not in the pool
    if ((j & 31) == 0 && j > 0) {
      ids = ids_next;
      ids_next = fetch_ids(j + 32);
    }
    const int id = __shfl_sync(0xffffffffu, ids, j & 31);
    if (id < 0) return false;
    const long long at = ((pool0 + id) * p.Hkv + u.g) * kRec;
    x.load(p.kc + at, p.vc + at, gid, tid);
    return true;
  };

  auto consume = [&](int j, Page<F, D>& x) {
    const int t0 = (pg0 + warp + j * kWarps) * kPage;  // the page's first local token
    const bool edge = t0 < u.a || t0 + kPage > u.l1;
    // ---- S^T: rows = tokens gid, gid + 8; columns = heads 2 tid, 2 tid + 1
    float s[NT][4];  // [token half * 2 + head]
    if constexpr (F == kQ4) {
      float c[NT][GR][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int gr = 0; gr < GR; ++gr)
#pragma unroll
          for (int e = 0; e < 4; ++e) c[nt][gr][e] = 0.f;
#pragma unroll
      for (int gr = 0; gr < GR; ++gr)
#pragma unroll
        for (int wi = 0; wi < 2; ++wi) {
          const uint32_t w0 = x.k[0].w[wi * GR + gr], w1 = x.k[1].w[wi * GR + gr];
          const int ks = gr * 4 + wi * 2;
          const uint32_t a0 = codes<0>(w0), a1 = codes<0>(w1), a2 = codes<1>(w0), a3 = codes<1>(w1);
          const uint32_t b0 = codes<2>(w0), b1 = codes<2>(w1), b2 = codes<3>(w0), b3 = codes<3>(w1);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma16816(c[nt][gr], a0, a1, a2, a3, qb[nt][ks][0], qb[nt][ks][1]);
            mma16816(c[nt][gr], b0, b1, b2, b3, qb[nt][ks + 1][0], qb[nt][ks + 1][1]);
          }
        }
      // q.k = sum over groups of 16 scale c + (minimum - 16 scale) sum(q), c = sum q (1 + n / 16)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float s16[GR], off[GR];
#pragma unroll
        for (int gr = 0; gr < GR; ++gr) {
          s16[gr] = 16.f * bf16_lo(x.ks[i].w[gr]);
          off[gr] = bf16_hi(x.ks[i].w[gr]) - s16[gr];
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float v = 0.f;
#pragma unroll
            for (int gr = 0; gr < GR; ++gr)
              v = fmaf(s16[gr], c[nt][gr][2 * i + h], fmaf(off[gr], qsum[nt][gr][h], v));
            s[nt][2 * i + h] = v;
          }
      }
    } else {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const int w = (ks % 2) * 2;
        const Piece<16>&k0 = x.k[0][ks / 2], &k1 = x.k[1][ks / 2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma16816(s[nt], k0.w[w], k1.w[w], k0.w[w + 1], k1.w[w + 1], qb[nt][ks][0], qb[nt][ks][1]);
      }
    }

    // ---- scores in log2 units, masked tokens at -inf
    const bool on0 = !edge || (t0 + gid >= u.a && t0 + gid < u.l1);
    const bool on1 = !edge || (t0 + gid + 8 >= u.a && t0 + gid + 8 < u.l1);
    float dist[2] = {0.f, 0.f};
    if constexpr (MOD) {
      if (p.slopes != nullptr) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const unsigned t = (unsigned)(t0 + gid + 8 * i), turn = t / (unsigned)p.I;
          const long long pos = (long long)turn * p.I * p.cp + (long long)u.r * p.I + (t - turn * p.I);
          dist[i] = (float)(u.L - 1 - pos);
        }
      }
    }
    bool grow = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float v = s[nt][e];
        if constexpr (MOD) {
          v = p.softcap > 0.f ? capped(v, cap) : v * scale_log2;
          v = fmaf(-slope[nt][e & 1], dist[e >> 1], v);
        } else {
          v *= scale_log2;
        }
        v = (e < 2 ? on0 : on1) ? v : -INFINITY;
        s[nt][e] = v;
        grow |= v > m[nt][e & 1] + kMaxGrowth;
      }
    // The reference moves only when some score exceeds it by more than 2^8 (fp32 sums hold that
    // with room to spare), so the reduction over the 8 rows of lanes is rare.
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float mx = fmaxf(s[nt][h], s[nt][2 + h]);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const float m_new = fmaxf(m[nt][h], mx);
          const float alpha = m_new == m[nt][h] ? 1.f : sm100::ex2(m[nt][h] - m_new);
          m[nt][h] = m_new;
          l[nt][h] *= alpha;
#pragma unroll
          for (int gr = 0; gr < GR; ++gr) corr[nt][gr][h] *= alpha;
#pragma unroll
          for (int i = 0; i < KS; ++i) {
            o[nt][i][h] *= alpha;
            o[nt][i][2 + h] *= alpha;
          }
        }
    }

    // ---- P^T as the B operand of O^T = V^T P^T, rounded to bf16 (a tensor-core operand; the sums
    // l keep 32 bits).  4-bit: each group's P times V's scale is what is rounded, and the sums of
    // the rounded values cancel the offset of the codes exactly.
    uint32_t pb[NT][GR][2];
    float sc[2][GR], mn[2][GR];
    if constexpr (F == kQ4) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int gr = 0; gr < GR; ++gr) {
          // scales of masked rows may be anything: 0
          const uint32_t w = (i == 0 ? on0 : on1) ? x.vs[i].w[gr] : 0u;
          sc[i][gr] = bf16_lo(w);
          mn[i][gr] = bf16_hi(w);
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float pr[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float ref = m[nt][e & 1];
        pr[e] = sm100::ex2(s[nt][e] - (ref == -INFINITY ? 0.f : ref));
      }
      l[nt][0] += pr[0] + pr[2];
      l[nt][1] += pr[1] + pr[3];
      if constexpr (F == kQ4) {
#pragma unroll
        for (int gr = 0; gr < GR; ++gr)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t r = pack2(pr[2 * i] * sc[i][gr], pr[2 * i + 1] * sc[i][gr]);
            corr[nt][gr][0] = fmaf(pr[2 * i], mn[i][gr], fmaf(-16.f, bf16_lo(r), corr[nt][gr][0]));
            corr[nt][gr][1] = fmaf(pr[2 * i + 1], mn[i][gr], fmaf(-16.f, bf16_hi(r), corr[nt][gr][1]));
            pb[nt][gr][i] = transpose8x8(r);
          }
      } else {
        pb[nt][0][0] = transpose8x8(pack2(pr[0], pr[1]));
        pb[nt][0][1] = transpose8x8(pack2(pr[2], pr[3]));
      }
    }

    // ---- O^T: rows = dims, columns = heads
    if constexpr (F == kQ4) {
#pragma unroll
      for (int gr = 0; gr < GR; ++gr) {
        const uint32_t ab0 = low_halves(x.v[0].w[gr], x.v[1].w[gr]), ab1 = high_halves(x.v[0].w[gr], x.v[1].w[gr]);
        const uint32_t cd0 = low_halves(x.v[2].w[gr], x.v[3].w[gr]), cd1 = high_halves(x.v[2].w[gr], x.v[3].w[gr]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma16816(o[nt][gr * 4 + 0], codes<0>(ab0), codes<0>(ab1), codes<0>(cd0), codes<0>(cd1), pb[nt][gr][0], pb[nt][gr][1]);
          mma16816(o[nt][gr * 4 + 1], codes<1>(ab0), codes<1>(ab1), codes<1>(cd0), codes<1>(cd1), pb[nt][gr][0], pb[nt][gr][1]);
          mma16816(o[nt][gr * 4 + 2], codes<2>(ab0), codes<2>(ab1), codes<2>(cd0), codes<2>(cd1), pb[nt][gr][0], pb[nt][gr][1]);
          mma16816(o[nt][gr * 4 + 3], codes<3>(ab0), codes<3>(ab1), codes<3>(cd0), codes<3>(cd1), pb[nt][gr][0], pb[nt][gr][1]);
        }
      }
    } else {
      if (edge) {  // rows behind the sequence may hold anything, and 0 times NaN is NaN
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = t0 + 2 * tid + (i & 1) + 8 * (i >> 1);
          if (t < u.a || t >= u.l1) {
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
#pragma unroll
              for (int w = 0; w < 4; ++w) x.v[i][c].w[w] = 0u;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        const int c = i / 4, w = i % 4;
        const uint32_t a0 = low_halves(x.v[0][c].w[w], x.v[1][c].w[w]), a1 = high_halves(x.v[0][c].w[w], x.v[1][c].w[w]);
        const uint32_t a2 = low_halves(x.v[2][c].w[w], x.v[3][c].w[w]), a3 = high_halves(x.v[2][c].w[w], x.v[3][c].w[w]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][i], a0, a1, a2, a3, pb[nt][0][0], pb[nt][0][1]);
      }
    }
  };

  bool bad = false;
  bool have = mine > 0 && load(0, cur);
  bad |= mine > 0 && !have;
  for (int j = 0; j < mine; j += 2) {
    bool have2 = false;
    if (j + 1 < mine) {
      have2 = load(j + 1, nxt);
      bad |= !have2;
    }
    if (have) consume(j, cur);
    have = false;
    if (j + 2 < mine) {
      have = load(j + 2, cur);
      bad |= !have;
    }
    if (have2) consume(j + 1, nxt);
  }
  if (bad && lane == 0) report(p.err, CP_ERR_DEVICE_BOUNDS);

  // ---- this warp's part: sums over the lanes that share a column, output rows per head
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) {
        l[nt][h] += __shfl_xor_sync(0xffffffffu, l[nt][h], x);
        if constexpr (F == kQ4) {
#pragma unroll
          for (int gr = 0; gr < GR; ++gr) corr[nt][gr][h] += __shfl_xor_sync(0xffffffffu, corr[nt][gr][h], x);
        }
      }
      const int head = 8 * nt + 2 * tid + h;
      if (gid == 0) {
        parts.m[warp][head] = m[nt][h];
        parts.l[warp][head] = l[nt][h];
      }
      float* row = &parts.o[warp][head][0];
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        if constexpr (F == kQ4) {  // MMA i: group i / 4, codes i % 4 and i % 4 + 4 of word gid
          const int gr = i / 4, d = 64 * gr + 8 * gid + i % 4;
          row[d] = fmaf(16.f, o[nt][i][h], corr[nt][gr][h]);
          row[d + 4] = fmaf(16.f, o[nt][i][2 + h], corr[nt][gr][h]);
        } else {
          const int d = 64 * (i / 4) + 8 * gid + 2 * (i % 4);
          row[d] = o[nt][i][h];
          row[d + 1] = o[nt][i][2 + h];
        }
      }
    }
  finish<T, D, HR>(p, parts, u.b, u.g, u.part, u.live);
}

// ------------------------------------------------------------------------------ fp32 caches
// fp32 K and V keep their 24 bits, so the products run on the CUDA cores: two lanes per token for
// q.k (half a row each), D / 4 lanes per token for P V; per page and warp as above.
template <int D, int HR>
__global__ void __launch_bounds__(kWarps * 32) decode_mod_f32_kernel(const ModParams p) {
  constexpr int NCH = D / 4;       // lanes per V row
  constexpr int TG = 32 / NCH;     // V rows a warp reads at a time
  __shared__ __align__(16) WarpParts<D, HR> parts;
  __shared__ __align__(16) float qs[HR][D];
  __shared__ float ps[kWarps][kPage][HR];
  Unit u;
  if (!take_unit<float, D>(p, u)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float* qg = static_cast<const float*>(p.q) + ((long long)u.b * p.Hq + (long long)u.g * p.G) * D;
  for (int i = threadIdx.x; i < HR * D; i += blockDim.x) (&qs[0][0])[i] = i < p.G * D ? qg[i] : 0.f;
  __syncthreads();
  float m[HR], l[HR], acc[HR][4];
#pragma unroll
  for (int h = 0; h < HR; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[h][e] = 0.f;
  }
  const int32_t* trow = p.tables + ((long long)u.r * p.B + u.b) * p.max_blocks;
  const int pg1 = (u.l1 + kPage - 1) / kPage;
  const int tk = lane >> 1, half = lane & 1, vc = lane % NCH, vt = lane / NCH;
  bool bad = false;
  for (int pg = u.l0 / kPage + warp; pg < pg1; pg += kWarps) {
    const int id = pg < p.max_blocks ? __ldg(trow + pg) : -1;
    if (id < 0 || id >= p.pool) {
      bad = true;
      continue;
    }
    const long long at = (((long long)u.r * p.pool + id) * p.Hkv + u.g) * (kPage * D);
    const float4* kr = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p.kc) + at + tk * D);
    const float4* vr = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p.vc) + at);
    const int t0 = pg * kPage, t = t0 + tk;
    const bool on = t >= u.a && t < u.l1;
    float s[HR];
#pragma unroll
    for (int h = 0; h < HR; ++h) s[h] = 0.f;
#pragma unroll 4
    for (int c = half; c < D / 4; c += 2) {  // the two lanes of a token alternate over its vectors
      const float4 k = __ldg(kr + c);
#pragma unroll
      for (int h = 0; h < HR; ++h) {
        const float4 q = *reinterpret_cast<const float4*>(&qs[h][4 * c]);
        s[h] += q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w;
      }
    }
    const unsigned turn = (unsigned)t / (unsigned)p.I;
    const long long pos = (long long)turn * p.I * p.cp + (long long)u.r * p.I + ((unsigned)t - turn * p.I);
    const float dist = (float)(u.L - 1 - pos);
    float alpha[HR];
#pragma unroll
    for (int h = 0; h < HR; ++h) {
      s[h] += __shfl_xor_sync(0xffffffffu, s[h], 1);
      float v = s[h] * p.scale;
      if (p.softcap > 0.f) v = p.softcap * tanhf(v / p.softcap);
      if (p.slopes != nullptr && h < p.G) v -= __ldg(p.slopes + u.g * p.G + h) * dist;
      v = on ? v * kLog2e : -INFINITY;
      const float m_new = fmaxf(m[h], warp_max(v));
      alpha[h] = m_new == m[h] ? 1.f : exp2f(m[h] - m_new);
      m[h] = m_new;
      const float e = exp2f(v - (m_new == -INFINITY ? 0.f : m_new));
      l[h] = l[h] * alpha[h] + (half == 0 ? e : 0.f);
      if (half == 0) ps[warp][tk][h] = e;
    }
    __syncwarp();
#pragma unroll
    for (int h = 0; h < HR; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[h][e] *= alpha[h];
#pragma unroll 4
    for (int i = vt; i < kPage; i += TG) {
      if (t0 + i < u.a || t0 + i >= u.l1) continue;  // 0 times whatever lies there could be NaN
      const float4 v = __ldg(vr + i * NCH + vc);
#pragma unroll
      for (int h = 0; h < HR; ++h) {
        const float w = ps[warp][i][h];
        acc[h][0] += w * v.x, acc[h][1] += w * v.y, acc[h][2] += w * v.z, acc[h][3] += w * v.w;
      }
    }
    __syncwarp();
  }
  if (bad && lane == 0) report(p.err, CP_ERR_DEVICE_BOUNDS);
#pragma unroll
  for (int h = 0; h < HR; ++h) {
    const float sum = warp_sum(l[h]);
    if (lane == 0) {
      parts.m[warp][h] = m[h];
      parts.l[warp][h] = sum;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int o = NCH; o < 32; o <<= 1) acc[h][e] += __shfl_xor_sync(0xffffffffu, acc[h][e], o);
    if (vt == 0)
      *reinterpret_cast<float4*>(&parts.o[warp][h][4 * vc]) = make_float4(acc[h][0], acc[h][1], acc[h][2], acc[h][3]);
  }
  finish<float, D, HR>(p, parts, u.b, u.g, u.part, u.live);
}

template <int F, int D, int NT>
void launch_bits(const ModParams& p, bool mod, dim3 grid, cudaStream_t s) {
  if (F == kBf16 || mod) decode_mod_kernel<F, D, NT, true><<<grid, kWarps * 32, 0, s>>>(p);
  else if constexpr (F == kQ4) decode_mod_kernel<F, D, NT, false><<<grid, kWarps * 32, 0, s>>>(p);
}
template <int D>
cudaError_t launch_d(const ModParams& p, int dtype, bool q4, bool mod, dim3 grid, cudaStream_t s) {
  if (dtype == CP_F32) {
    if (p.G <= 2) decode_mod_f32_kernel<D, 2><<<grid, kWarps * 32, 0, s>>>(p);
    else if (p.G <= 4) decode_mod_f32_kernel<D, 4><<<grid, kWarps * 32, 0, s>>>(p);
    else decode_mod_f32_kernel<D, 8><<<grid, kWarps * 32, 0, s>>>(p);
  } else if (q4) {
    if (p.G <= 8) launch_bits<kQ4, D, 1>(p, mod, grid, s);
    else launch_bits<kQ4, D, 2>(p, mod, grid, s);
  } else {
    if (p.G <= 8) launch_bits<kBf16, D, 1>(p, mod, grid, s);
    else launch_bits<kBf16, D, 2>(p, mod, grid, s);
  }
  return cudaGetLastError();
}

}  // namespace
}  // namespace cpattn

cudaError_t cp_launch_decode_mod(const cp_decode_args& a, const cp_score_mod& mod, bool q4, float scale,
                                 const CpDecodeWorkspace* ws, void* out, float* out_lse,
                                 cudaStream_t s) {
  using namespace cpattn;
  ModParams p;
  p.B = a.num_seqs;
  p.Hq = a.num_q_heads;
  p.Hkv = a.num_kv_heads;
  p.G = a.num_q_heads / a.num_kv_heads;
  p.cp = a.cp;
  p.I = a.interleave;
  p.S = a.num_splits;
  p.ST = a.split_tokens;
  p.max_blocks = a.max_blocks;
  p.window = mod.window;
  p.pool = a.pool_pages;
  p.scale = scale;
  p.softcap = mod.softcap;
  p.q = a.q;
  p.kc = static_cast<const uint8_t*>(a.k_cache);
  p.vc = static_cast<const uint8_t*>(a.v_cache);
  p.tables = a.block_tables;
  p.seq_lens = a.seq_lens;
  p.slopes = mod.alibi_slopes;
  p.kv_start = mod.kv_start;
  p.out = ws ? ws->partial_out : a.out;
  p.lse = ws ? ws->partial_lse : a.lse;
  p.err = a.err;
  p.fused = ws != nullptr;
  p.counters = ws ? ws->counters : nullptr;
  p.final_out = out;
  p.final_lse = out_lse;
  // kv_start and window only move the ranges; the scores themselves change with the other two
  const bool scores = mod.softcap > 0.f || mod.alibi_slopes != nullptr;
  const dim3 grid(a.num_splits, a.num_kv_heads, a.cp * a.num_seqs);
  return a.head_dim == 64 ? launch_d<64>(p, a.dtype, q4, scores, grid, s)
                          : launch_d<128>(p, a.dtype, q4, scores, grid, s);
}
