// What the decode kernels with modified scores and over the 4-bit cache share: the visible range of a
// split, the score modifications, tensor-core helpers and the way from the warps' parts to a result.
#pragma once

#include <math.h>
#include <string.h>

#include "common.cuh"
#include "sm100.cuh"

namespace cpattn {
namespace {

constexpr int kWarps = 4;
constexpr int kPage = 16;
constexpr int kMaxPartials = 256;  // cp * splits of one fused call
constexpr int kMaxCluster = 8;
constexpr float kMaxGrowth = 8.f;  // log2: how far a score may exceed the running reference

// n / d for 0 <= n < 2^31 and a divisor fixed for the launch, as one multiply and one shift
// (Granlund and Montgomery, "Division by invariant integers using multiplication", 1994): a CTA's
// start runs a chain of these before its first load has an address.
struct FastDiv {
  uint32_t d, m, s;
};
FastDiv make_fastdiv(long long d) {
  if (d > 0x7fffffff) d = 0x7fffffff;  // beyond every position: 0 whole periods either way
  uint32_t l = 0;
  while ((1ll << l) < d) ++l;
  const unsigned long long num = 1ull << (31 + l);
  return FastDiv{(uint32_t)d, (uint32_t)((num + (unsigned long long)d - 1) / (unsigned long long)d), 31 + l};
}
CP_DEV int fdiv(int n, const FastDiv& f) { return (int)(((unsigned long long)(uint32_t)n * f.m) >> f.s); }

struct ModParams {
  int B, Hq, Hkv, G, cp, I, S, ST, max_blocks, window;
  FastDiv f_period, f_I;  // I cp, I
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
  int cluster;  // CTAs per cluster (1: none)
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
  if (p.kv_start != nullptr) lo = max(lo, ld(p.kv_start + b));
  return min(lo, max(L, 0));
}
// Tokens of rank r among positions [0, L), L >= 0.
CP_DEV int local_len(const ModParams& p, int L, int r) {
  const int q = fdiv(L, p.f_period);
  const long long rem = (long long)(L - q * (long long)p.f_period.d) - (long long)r * p.I;
  return q * p.I + (int)(rem < 0 ? 0 : (rem > p.I ? p.I : rem));
}
CP_DEV Span rank_span(const ModParams& p, int L, int lo, int r) {
  Span s;
  s.n = L > 0 ? local_len(p, L, r) : 0;
  s.a = lo > 0 ? local_len(p, lo, r) : 0;
  s.a0 = s.a & ~(kPage - 1);
  return s;
}
CP_DEV int live_splits(const ModParams& p, const Span& s) {
  return s.a < s.n ? min(p.S, (int)(((unsigned)(s.n - s.a0) + (unsigned)p.ST - 1u) / (unsigned)p.ST)) : 0;
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

// The CTA's four warps as one: reference and sum of head hh, and (unnormalised) four of its dims.
template <int D, int HR>
CP_DEV void combine_warps(const WarpParts<D, HR>& w, int hh, int dd, float& M, float& L, float4& o) {
  M = -INFINITY;
#pragma unroll
  for (int k = 0; k < kWarps; ++k) M = fmaxf(M, w.m[k][hh]);
  L = 0.f;
  o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int k = 0; k < kWarps; ++k) {
    const float mk = w.m[k][hh];
    // (a warp whose reference is -inf saw no finite score: its sums are 0, or NaN)
    const float e = mk == M || mk == -INFINITY ? 1.f : exp2f(mk - M);
    const float4 x = *reinterpret_cast<const float4*>(&w.o[k][hh][dd]);
    L += e * w.l[k][hh];
    o.x += e * x.x, o.y += e * x.y, o.z += e * x.z, o.w += e * x.w;
  }
}
CP_DEV void scale4(float4& o, float f) { o.x *= f, o.y *= f, o.z *= f, o.w *= f; }
// A sum of weights that is zero means no visible key; NaN stays NaN.
CP_DEV float inverse_sum(float L) { return L == 0.f ? 0.f : 1.f / L; }
CP_DEV float natural_lse(float M, float L) {
  return L == 0.f ? -INFINITY : ((M == -INFINITY ? 0.f : M) + log2f(L)) * kLn2;
}

// Partials in the workspace -> result.  Every CTA publishes what it wrote with one acquire-release
// count per (sequence, kv head) after a CTA barrier; the one that counts last (`arrivals` in all) reads
// the P partials through L2, weighs them by 2^(lse - max) and returns the counter to zero.  No CTA
// waits for another.  live(k): partial k was written.
template <typename T, int D, int HR, typename Live>
CP_DEV void merge_partials(const ModParams& p, WarpParts<D, HR>& w, int b, int g, int P, int arrivals, Live live) {
  constexpr int V = D / 4;  // threads (of 4 dims) per head
  const long long unit0 = (long long)b * p.Hq + (long long)g * p.G;
  const long long stride = (long long)p.B * p.Hq;
  __shared__ int s_last;
  __syncthreads();
  if (threadIdx.x == 0) {
    int prev;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;"
                 : "=r"(prev)
                 : "l"(p.counters + (long long)b * p.Hkv + g)
                 : "memory");
    s_last = prev == arrivals - 1;
  }
  __syncthreads();
  if (!s_last) return;
  // per (partial, head) weights over the warp parts (free now), a warp per head and its partials
  // across the lanes; then the weighted rows
  float* wt = &w.o[0][0][0];
  static_assert(sizeof(w.o) >= kMaxPartials * HR * sizeof(float), "merge weights");
  float* s_M = &w.m[0][0];
  float* s_L = &w.l[0][0];
  const int lane = threadIdx.x & 31;
  for (int hh = threadIdx.x >> 5; hh < p.G; hh += kWarps) {
    float x[kMaxPartials / 32];
    float M = -INFINITY, sum = 0.f;
#pragma unroll
    for (int t = 0; t < kMaxPartials / 32; ++t) {
      const int k = lane + 32 * t;
      x[t] = k < P && live(k) ? __ldcg(p.lse + k * stride + unit0 + hh) * kLog2e : -INFINITY;
    }
#pragma unroll
    for (int t = 0; t < kMaxPartials / 32; ++t) M = fmaxf(M, x[t]);
    M = warp_max(M);
#pragma unroll
    for (int t = 0; t < kMaxPartials / 32; ++t) {
      const float e = x[t] == -INFINITY ? 0.f : exp2f(x[t] - (M == -INFINITY ? 0.f : M));  // NaN stays
      sum += e;
      if (lane + 32 * t < P) wt[(lane + 32 * t) * p.G + hh] = e;
    }
    sum = warp_sum(sum);
    if (lane == 0) {
      s_M[hh] = M;
      s_L[hh] = sum;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.G * V; i += blockDim.x) {
    const int hh = i / V, dd = (i % V) * 4;
    const float* src = p.out + (unit0 + hh) * D + dd;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int U = 16;  // partial rows in flight
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
    const float sum = s_L[hh];
    scale4(acc, inverse_sum(sum));
    put4<T>(p.final_out, (unit0 + hh) * D + dd, acc);
    if (dd == 0 && p.final_lse) p.final_lse[unit0 + hh] = natural_lse(s_M[hh], sum);
  }
  if (threadIdx.x == 0) p.counters[(long long)b * p.Hkv + g] = 0;
}

// ---- clusters: a fused call of few CTAs runs in clusters of neighbouring splits (and ranks), whose
// partials meet in distributed shared memory.  Each CTA merges its share of the heads' dims over the
// cluster; one cluster per (sequence, kv head) writes the result at once, several write one partial
// each for merge_partials.  Against a partial per CTA in global memory this takes a batch of one
// sequence of 1777 tokens (16/2 heads) from 13.2 to 7.7 us.
CP_DEV uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
CP_DEV void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
CP_DEV uint32_t peer_addr(const void* mine, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(sm100::smem_u32(mine)), "r"(rank));
  return a;
}
CP_DEV float peer_ld(uint32_t a) {
  float x;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(a) : "memory");
  return x;
}
CP_DEV float4 peer_ld4(uint32_t a) {
  float4 x;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(a) : "memory");
  return x;
}
// worked: this CTA's warps have parts; else it only takes part in the merge.
template <typename T, int D, int HR>
CP_DEV void finish_cluster(const ModParams& p, WarpParts<D, HR>& w, int b, int g, bool worked) {
  constexpr int V = D / 4;
  __shared__ float c_M[HR], c_L[HR];
  const int C = p.cluster;
  const long long unit0 = (long long)b * p.Hq + (long long)g * p.G;
  const long long stride = (long long)p.B * p.Hq;
  __syncthreads();
  for (int i = threadIdx.x; i < p.G * V; i += blockDim.x) {
    const int hh = i / V, dd = (i % V) * 4;
    float M = -INFINITY, L = 0.f;
    if (worked) {
      float4 o;
      combine_warps(w, hh, dd, M, L, o);
      *reinterpret_cast<float4*>(&w.o[0][hh][dd]) = o;  // (only this thread read these)
    }
    if (dd == 0) {
      c_M[hh] = M;
      c_L[hh] = L;
    }
  }
  cluster_sync();
  const uint32_t rank = cluster_rank();
  const int clusters = (int)gridDim.x / C, mine = (int)blockIdx.x / C;
  for (int i = (int)rank + C * (int)threadIdx.x; i < p.G * V; i += C * (int)blockDim.x) {
    const int hh = i / V, dd = (i % V) * 4;
    float m[kMaxCluster], l[kMaxCluster], M = -INFINITY, L = 0.f;
    float4 x[kMaxCluster], o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c) {
      m[c] = -INFINITY, l[c] = 0.f;
      if (c < C) {
        m[c] = peer_ld(peer_addr(&c_M[hh], c));
        l[c] = peer_ld(peer_addr(&c_L[hh], c));
        x[c] = peer_ld4(peer_addr(&w.o[0][hh][dd], c));
      }
    }
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c) M = fmaxf(M, m[c]);
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c)
      if (l[c] != 0.f) {  // (a CTA without work left its rows as they were)
        const float e = m[c] == M || m[c] == -INFINITY ? 1.f : exp2f(m[c] - M);
        L += e * l[c];
        o.x += e * x[c].x, o.y += e * x[c].y, o.z += e * x[c].z, o.w += e * x[c].w;
      }
    scale4(o, inverse_sum(L));
    if (clusters == 1) {
      put4<T>(p.final_out, (unit0 + hh) * D + dd, o);
      if (dd == 0 && p.final_lse) p.final_lse[unit0 + hh] = natural_lse(M, L);
    } else {
      const long long at = mine * stride + unit0 + hh;
      *reinterpret_cast<float4*>(p.out + at * D + dd) = o;
      if (dd == 0) p.lse[at] = natural_lse(M, L);
    }
  }
  cluster_sync();  // no CTA leaves while another reads its shared memory
  if (clusters > 1)
    merge_partials<T, D, HR>(p, w, b, g, clusters, clusters * C, [](int) { return true; });
}

// Warps -> the CTA's partial, and in a fused call partials -> result.  A (sequence, kv head) with one
// live split writes its result at once.
template <typename T, int D, int HR>
CP_DEV void finish(const ModParams& p, WarpParts<D, HR>& w, int b, int g, int part, int live) {
  constexpr int V = D / 4;
  if (p.cluster > 1) return finish_cluster<T, D, HR>(p, w, b, g, true);
  const long long unit0 = (long long)b * p.Hq + (long long)g * p.G;
  const bool direct = p.fused && live == 1;
  __syncthreads();
  for (int i = threadIdx.x; i < p.G * V; i += blockDim.x) {
    const int hh = i / V, dd = (i % V) * 4;
    float M, L;
    float4 o;
    combine_warps(w, hh, dd, M, L, o);
    scale4(o, inverse_sum(L));
    if (direct) {
      put4<T>(p.final_out, (unit0 + hh) * D + dd, o);
      if (dd == 0 && p.final_lse) p.final_lse[unit0 + hh] = natural_lse(M, L);
    } else {
      const long long at = (long long)part * p.B * p.Hq + unit0 + hh;
      if (L != 0.f || p.fused) *reinterpret_cast<float4*>(p.out + at * D + dd) = o;
      if (dd == 0) p.lse[at] = natural_lse(M, L);
    }
  }
  if (!p.fused || direct) return;
  const int L = ld(p.seq_lens + b), lo = first_visible(p, b, L);
  merge_partials<T, D, HR>(p, w, b, g, p.cp * p.S, live, [&](int k) {
    return k % p.S < live_splits(p, rank_span(p, L, lo, k / p.S));
  });
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

// The CTA's unit of work; false: no visible token falls in it, and what there is to do for it is done.
struct Unit {
  int split, g, r, b, part, live, L;
  int l0, l1, a;  // local tokens [max(l0, a), l1); l0 is the first one of a page
};
template <typename T, int D, int HR>
CP_DEV bool take_unit(const ModParams& p, WarpParts<D, HR>& parts, Unit& u) {
  chained_start();
  u.g = blockIdx.y;
  if (p.cluster > 1) {  // a cluster's CTAs are neighbours in x: parts in order, a few past the last
    u.b = blockIdx.z;
    u.part = blockIdx.x;
    u.r = u.part / p.S;
    u.split = u.part - u.r * p.S;
  } else {
    u.split = blockIdx.x;
    u.r = (int)(blockIdx.z % (unsigned)p.cp);
    u.b = (int)(blockIdx.z / (unsigned)p.cp);
    u.part = u.r * p.S + u.split;
  }
  u.L = ld(p.seq_lens + u.b);
  const int lo = first_visible(p, u.b, u.L);
  u.live = p.fused && p.cluster <= 1 ? live_total(p, u.L, lo) : 0;
  if (u.r < p.cp) {
    const Span s = rank_span(p, u.L, lo, u.r);
    if (s.a < s.n && (long long)p.S * p.ST < s.n - s.a0 && u.split == 0 && threadIdx.x == 0)
      report(p.err, CP_ERR_DEVICE_BOUNDS);  // the plan does not cover this sequence
    const long long l0 = s.a0 + (long long)u.split * p.ST;
    if (s.a < s.n && l0 < s.n) {
      u.a = s.a;
      u.l0 = (int)l0;
      u.l1 = (int)min((long long)s.n, l0 + p.ST);
      return true;
    }
  }
  if (p.cluster > 1) finish_cluster<T, D, HR>(p, parts, u.b, u.g, false);
  else finish_empty<T, D>(p, u.b, u.g, u.r, u.split, u.part, u.live);
  return false;
}

// ------------------------------------------------------------------------------ scores
// cap tanh(x / cap), x = scale q.k, in log2 units: out = cap log2(e), y = x / cap.  Away from 0 as
// 1 - 2 / (1 + e^2y), off by 2^-22 of the cap; near it, where that would be a large part of the score,
// by the series of tanh (next term below 2^-21 of it at |y| = 1/4).
CP_DEV float capped(float x, float inv, float out) {
  const float y = x * inv, u = y * y;
  const float near = x * fmaf(u, fmaf(u, fmaf(u, -17.f / 315.f, 2.f / 15.f), -1.f / 3.f), 1.f);
  const float far = out - __fdividef(2.f * out, 1.f + sm100::ex2(y * (2.f * kLog2e)));
  return fabsf(y) < 0.25f ? near : far;  // (NaN: far, and NaN)
}

// Positions between the query and rank-local token t of the unit's rank.
CP_DEV float distance(const ModParams& p, const Unit& u, int t) {
  const int turn = fdiv(t, p.f_I);
  const long long pos = (long long)turn * p.I * p.cp + (long long)u.r * p.I + (t - turn * p.I);
  return (float)(u.L - 1 - pos);
}

// The modifications of a thread's scores: rows = tokens t, t + 8 (rank-local), columns = heads
// 2 tid, 2 tid + 1 of each tile of 8; log2 units in and out.
template <int NT>
struct Mods {
  float slope[NT][2], cap_in, cap_out;
  CP_DEV Mods(const ModParams& p, const Unit& u, int tid) {
    cap_out = p.softcap * kLog2e;
    cap_in = p.softcap > 0.f ? 1.f / cap_out : 0.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int head = 8 * nt + 2 * tid + c;
        slope[nt][c] = p.slopes != nullptr && head < p.G ? ld(p.slopes + u.g * p.G + head) * kLog2e : 0.f;
      }
  }
  CP_DEV void apply(float (&s)[NT][4], const ModParams& p, const Unit& u, int t) const {
    if (p.softcap > 0.f) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] = capped(s[nt][e], cap_in, cap_out);
    }
    if (p.slopes != nullptr) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float dist = distance(p, u, t + 8 * h);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) s[nt][2 * h + c] = fmaf(-slope[nt][c], dist, s[nt][2 * h + c]);
      }
    }
  }
};

// The reference m (log2) of a head moves up to the largest of this iteration's scores (x: this
// thread's) over the 8 rows of lanes; the factor its sums shrink by.
CP_DEV float new_reference(float x, float& m, float& neg) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
  const float m_new = fmaxf(m, x);
  const float alpha = m_new == m ? 1.f : sm100::ex2(m - m_new);
  m = m_new;
  neg = m_new == -INFINITY ? 0.f : -m_new;
  return alpha;
}
CP_DEV float column_sum(float x) {  // over the 8 lanes with the same columns
  x += __shfl_xor_sync(0xffffffffu, x, 4);
  x += __shfl_xor_sync(0xffffffffu, x, 8);
  x += __shfl_xor_sync(0xffffffffu, x, 16);
  return x;
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

inline ModParams decode_mod_params(const cp_decode_args& a, const cp_score_mod& mod, float scale,
                                   const CpDecodeWorkspace* ws, void* out, float* out_lse) {
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
  p.f_period = make_fastdiv((long long)a.interleave * a.cp);
  p.f_I = make_fastdiv(a.interleave);
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
  p.cluster = 1;
  p.counters = ws ? ws->counters : nullptr;
  p.final_out = out;
  p.final_lse = out_lse;
  return p;
}
// kv_start and window only move the ranges; the scores themselves change with the other two
inline bool changes_scores(const cp_score_mod& mod) { return mod.softcap > 0.f || mod.alibi_slopes != nullptr; }

// Launch of a decode kernel of which per_sm CTAs fit on an SM: fused calls whose CTAs all run at once in
// clusters of up to eight of a (sequence, kv head)'s parts; larger ones without, since a cluster's CTAs
// start and stay together and the empty splits of short sequences would hold their places.  (Clusters of
// eight fill 8 of 9 places: of 152 SMs, up to 405 CTAs at three per SM and 270 at two.)
inline cudaError_t launch_decode(void (*kern)(const ModParams), ModParams p, size_t smem, int per_sm, cudaStream_t s) {
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  const int parts = p.cp * p.S;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  p.cluster = parts > 4 ? 8 : (parts > 2 ? 4 : 2);
  const long long ctas = (long long)(parts + p.cluster - 1) / p.cluster * p.cluster * p.Hkv * p.B;
  if (!p.fused || parts == 1 || 9 * ctas > 8ll * per_sm * sms) p.cluster = 1;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see launch_chained
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (p.cluster > 1) {
    cfg.gridDim = dim3((parts + p.cluster - 1) / p.cluster * p.cluster, p.Hkv, p.B);
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = p.cluster;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  } else {
    cfg.gridDim = dim3(p.S, p.Hkv, p.cp * p.B);
  }
  return cudaLaunchKernelEx(&cfg, kern, (const ModParams)p);
}

}  // namespace
}  // namespace cpattn
