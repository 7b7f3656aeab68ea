// Beam search over a model's logits and its paged round-robin caches: cp_beam_select (the best continuations
// over beams and vocabulary) and cp_beam_reorder (the beams' tables and partly filled pages follow the
// selection).  No counterpart on the pages, whose caches these are: "[Feature] Prefill Context Parallel (PCP)
// basic support" (vLLM PR 28718), Purpose: per-rank block tables.
#include "common.cuh"

namespace cpattn {
namespace {

// ================================================================================ selection
//   score(k, v) = scores[k] + x[k][v] - log sum_u exp(x[k][u])
//
// One pass over the logits.  A row is cut into slices; a CTA holds one in registers (up to eight 16-byte
// vectors a thread, all in flight at once), takes its largest value and its sum of exp(x - largest), and keeps its
// num_candidates largest values: every one of the M best continuations of a beam is among them.  The CTA that
// finishes a sequence's last slice turns slices into beams and beams into the result.
//
// The M largest of many, without sorting: each warp finds the w-th largest of its lanes' maxima, w = ceil(M / 8);
// the least of the eight warps' is a bound that at least M values reach, and few more do (about 3 M of random
// ones), so only those are compared with one another.  Where too many reach it (equal values), the M are taken
// one after the other.
//
// Bound: HBM.  An element costs about six instructions (unpacking, maximum, packed difference, exponential, sum), which
// eight resident warps a sub-partition keep below the time of its load.
constexpr int kThreads = 256, kWarps = 8;
constexpr int kList = 1024;           // values that a CTA compares with one another
constexpr int kMaxBeams = 32, kMaxCandidates = 64;

struct SelectParams {
  int K, V, M, S, eos;
  long long stride;  // elements between rows
  const void* logits;
  const float* scores;
  int32_t* counters;  // [B], zero between calls
  float2* stats;      // [B K][S] largest value and sum
  uint2* best;        // [B K][S][M] value, token (-1: none)
  float *next_score, *cand_score;
  int32_t *next_beam, *next_token, *cand_beam, *cand_token;
};

// Unsigned numbers in the order of the values (no NaN; 0 and -0 are one).
CP_DEV uint32_t order32(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
CP_DEV float value32(uint32_t k) { return __uint_as_float(k ^ ((uint32_t)((int32_t)~k >> 31) | 0x80000000u)); }
CP_DEV unsigned long long order64(double x) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(x + 0.0);
  return u ^ ((unsigned long long)((long long)u >> 63) | 0x8000000000000000ull);
}
CP_DEV double value64(unsigned long long k) {
  return __longlong_as_double((long long)(k ^ ((unsigned long long)((long long)~k >> 63) | 0x8000000000000000ull)));
}

// The w-th largest of the lanes' keys (equal ones count as often as they come).
CP_DEV uint32_t wth_largest(uint32_t key, int w, uint32_t& largest) {
  const uint32_t lane = threadIdx.x & 31;
  uint32_t cur = largest = __reduce_max_sync(0xffffffffu, key);
  for (int i = 1; i < w; ++i) {
    if ((uint32_t)__ffs(__ballot_sync(0xffffffffu, key == cur)) - 1 == lane) key = 0;
    cur = __reduce_max_sync(0xffffffffu, key);
  }
  return cur;
}

// A 16-byte vector of logits as it was loaded, and its elements.  pin: what was made of it before is not kept in
// registers for later (a slice's unpacked values are twice its size: 1 KB of spills a thread).
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  float x[4];
  CP_DEV void load(const float* p) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  }
  CP_DEV void clear() { x[0] = x[1] = x[2] = x[3] = -INFINITY; }
  CP_DEV void put(int i, float v) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j == i) x[j] = v;
  }
  CP_DEV float get(int i) const { return x[i]; }
  CP_DEV float max() const { return fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])); }  // (a NaN is passed over)
  CP_DEV void pin() { asm volatile("" : "+f"(x[0]), "+f"(x[1]), "+f"(x[2]), "+f"(x[3])); }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  uint32_t x[4];
  CP_DEV void load(const __nv_bfloat16* p) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  }
  CP_DEV void clear() { x[0] = x[1] = x[2] = x[3] = 0xff80ff80u; }
  CP_DEV void put(int i, __nv_bfloat16 v) {
    const uint32_t u = (uint32_t)__bfloat16_as_ushort(v);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j == i >> 1) x[j] = (i & 1) ? (x[j] & 0xffffu) | (u << 16) : (x[j] & 0xffff0000u) | u;
  }
  CP_DEV float get(int i) const { return __uint_as_float((i & 1) ? x[i >> 1] & 0xffff0000u : x[i >> 1] << 16); }
  static CP_DEV __nv_bfloat162 pair(uint32_t u) { return *reinterpret_cast<const __nv_bfloat162*>(&u); }
  CP_DEV float max() const {
    const __nv_bfloat162 m = __hmax2(__hmax2(pair(x[0]), pair(x[1])), __hmax2(pair(x[2]), pair(x[3])));
    return fmaxf(__low2float(m), __high2float(m));
  }
  CP_DEV void pin() { asm volatile("" : "+r"(x[0]), "+r"(x[1]), "+r"(x[2]), "+r"(x[3])); }
};

CP_DEV float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// exp(x - top) of a pair, added to sum (packed fp32).  The difference comes first: a logit's own size stays out of it.
CP_DEV void add_exp2(uint64_t& sum, float x, float y, uint64_t minus_top) {
  const float e = kLog2e;
  uint64_t v, w;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
  asm("mov.b64 %0, {%1, %1};" : "=l"(w) : "f"(e));
  asm("add.f32x2 %0, %0, %1;" : "+l"(v) : "l"(minus_top));
  asm("mul.f32x2 %0, %0, %1;" : "+l"(v) : "l"(w));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
  x = ex2_approx(x);
  y = ex2_approx(y);
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
  asm("add.f32x2 %0, %0, %1;" : "+l"(sum) : "l"(v));
}

// The block's sum, the same for every thread.
CP_DEV float block_sum(float x, float* s_warp) {
  x = warp_sum(x);
  if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = x;
  __syncthreads();
  float r = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) r += s_warp[w];
  return r;
}
// The largest (key, lower index first) of the block; s_key / s_at hold a pair of each warp.
CP_DEV void block_best(unsigned long long& key, unsigned long long& at, unsigned long long* s_key,
                       unsigned long long* s_at) {
  auto take = [&](unsigned long long k, unsigned long long a) {
    if (k > key || (k == key && a < at)) key = k, at = a;
  };
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long k = __shfl_xor_sync(0xffffffffu, key, o), a = __shfl_xor_sync(0xffffffffu, at, o);
    take(k, a);
  }
  __syncthreads();  // (the pairs of the round before have been read)
  if ((threadIdx.x & 31) == 0) s_key[threadIdx.x >> 5] = key, s_at[threadIdx.x >> 5] = at;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) take(s_key[w], s_at[w]);
}

// log2 of a positive sum: its exponent apart, so that the logarithm's rounding is that of a number below 0.6.
CP_DEV double log2_split(float s) {
  const int e = (int)((__float_as_uint(s) + 0x004afb0du) >> 23) - 127;  // s / 2^e in about [0.71, 1.42)
  return (double)e + (double)log2f(ldexpf(s, -e));
}
constexpr double kLn2d = 0.69314718055994530942;

struct SelectShared {
  unsigned long long key[kList], at[kList];
  unsigned long long w_key[kWarps], w_at[kWarps];
  double base[kMaxBeams];  // score of the beam's largest logit
  float top[kMaxBeams];    // that logit
  unsigned long long top_key[kMaxCandidates], top_at[kMaxCandidates];
  uint32_t w_max[kWarps], w_th[kWarps];
  float w_sum[kWarps];
  int n, last;
  unsigned char full[kMaxBeams], taken[kMaxCandidates];
};

// The M best of a sequence, from its slices' sums and values, and the result.
CP_DEV void finish_sequence(const SelectParams& p, SelectShared& sh, int b) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // ---- beams: largest logit and its score.  full: some logit is +inf, and the probability lies on those alone.
  for (int k = warp; k < p.K; k += kWarps) {
    const long long row = (long long)b * p.K + k;
    const float2* st = p.stats + row * p.S;
    float top = -INFINITY, sum = 0.f;
    for (int s = lane; s < p.S; s += 32) top = fmaxf(top, __ldcg(&st[s]).x);
    top = warp_max(top);
    for (int s = lane; s < p.S; s += 32) {
      const float2 x = __ldcg(&st[s]);
      if (x.x > -INFINITY) sum += x.y * (x.x == top ? 1.f : exp2f((x.x - top) * kLog2e));
    }
    sum = warp_sum(sum);
    if (lane == 0) {
      const float from = ld(p.scores + row);
      sh.full[k] = top == INFINITY;
      sh.top[k] = top;
      sh.base[k] = sum > 0.f && from > -INFINITY ? (double)from - kLn2d * log2_split(sum) : -INFINITY;
    }
  }
  if (tid == 0) sh.n = 0;
  __syncthreads();
  // ---- continuations in the order of (score, lower beam and token first)
  const int per = p.S * p.M, n_all = p.K * per;
  const uint2* best = p.best + (long long)b * n_all;
  auto entry = [&](int i, unsigned long long& key, unsigned long long& at) -> bool {  // false: no probability
    const uint2 e = __ldcg(best + i);
    const int k = i / per;
    const double base = sh.base[k];
    const float x = __uint_as_float(e.x);
    if ((int32_t)e.y < 0 || base == -INFINITY || (sh.full[k] && x != INFINITY)) return false;
    key = order64(sh.full[k] ? base : base + ((double)x - (double)sh.top[k]));
    at = (unsigned long long)k * (unsigned)p.V + e.y;
    return true;
  };
  uint32_t mine = 0;
  for (int i = tid; i < n_all; i += kThreads) {
    unsigned long long key, at;
    if (entry(i, key, at)) mine = max(mine, (uint32_t)(key >> 32));
  }
  uint32_t largest;
  const uint32_t wth = wth_largest(mine, (p.M + kWarps - 1) / kWarps, largest);
  if (lane == 0) sh.w_th[warp] = wth;
  __syncthreads();
  uint32_t bound = 0xffffffffu;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) bound = min(bound, sh.w_th[w]);
  for (int i = tid; i < n_all; i += kThreads) {
    unsigned long long key, at;
    if (entry(i, key, at) && (uint32_t)(key >> 32) >= bound) {
      const int j = atomicAdd(&sh.n, 1);
      if (j < kList) sh.key[j] = key, sh.at[j] = at;
    }
  }
  __syncthreads();
  int n = sh.n;
  if (n <= kList) {
    for (int i = tid; i < n; i += kThreads) {
      const unsigned long long key = sh.key[i], at = sh.at[i];
      int rank = 0;
      for (int j = 0; j < n; ++j) rank += sh.key[j] > key || (sh.key[j] == key && sh.at[j] < at);
      if (rank < p.M) sh.top_key[rank] = key, sh.top_at[rank] = at;
    }
    n = min(n, p.M);
  } else {  // many equal scores: one after the other
    unsigned long long last_key = ~0ull, last_at = 0;
    n = p.M;
    for (int r = 0; r < p.M; ++r) {
      unsigned long long key = 0, at = ~0ull;
      for (int i = tid; i < n_all; i += kThreads) {
        unsigned long long k, a;
        if (!entry(i, k, a)) continue;
        if ((k < last_key || (k == last_key && a > last_at)) && (k > key || (k == key && a < at))) key = k, at = a;
      }
      block_best(key, at, sh.w_key, sh.w_at);
      if (tid == 0) sh.top_key[r] = key, sh.top_at[r] = at;
      last_key = key, last_at = at;
    }
  }
  __syncthreads();
  // ---- fewer than M with a probability: the rest are the first of the others, of score -inf
  if (n < p.M) {
    if (tid < kMaxCandidates) sh.taken[tid] = 0;
    __syncthreads();
    if (tid < n && sh.top_at[tid] < kMaxCandidates) sh.taken[sh.top_at[tid]] = 1;
    __syncthreads();
    if (tid == 0)
      for (int r = n, f = 0; r < p.M; ++f)
        if (!sh.taken[f]) sh.top_key[r] = order64(-INFINITY), sh.top_at[r] = (unsigned long long)f, ++r;
    __syncthreads();
  }
  // ---- all M, and the first K that go on
  if (warp == 0) {
    int on = 0;
    for (int r0 = 0; r0 < p.M; r0 += 32) {
      const int r = r0 + lane;
      const bool real = r < p.M;
      const unsigned long long at = real ? sh.top_at[r] : 0ull;
      const int beam = (int)(at / (unsigned)p.V), token = (int)(at % (unsigned)p.V);
      const float score = real ? (float)value64(sh.top_key[r]) : 0.f;
      if (real) {
        const long long o = (long long)b * p.M + r;
        p.cand_score[o] = score, p.cand_beam[o] = beam, p.cand_token[o] = token;
      }
      const bool goes = real && token != p.eos;
      const uint32_t mask = __ballot_sync(0xffffffffu, goes);
      const int j = on + __popc(mask & ((1u << lane) - 1u));
      if (goes && j < p.K) {
        const long long o = (long long)b * p.K + j;
        p.next_score[o] = score, p.next_beam[o] = beam, p.next_token[o] = token;
      }
      on += __popc(mask);
    }
  }
}

// NV: vectors a thread holds; a slice is NV * 256 of them, counted from the row's first 16-byte boundary.
template <typename T, int NV>
__global__ void __launch_bounds__(kThreads, NV >= 8 ? 4 : 5) select_kernel(const SelectParams p) {
  using W = Vec<T>;
  __shared__ SelectShared sh;
  chained_start();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long row = blockIdx.x / (unsigned)p.S;
  const int slice = (int)(blockIdx.x % (unsigned)p.S), b = (int)(row / p.K);
  const T* x = static_cast<const T*>(p.logits) + row * p.stride;
  const int skew = (int)((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));  // elements before the row in its first vector
  if (tid == 0) sh.n = 0;

  // ---- the slice in registers, what is no token as -inf
  W v[NV];
  int e0 = (slice * (NV * kThreads) + tid) * W::N - skew;
  auto first = [&](int i) -> int { return e0 + i * (kThreads * W::N); };  // element of v[i].get(0)
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = first(i);
    if (e >= 0 && e + W::N <= p.V) {
      v[i].load(x + e);
    } else {
      v[i].clear();
#pragma unroll
      for (int j = 0; j < W::N; ++j)
        if (e + j >= 0 && e + j < p.V) v[i].put(j, x[e + j]);
    }
  }
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < NV; ++i) top = fmaxf(top, v[i].max());

  // ---- the slice's largest value, and a bound that at least M values reach
  uint32_t largest;
  const uint32_t wth = wth_largest(order32(top), (p.M + kWarps - 1) / kWarps, largest);
  if (lane == 0) sh.w_max[warp] = largest, sh.w_th[warp] = wth;
  __syncthreads();
  uint32_t bound = 0xffffffffu;
  largest = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) largest = max(largest, sh.w_max[w]), bound = min(bound, sh.w_th[w]);
  const float most = value32(largest), least = value32(bound);

  auto pin = [&]() {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i].pin();
  };
  pin();
  // ---- sum, relative to the largest
  float sum = 0.f;
  if (most > -INFINITY) {
    uint64_t part[2] = {0ull, 0ull}, minus;  // pairs of sums
    asm("mov.b64 %0, {%1, %1};" : "=l"(minus) : "f"(-most));
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < W::N; j += 2) add_exp2(part[(j >> 1) & 1], v[i].get(j), v[i].get(j + 1), minus);
    float s[4];
    asm("mov.b64 {%0, %1}, %2;" : "=f"(s[0]), "=f"(s[1]) : "l"(part[0]));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(s[2]), "=f"(s[3]) : "l"(part[1]));
    sum = (s[0] + s[1]) + (s[2] + s[3]);
    if (!(sum < INFINITY)) {  // a NaN, which counts as -inf, or infinities, which share the probability
      sum = 0.f;
      pin();
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < W::N; ++j) {
          const float y = v[i].get(j);
          sum += y == most ? 1.f : y < most ? ex2_approx((y - most) * kLog2e) : 0.f;
        }
    }
  }

  pin();
  // ---- the values that reach the bound
  if (top >= least && top > -INFINITY) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (v[i].max() >= least)
#pragma unroll
        for (int j = 0; j < W::N; ++j) {
          const float y = v[i].get(j);
          if (y >= least && y > -INFINITY) {
            const int at = atomicAdd(&sh.n, 1);
            if (at < kList) sh.key[at] = ((unsigned long long)order32(y) << 32) | (0xffffffffu - (uint32_t)(first(i) + j));
          }
        }
  }
  sum = block_sum(sum, sh.w_sum);  // (a barrier: the list is complete)
  const long long part = row * p.S + slice;
  uint2* best = p.best + part * p.M;
  const int n = sh.n;
  auto keep = [&](int r, unsigned long long key) {
    best[r] = make_uint2(__float_as_uint(value32((uint32_t)(key >> 32))), 0xffffffffu - (uint32_t)key);
  };
  if (n <= kList) {
    for (int i = tid; i < n; i += kThreads) {
      const unsigned long long key = sh.key[i];
      int rank = 0;
      for (int j = 0; j < n; ++j) rank += sh.key[j] > key;
      if (rank < p.M) keep(rank, key);
    }
    for (int r = n + tid; r < p.M; r += kThreads) best[r] = make_uint2(0xff800000u, 0xffffffffu);
  } else {  // many equal values: one after the other
    unsigned long long last = ~0ull;
    for (int r = 0; r < p.M; ++r) {
      unsigned long long key = 0, none = 0;
      pin();
      asm volatile("" : "+r"(e0));
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < W::N; ++j) {
          const float y = v[i].get(j);
          if (y >= least && y > -INFINITY) {
            const unsigned long long k = ((unsigned long long)order32(y) << 32) | (0xffffffffu - (uint32_t)(first(i) + j));
            if (k < last && k > key) key = k;
          }
        }
      block_best(key, none, sh.w_key, sh.w_at);
      if (tid == 0) keep(r, key);
      last = key;
    }
  }
  if (tid == 0) p.stats[part] = make_float2(most, sum);

  // ---- the CTA that counts last has every slice of the sequence before it
  __syncthreads();
  if (tid == 0) {
    int before;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(before) : "l"(p.counters + b) : "memory");
    sh.last = before == p.K * p.S - 1;
    if (sh.last) p.counters[b] = 0;
  }
  __syncthreads();
  if (sh.last) finish_sequence(p, sh, b);
}

// Slices: as long as leaves every SM some CTAs (the shorter ones cost more merging).
struct SelectPlan {
  int NV, S;
};
SelectPlan select_plan(long long rows, int V, int elem) {
  // 16-byte vectors that a row touches, which may start anywhere in one
  const long long vecs = ((long long)V * elem + 16 - elem + 15) / 16;
  for (int NV = 8; NV > 1; NV /= 2) {
    const long long S = (vecs + NV * kThreads - 1) / (NV * kThreads);
    if (rows * S >= 2 * 152) return {NV, (int)S};
  }
  return {1, (int)((vecs + kThreads - 1) / kThreads)};
}
// Workspace: counters, each slice's sum, each slice's values.
size_t select_layout(size_t slices, int M, size_t* stats, size_t* best) {
  const size_t c = cp_align256(kCpDecodeCounters * sizeof(int32_t)), st = cp_align256(slices * sizeof(float2));
  *stats = c;
  *best = c + st;
  return c + st + cp_align256(slices * M * sizeof(uint2));
}

template <typename T>
cudaError_t launch_select(const cp_beam_select_args& a, void* workspace, cudaStream_t s) {
  const SelectPlan plan = select_plan((long long)a.num_seqs * a.num_beams, a.vocab, sizeof(T));
  size_t o_stats, o_best;
  select_layout((size_t)a.num_seqs * a.num_beams * plan.S, a.num_candidates, &o_stats, &o_best);
  SelectParams p;
  p.K = a.num_beams;
  p.V = a.vocab;
  p.M = a.num_candidates;
  p.S = plan.S;
  p.eos = a.eos_token;
  p.stride = a.logits_stride;
  p.logits = a.logits;
  p.scores = a.scores;
  p.counters = static_cast<int32_t*>(workspace);
  p.stats = reinterpret_cast<float2*>(static_cast<char*>(workspace) + o_stats);
  p.best = reinterpret_cast<uint2*>(static_cast<char*>(workspace) + o_best);
  p.next_score = a.next_scores, p.next_beam = a.next_beams, p.next_token = a.next_tokens;
  p.cand_score = a.cand_scores, p.cand_beam = a.cand_beams, p.cand_token = a.cand_tokens;
  const dim3 grid((unsigned)((long long)a.num_seqs * a.num_beams * plan.S));
  auto kern = plan.NV == 8   ? select_kernel<T, 8>
              : plan.NV == 4 ? select_kernel<T, 4>
              : plan.NV == 2 ? select_kernel<T, 2>
                             : select_kernel<T, 1>;
  return launch_chained(kern, grid, kThreads, 0, s, p);
}

// ================================================================================ reordering
// Beam j of a sequence goes on from parent p_j.  Of its L cached tokens rank r holds L_r: columns before
// L_r / 16 are full pages, shared by table; the page being filled belongs to one beam, so its L_r mod 16 rows are
// copied from the parent's to beam j's own.
//
// A beam's own page may be another's source, so nothing is written before all that it replaces has been read: a
// thread owns one 16-byte place of the page (row, vector), loads it from the K parents' pages and stores it to the
// K beams' pages.  No shared memory, no barrier, K loads in flight a thread.  The tables go the same way, a
// thread a column.  Tables that are replaced in place wait for the pages' copies in a launch of their own.
// Bound: HBM for the full batch, else the launch and one chain of dependent loads (length, table entry, rows).
struct ReorderParams {
  int B, K, cp, I, max_blocks, Hkv, layers2, chunks;  // layers2: pools of K and of V; chunks: CTAs a pool
  int row_vecs, head_vecs, tail_at, tail_words;       // 16-byte vectors of a row and of a head's page; 4-bit records: place and words a row of the scales
  long long pool, layer_vecs;
  const int32_t *parents, *seq_lens, *tables_in, *own;
  int32_t* tables_out;  // null: pages only
  uint4 *k, *v;         // null: tables only
  int32_t* err;
};

// 1-D grid: (sequence, rank) slowest; within it the tables' CTA first (it has the most to do), then pools and chunks.
template <int KMAX>
__global__ void __launch_bounds__(256) reorder_kernel(const ReorderParams p) {
  __shared__ int s_parent[KMAX];
  __shared__ long long s_src[KMAX], s_dst[KMAX];  // pages; -1: nothing to copy
  chained_start();
  const int tables = p.tables_out != nullptr ? 1 : 0;
  const unsigned per = (unsigned)(tables + (p.k != nullptr ? p.layers2 * p.chunks : 0));
  const unsigned unit = blockIdx.x / per, job = blockIdx.x % per;
  const int b = (int)(unit / (unsigned)p.cp), r = (int)(unit % (unsigned)p.cp);
  const int L = ld(p.seq_lens + b);
  const int held = L > 0 ? rank_local_len(L, r, p.cp, p.I) : 0;
  const int col = held / 16, fill = held % 16;
  const long long row0 = ((long long)r * p.B + b) * p.K;  // of the tables
  // the tables do not hold so many tokens (rank 0 has the most)
  const bool bad = L < 0 || (L > 0 ? rank_local_len(L, 0, p.cp, p.I) : 0) > 16ll * p.max_blocks;
  const bool first = job == 0;
  if (bad) {
    if (first && threadIdx.x == 0) report(p.err, CP_ERR_DEVICE_BOUNDS);
    return;
  }
  if (threadIdx.x < p.K) {
    const int j = threadIdx.x;
    int parent = ld(p.parents + (long long)b * p.K + j);
    if (parent < 0 || parent >= p.K) {
      if (first) report(p.err, CP_ERR_DEVICE_BOUNDS);
      parent = -1;
    }
    s_parent[j] = parent;
    long long src = -1, dst = -1;
    if (parent >= 0 && col < p.max_blocks) {
      dst = ld(p.own + (row0 + j) * p.max_blocks + col);
      if (dst < 0 || dst >= p.pool) {
        if (first) report(p.err, CP_ERR_DEVICE_BOUNDS);
        dst = -1;
      } else if (fill > 0) {
        src = ld(p.tables_in + (row0 + parent) * p.max_blocks + col);
        if (src < 0 || src >= p.pool) {
          if (first) report(p.err, CP_ERR_DEVICE_BOUNDS);
          src = -1;
        }
      }
    }
    s_src[j] = src;
    s_dst[j] = dst;
  }
  __syncthreads();

  if (tables && job == 0) {
    for (int c = threadIdx.x; c <= col && c < p.max_blocks; c += blockDim.x) {
      int32_t id[KMAX];
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if (j < p.K && s_parent[j] >= 0)
          id[j] = c == col && s_dst[j] >= 0 ? (int32_t)s_dst[j] : ld(p.tables_in + (row0 + s_parent[j]) * p.max_blocks + c);
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if (j < p.K && s_parent[j] >= 0) p.tables_out[(row0 + j) * p.max_blocks + c] = id[j];
    }
    return;
  }
  if (fill == 0) return;
  const int pool = (int)(job - tables) / p.chunks, chunk = (int)(job - tables) % p.chunks;
  uint4* base = ((pool & 1) ? p.v : p.k) + (pool >> 1) * p.layer_vecs + (long long)r * p.pool * p.Hkv * p.head_vecs;
  const long long page = (long long)p.Hkv * p.head_vecs;
  auto moves = [&](int j) -> bool { return j < p.K && s_src[j] >= 0 && s_dst[j] >= 0 && s_src[j] != s_dst[j]; };
  for (int i = chunk * 256 + threadIdx.x; i < p.Hkv * fill * p.row_vecs; i += p.chunks * 256) {
    const int q = i / p.row_vecs, h = q / fill;
    uint4* place = base + (long long)h * p.head_vecs + (q % fill) * p.row_vecs + i % p.row_vecs;
    uint4 x[KMAX];
#pragma unroll
    for (int j = 0; j < KMAX; ++j)
      if (moves(j)) x[j] = place[s_src[j] * page];
#pragma unroll
    for (int j = 0; j < KMAX; ++j)
      if (moves(j)) place[s_dst[j] * page] = x[j];
  }
  if (p.tail_words > 0) {  // 4-bit records: the rows' scales and minima
    for (int i = chunk * 256 + threadIdx.x; i < p.Hkv * fill * p.tail_words; i += p.chunks * 256) {
      const int h = i / (fill * p.tail_words);
      uint32_t* place = reinterpret_cast<uint32_t*>(base + (long long)h * p.head_vecs + p.tail_at) + i % (fill * p.tail_words);
      uint32_t x[KMAX];
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if (moves(j)) x[j] = place[s_src[j] * page * 4];
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if (moves(j)) place[s_dst[j] * page * 4] = x[j];
    }
  }
}

cudaError_t reorder_launch(const ReorderParams& p, cudaStream_t s) {
  const long long per = (p.tables_out != nullptr ? 1 : 0) + (p.k != nullptr ? (long long)p.layers2 * p.chunks : 0);
  const long long grid = (long long)p.B * p.cp * per;
  if (grid == 0) return cudaSuccess;
  if (grid >= (1ll << 31)) return cudaErrorInvalidConfiguration;
  auto kern = p.K <= 4 ? reorder_kernel<4> : p.K <= 8 ? reorder_kernel<8> : p.K <= 16 ? reorder_kernel<16> : reorder_kernel<32>;
  return launch_chained(kern, dim3((unsigned)grid), 256, 0, s, p);
}

}  // namespace
}  // namespace cpattn

// Enough for either type and for every smaller size: shorter slices are taken only where there are fewer than 2 * 152
// of twice their length.
size_t cp_beam_select_bytes(int32_t num_seqs, int32_t num_beams, int32_t vocab, int32_t num_candidates) {
  using namespace cpattn;
  const size_t rows = (size_t)num_seqs * num_beams;
  const size_t longest = rows * (((size_t)vocab * 4 + 15) / 16 / (8 * kThreads) + 1);
  size_t a, b;
  return select_layout(longest > 4 * 152 ? longest : 4 * 152, num_candidates, &a, &b);
}
long long cp_beam_select_ctas(const cp_beam_select_args& a) {
  const long long rows = (long long)a.num_seqs * a.num_beams;
  return rows * cpattn::select_plan(rows, a.vocab, a.dtype == CP_BF16 ? 2 : 4).S;
}
cudaError_t cp_launch_beam_select(const cp_beam_select_args& a, void* workspace, cudaStream_t s) {
  return a.dtype == CP_BF16 ? cpattn::launch_select<__nv_bfloat16>(a, workspace, s)
                            : cpattn::launch_select<float>(a, workspace, s);
}

cudaError_t cp_launch_beam_reorder(const cp_beam_reorder_args& a, cudaStream_t s) {
  cpattn::ReorderParams p;
  p.B = a.num_seqs;
  p.K = a.num_beams;
  p.cp = a.cp;
  p.I = a.interleave;
  p.max_blocks = a.max_blocks;
  p.Hkv = a.num_kv_heads;
  p.layers2 = 2 * a.num_layers;
  const int row_bytes = a.cache_q4 ? a.head_dim / 2 : a.head_dim * (a.dtype == CP_BF16 ? 2 : 4);
  p.row_vecs = row_bytes / 16;
  p.head_vecs = (a.cache_q4 ? 9 * a.head_dim : 16 * row_bytes) / 16;
  p.tail_at = a.cache_q4 ? 8 * a.head_dim / 16 : 0;
  p.tail_words = a.cache_q4 ? a.head_dim / 64 : 0;
  p.chunks = (p.Hkv * 15 * p.row_vecs + 511) / 512;  // two places a thread at most
  p.pool = a.pool_pages;
  p.layer_vecs = (long long)a.cp * a.pool_pages * a.num_kv_heads * p.head_vecs;
  p.parents = a.parents;
  p.seq_lens = a.seq_lens;
  p.tables_in = a.tables_in;
  p.own = a.own_pages;
  p.tables_out = a.tables_out;
  p.k = static_cast<uint4*>(a.k_cache);
  p.v = static_cast<uint4*>(a.v_cache);
  p.err = a.err;
  if (a.tables_out != a.tables_in || p.k == nullptr) return cpattn::reorder_launch(p, s);
  p.tables_out = nullptr;
  const cudaError_t e = cpattn::reorder_launch(p, s);
  if (e != cudaSuccess) return e;
  p.tables_out = a.tables_out;
  p.k = p.v = nullptr;
  return cpattn::reorder_launch(p, s);
}
