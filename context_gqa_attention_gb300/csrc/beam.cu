// Beam search over a model's logits and its paged round-robin caches: cp_beam_select (the best continuations
// over beams and vocabulary) and cp_beam_reorder (the beams' tables and partly filled pages follow the
// selection).  No counterpart on the pages, whose caches these are: "[Feature] Prefill Context Parallel (PCP)
// basic support" (vLLM PR 28718), Purpose: per-rank block tables.
#include <type_traits>

#include "common.cuh"

namespace cpattn {
namespace {

// ================================================================================ selection
//   score(k, v) = scores[k] + x[k][v] - log sum_u exp(x[k][u])
//
// One pass over the logits.  A row is cut into chunks, one a CTA (one a row when there are rows for the whole GPU).
// A CTA streams its chunk through registers, the next vectors on their way while these are worked on, sums
// exp(x - reference) and keeps what may be among its num_candidates largest values: every one of the M best
// continuations of a beam is among those.  The CTA that finishes a sequence's last chunk turns chunks into beams and
// beams into the result.
//
// The M largest of many, without sorting: a lane knows the largest value it has met.  The w-th largest of a warp's 32
// is a number that w values of the warp reach, so with w = ceil(M / 8) the least of the eight warps' is one that at least
// M values reach.  Vectors below it are passed over; the others (about 30 in the first 16 KB, then ever fewer, as the
// bound rises with the chunk) go to a list, and at the end those of their values that reach the last bound are
// compared with one another.  Only the first bound takes a barrier: an older one is as valid.
// A list that overflows (rising or equal values) is made again with the last bound, and if that fails too the M are
// taken one after the other.
//
// Bound: HBM.  An element costs about five instructions (unpacking, maximum, packed difference and product,
// exponential, sum), half of what the SM could issue in the time of its load.  64 x 8 rows of 128000 bf16 logits take 32.3
// us (4.06 TB/s, 60% of the copy): 21 us of stream at the copy's rate, then 7 in which all rows sum, list and rank at once.
// One sequence of 4 x 32000 f32: 5.5 us, latency.  Not kept: two to four chunks a row for that batch (38 to 40 us), three CTAs
// an SM, scalar exponentials (the same).
constexpr int kThreads = 256, kWarps = 8;
constexpr int kVecs = 512;            // vectors that a chunk's values are taken from
constexpr int kList = 1024;           // values that a CTA compares with one another
constexpr int kDirect = 96;           // of few values every thread counts those before its own; of more, four threads
constexpr int kMaxBeams = 32, kMaxCandidates = 64;
constexpr float kMaxGrowth = 11.f;    // a lane's values may exceed what its sum is relative to (in log2 units below 16, where
                                      // an exponent is rounded by 2^-21 at most)
constexpr float kMaxLogit = 1e5f;     // beyond, the rounding of log2(e) times a logit is too coarse for one pass
constexpr float kMost = 3.402823466e38f;  // the largest finite value

struct SelectParams {
  int K, V, M, S, chunk, eos;  // S: chunks of a row, chunk: their 16-byte vectors
  long long stride;  // elements between rows
  const void* logits;
  const float* scores;
  int32_t* counters;  // [B], zero between calls
  float2* stats;      // [B K][S] largest value, sum of exp(x - largest)
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

CP_DEV float to_float(float x) { return x; }
CP_DEV float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
// A 16-byte vector of logits as it was loaded, and its elements.
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
  CP_DEV uint4 raw() const {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
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
  CP_DEV uint4 raw() const { return make_uint4(x[0], x[1], x[2], x[3]); }
};

CP_DEV float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^(x log2(e) - c) of a pair, added to sum (packed fp32).
CP_DEV void add_exp2(uint64_t& sum, float x, float y, uint64_t log2e, uint64_t minus_c) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
  asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(v) : "l"(log2e), "l"(minus_c));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
  x = ex2_approx(x);
  y = ex2_approx(y);
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
  asm("add.f32x2 %0, %0, %1;" : "+l"(sum) : "l"(v));
}
CP_DEV float low(uint64_t pair) { return __uint_as_float((uint32_t)pair); }
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

// A number as the sum of two fp32, the first of them the rounded sum: 48 bits, in fp32 arithmetic (Knuth's and Dekker's
// exact sums), since fp64 is slow here.  Scores of different beams are compared in it.
struct Pair {
  float hi, lo;
};
CP_DEV Pair exact_sum(float a, float b) {
  const float s = __fadd_rn(a, b), z = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, z)), __fsub_rn(b, z))};
}
CP_DEV Pair add(Pair a, Pair b) {
  const Pair s = exact_sum(a.hi, b.hi);
  const float e = __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)), hi = __fadd_rn(s.hi, e);
  return {hi, fabsf(hi) <= kMost ? __fsub_rn(e, __fsub_rn(hi, s.hi)) : 0.f};
}
CP_DEV unsigned long long order_pair(Pair x) { return ((unsigned long long)order32(x.hi) << 32) | order32(x.lo); }
// -log of a positive sum: the exponent apart, ln 2 in two parts of which the first has 15 bits (its products are exact),
// so that the roundings are those of numbers below 0.5.
CP_DEV Pair minus_log(float s) {
  const int e = (int)((__float_as_uint(s) + 0x004afb0du) >> 23) - 127;  // s / 2^e in about [0.71, 1.42)
  const float n = (float)e, l = logf(__uint_as_float(__float_as_uint(s) - ((uint32_t)e << 23)));
  return exact_sum(-n * 0.693145751953125f, -fmaf(n, 1.42860682030941723e-6f, l));
}

struct SelectShared {
  uint4 vec[kVecs];  // of the chunk; then places [kList] of a sequence's candidates
  unsigned long long key[kList];
  int id[kVecs], rank[kList];
  unsigned long long w_key[kWarps], w_at[kWarps];
  unsigned long long top_key[kMaxCandidates], top_at[kMaxCandidates];
  Pair base[kMaxBeams];  // score of the beam's largest logit
  float top[kMaxBeams];  // that logit
  uint32_t w_max[kWarps];
  alignas(16) uint32_t w_th[kWarps];
  float w_sum[kWarps];
  int n, n2, last;
  unsigned char taken[kMaxCandidates];
  // what each warp publishes, as of now: the least of them
  CP_DEV uint32_t bound() const {
    uint32_t k[kWarps];
    const uint32_t a = (uint32_t)__cvta_generic_to_shared(w_th);
#pragma unroll
    for (int i = 0; i < kWarps; i += 4)
      asm volatile("ld.volatile.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(k[i]), "=r"(k[i + 1]), "=r"(k[i + 2]), "=r"(k[i + 3]) : "r"(a + 4u * i) : "memory");
#pragma unroll
    for (int i = 1; i < kWarps; ++i) k[0] = min(k[0], k[i]);
    return k[0];
  }
  CP_DEV unsigned long long* at() { return reinterpret_cast<unsigned long long*>(vec); }
};
static_assert(sizeof(uint4) * kVecs >= sizeof(unsigned long long) * kList, "places");

// rank[i]: how many of the list's n entries come before entry i (which starts at 0).  Four threads an entry.
template <bool PLACES>
CP_DEV void count_before(SelectShared& sh, int n) {
  const int per = (n + 3) / 4, j0 = ((int)threadIdx.x >> 6) * per, j1 = min(n, j0 + per);
#pragma unroll 1
  for (int i = threadIdx.x & 63; i < n; i += 64) {
    const unsigned long long key = sh.key[i], at = PLACES ? sh.at()[i] : 0ull;
    int r = 0;
#pragma unroll 4
    for (int j = j0; j < j1; ++j)
      r += sh.key[j] > key || (PLACES && sh.key[j] == key && sh.at()[j] < at);
    if (r > 0) atomicAdd(&sh.rank[i], r);
  }
  __syncthreads();
}

// One of a sequence's candidates as (score, place), which order them; false: it has no probability.
CP_DEV bool candidate(const SelectShared& sh, uint2 e, int k, unsigned long long& key, unsigned long long& at) {
  const Pair base = sh.base[k];
  const float x = __uint_as_float(e.x), top = sh.top[k];
  const Pair score = top == INFINITY ? base : add(base, exact_sum(x, -top));
  key = order_pair(score);
  at = ((unsigned long long)k << 32) | e.y;
  return (int32_t)e.y >= 0 && base.hi > -INFINITY && score.hi > -INFINITY && (top < INFINITY || x == INFINITY);
}
// Many equal scores: the M best one after the other.
__device__ __noinline__ void slow_finish(const uint2* best, int n_all, int per, int M, SelectShared& sh) {
  unsigned long long last_key = ~0ull, last_at = 0;
  for (int r = 0; r < M; ++r) {
    unsigned long long key = 0, at = ~0ull;
    for (int i = threadIdx.x; i < n_all; i += kThreads) {
      unsigned long long k, a;
      if (!candidate(sh, __ldcg(best + i), i / per, k, a)) continue;
      if ((k < last_key || (k == last_key && a > last_at)) && (k > key || (k == key && a < at))) key = k, at = a;
    }
    block_best(key, at, sh.w_key, sh.w_at);
    if (threadIdx.x == 0) sh.top_key[r] = key, sh.top_at[r] = at;
    last_key = key, last_at = at;
  }
}
// Fewer than M with a probability: the rest are the first of the others, of score -inf.
__device__ __noinline__ void fill_up(int n, int M, int V, SelectShared& sh) {
  const int tid = threadIdx.x;
  if (tid < kMaxCandidates) sh.taken[tid] = 0;
  __syncthreads();
  if (tid < n) {
    const unsigned long long flat = (sh.top_at[tid] >> 32) * (unsigned)V + (uint32_t)sh.top_at[tid];
    if (flat < kMaxCandidates) sh.taken[flat] = 1;
  }
  __syncthreads();
  if (tid == 0)
    for (int r = n, f = 0; r < M; ++f)
      if (!sh.taken[f]) {
        sh.top_key[r] = order_pair({-INFINITY, 0.f});
        sh.top_at[r] = ((unsigned long long)(f / V) << 32) | (unsigned)(f % V);
        ++r;
      }
}

// The M best of a sequence, from its chunks' sums and values, and the result.
CP_DEV void finish_sequence(const SelectParams& p, SelectShared& sh, int b) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = p.S * p.M, n_all = p.K * per;
  const uint2* best = p.best + (long long)b * n_all;
  // every warp has its share of a few candidates, and of each place in the chunks' lists
  const int i0 = lane * kWarps + ((warp + lane) & (kWarps - 1));
  const uint2 e0 = i0 < n_all ? __ldcg(best + i0) : make_uint2(0u, 0xffffffffu);  // on its way meanwhile
  // ---- beams: largest logit and its score.  Where that logit is +inf, the probability lies on those alone.
#pragma unroll 1
  for (int k = warp; k < p.K; k += kWarps) {
    const long long row = (long long)b * p.K + k;
    const float2* st = p.stats + row * p.S;
    const float from = ld(p.scores + row);
    const float2 first = lane < p.S ? __ldcg(st + lane) : make_float2(-INFINITY, 0.f);
    float top = first.x, sum = first.y;  // of the lane's chunks, then of all
#pragma unroll 1
    for (int s = lane + 32; s < p.S; s += 32) {
      const float2 x = __ldcg(st + s);
      if (x.x > -INFINITY) {
        const float m = fmaxf(top, x.x);
        sum = (top == m ? sum : sum * exp2f((top - m) * kLog2e)) + (x.x == m ? x.y : x.y * exp2f((x.x - m) * kLog2e));
        top = m;
      }
    }
    const float most = value32(__reduce_max_sync(0xffffffffu, order32(top)));
    sum = top == most ? sum : sum * exp2f((top - most) * kLog2e);
    if (p.S > 1) sum = warp_sum(sum);
    if (lane == 0) {
      sh.top[k] = most;
      sh.base[k] = sum > 0.f && from > -INFINITY ? add({from, 0.f}, minus_log(sum)) : Pair{-INFINITY, 0.f};
    }
  }
  if (tid == 0) sh.n = 0;
  __syncthreads();
  // ---- candidates: a score that at least M reach, and those that reach it
  // (a thread keeps its two best; only where both are among them does it look through its others once more)
  unsigned long long key[2] = {0, 0}, at[2] = {0, 0};
  auto keep = [&](uint2 e, int i) {
    unsigned long long k, a;
    if (!candidate(sh, e, i / per, k, a) || k <= key[1]) return;
    if (k > key[0]) key[1] = key[0], at[1] = at[0], key[0] = k, at[0] = a;
    else key[1] = k, at[1] = a;
  };
  keep(e0, min(i0, n_all - 1));
#pragma unroll 2
  for (int i = i0 + kThreads; i < n_all; i += kThreads) keep(__ldcg(best + i), i);
  uint32_t largest;
  const uint32_t wth = wth_largest((uint32_t)(key[0] >> 32), (p.M + kWarps - 1) / kWarps, largest);
  if (lane == 0) sh.w_th[warp] = wth;
  __syncthreads();
  const uint32_t bound = sh.bound();
  unsigned long long* place = sh.at();
  auto take = [&](unsigned long long key, unsigned long long at) {
    const int j = atomicAdd(&sh.n, 1);
    if (j < kList) sh.key[j] = key, place[j] = at, sh.rank[j] = 0;
  };
  if (key[1] > 0 && (uint32_t)(key[1] >> 32) >= bound) {
#pragma unroll 1
    for (int i = i0; i < n_all; i += kThreads) {
      unsigned long long k, a;
      if (candidate(sh, __ldcg(best + i), i / per, k, a) && (uint32_t)(k >> 32) >= bound) take(k, a);
    }
  } else if (key[0] > 0 && (uint32_t)(key[0] >> 32) >= bound) {
    take(key[0], at[0]);
  }
  __syncthreads();
  int n = sh.n;
  if (n >= p.M && n <= kDirect) {
    // a thread an entry: how many come before it, and how many of those go on
    if (tid < n) {
      const unsigned long long key = sh.key[tid], at = place[tid];
      int rank = 0, on = 0;
#pragma unroll 4
      for (int j = 0; j < n; ++j) {
        const unsigned long long a = place[j], k = sh.key[j];
        const bool before = k > key || (k == key && a < at);
        rank += before;
        on += before && (int)(uint32_t)a != p.eos;
      }
      const int beam = (int)(at >> 32), token = (int)(uint32_t)at;
      const float score = value32((uint32_t)(key >> 32));
      if (rank < p.M) {
        const long long o = (long long)b * p.M + rank;
        p.cand_score[o] = score, p.cand_beam[o] = beam, p.cand_token[o] = token;
        if (token != p.eos && on < p.K) {
          const long long to = (long long)b * p.K + on;
          p.next_score[to] = score, p.next_beam[to] = beam, p.next_token[to] = token;
        }
      }
    }
    return;
  }
  if (n > kList) {
    slow_finish(best, n_all, per, n = p.M, sh);
  } else {
    count_before<true>(sh, n);
#pragma unroll 1
    for (int i = tid; i < n; i += kThreads)
      if (sh.rank[i] < p.M) sh.top_key[sh.rank[i]] = sh.key[i], sh.top_at[sh.rank[i]] = place[i];
    n = min(n, p.M);
  }
  __syncthreads();
  if (n < p.M) {
    fill_up(n, p.M, p.V, sh);
    __syncthreads();
  }
  // ---- all M, and the first K that go on
  if (warp == 0) {
    int on = 0;
#pragma unroll 1
    for (int r0 = 0; r0 < p.M; r0 += 32) {
      const int r = r0 + lane;
      const bool real = r < p.M;
      const unsigned long long at = real ? sh.top_at[r] : 0ull;
      const int beam = (int)(at >> 32), token = (int)(uint32_t)at;
      const float score = real ? value32((uint32_t)(sh.top_key[r] >> 32)) : 0.f;
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

// A CTA's chunk of a row: the row's whole vectors [va, vb), and the elements before its first or behind its last one.
template <typename T>
struct Chunk {
  const T *x, *vecs;  // the row, its first whole vector
  int va, vb, V;
  bool head, tail;
  CP_DEV int first(int v) const { return (int)(vecs - x) + v * Vec<T>::N; }  // element of a vector's first place
  CP_DEV void load(Vec<T>& r, int v) const {
    if (v < vb) r.load(vecs + (long long)v * Vec<T>::N);
    else r.clear();
  }
  // vectors va - 1 and vb: what the row has of them, if they are this chunk's
  CP_DEV bool has_end(int v) const { return v < va ? head : tail; }
  CP_DEV void load_end(Vec<T>& r, int v) const {
    r.clear();
    const int e = first(v);
    if (has_end(v))
#pragma unroll
      for (int j = 0; j < Vec<T>::N; ++j)
        if (e + j >= 0 && e + j < V) r.put(j, x[e + j]);
  }
  // any of the chunk's vectors in turn, for the slow ways: i = 0, 1 are its ends
  CP_DEV int count() const { return vb - va + 2; }
  CP_DEV int get(Vec<T>& r, int i) const {
    const int v = i == 0 ? va - 1 : i == 1 ? vb : va + i - 2;
    if (i < 2) load_end(r, v);
    else load(r, v);
    return first(v);
  }
};
CP_DEV unsigned long long list_key(float y, int token) {
  return ((unsigned long long)order32(y) << 32) | (0xffffffffu - (uint32_t)token);
}

// Sum of exp(x - most) where a NaN counts as -inf, and infinities share the probability.
template <typename T>
__device__ __noinline__ float slow_sum(const Chunk<T> c, float most) {
  float sum = 0.f;
#pragma unroll 1
  for (int i = threadIdx.x; i < c.count(); i += kThreads) {
    Vec<T> r;
    c.get(r, i);
#pragma unroll
    for (int j = 0; j < Vec<T>::N; ++j) {
      const float y = r.get(j);
      sum += y == most ? 1.f : y < most ? ex2_approx((y - most) * kLog2e) : 0.f;
    }
  }
  return sum;
}
// The chunk's values that reach `least`, or where they are too many its M largest one after the other (into key[0 .. M)).
template <typename T>
__device__ __noinline__ int slow_list(const Chunk<T> c, float least, int M, SelectShared& sh) {
  __syncthreads();
  if (threadIdx.x == 0) sh.n = 0;
  __syncthreads();
#pragma unroll 1
  for (int i = threadIdx.x; i < c.count(); i += kThreads) {
    Vec<T> r;
    const int e = c.get(r, i);
#pragma unroll
    for (int j = 0; j < Vec<T>::N; ++j) {
      const float y = r.get(j);
      if (y >= least) {
        const int at = atomicAdd(&sh.n, 1);
        if (at < kList) sh.key[at] = list_key(y, e + j), sh.rank[at] = 0;
      }
    }
  }
  __syncthreads();
  const int n = sh.n;
  if (n <= kList) return n;
  unsigned long long last = ~0ull;
  for (int m = 0; m < M; ++m) {
    unsigned long long best = 0, none = 0;
#pragma unroll 1
    for (int i = threadIdx.x; i < c.count(); i += kThreads) {
      Vec<T> r;
      const int e = c.get(r, i);
#pragma unroll
      for (int j = 0; j < Vec<T>::N; ++j) {
        const float y = r.get(j);
        if (y >= least) {
          const unsigned long long k = list_key(y, e + j);
          if (k < last && k > best) best = k;
        }
      }
    }
    block_best(best, none, sh.w_key, sh.w_at);
    if (threadIdx.x == 0) sh.key[m] = best, sh.rank[m] = 0;
    last = best;
  }
  __syncthreads();
  return M;
}

// NV: vectors a thread takes at a time.
template <typename T, int NV>
__global__ void __launch_bounds__(kThreads, 4) select_kernel(const SelectParams p) {
  using W = Vec<T>;
  __shared__ SelectShared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long row = blockIdx.x / (unsigned)p.S;
  const int part = (int)(blockIdx.x % (unsigned)p.S), b = (int)(row / p.K);
  Chunk<T> c;
  c.x = static_cast<const T*>(p.logits) + row * p.stride;
  const int before = (int)((0u - (uint32_t)reinterpret_cast<uintptr_t>(c.x)) & 15u) / (int)sizeof(T);
  const int vecs = max(0, p.V - before) / W::N;  // whole ones
  c.vecs = c.x + before;
  c.V = p.V;
  c.va = min(part * p.chunk, vecs);
  c.vb = min(c.va + p.chunk, vecs);
  c.head = part == 0 && before > 0;
  c.tail = part == p.S - 1 && before + vecs * W::N < p.V;
  // warps whose lanes all have a vector in the first round, and how many of each one's values the bound counts
  const int full_warps = min(kWarps, (c.vb - c.va) / 32), w = (p.M + max(full_warps, 1) - 1) / max(full_warps, 1);
  if (tid == 0) sh.n = sh.n2 = 0;
  if (lane == 0) sh.w_th[warp] = warp < full_warps ? order32(-INFINITY) : 0xffffffffu;

  // this lane's largest value, and what its sum is relative to (values far below any that counts, a mask's lowest ones,
  // do not move it)
  float top = -INFINITY, ref = -kMaxLogit;
  // pairs of sums of 2^(x log2(e) - c), c = ref log2(e) rounded.  They move by differences of the c's as they were rounded
  // (up to 2^-7, for logits near 1e5), not of the references
  uint64_t part_sum[2] = {0ull, 0ull}, minus_c, log2e;
  asm("mov.b64 %0, {%1, %1};" : "=l"(log2e) : "f"(kLog2e));
  asm("mov.b64 %0, {%1, %1};" : "=l"(minus_c) : "f"(kMaxLogit * kLog2e));
  volatile uint32_t* th = sh.w_th;
  // the w-th largest of the warp's lanes' largest values, published; and the bound as it stands
  auto publish = [&]() {
    uint32_t largest;
    const uint32_t k = wth_largest(order32(top), w, largest);
    if (lane == 0 && warp < full_warps) th[warp] = k;
  };
  const bool counted = full_warps > 0 && w <= 32;
  auto bound = [&]() -> float { return counted ? fmaxf(value32(sh.bound()), -kMost) : -kMost; };  // (-inf reaches none)
  // one round of vectors: sum, largest value, and the list
  auto work = [&](auto& v, int v0, bool first_round) {
    constexpr int kN = sizeof(v) / sizeof(W);
    float vm[kN], mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      vm[i] = v[i].max();
      mx = fmaxf(mx, vm[i]);
    }
    top = fmaxf(top, mx);
    if (top > ref + kMaxGrowth) {  // (the first time, and rarely again)
      const float now = __fmul_rn(-top, kLog2e), f = ex2_approx(__fsub_rn(now, low(minus_c)));
      uint64_t f2;
      asm("mov.b64 %0, {%1, %1};" : "=l"(f2) : "f"(f));
#pragma unroll
      for (int i = 0; i < 2; ++i) asm("mul.f32x2 %0, %0, %1;" : "+l"(part_sum[i]) : "l"(f2));
      ref = top;
      asm("mov.b64 %0, {%1, %1};" : "=l"(minus_c) : "f"(now));
    }
#pragma unroll
    for (int i = 0; i < kN; ++i)
#pragma unroll
      for (int j = 0; j < W::N; j += 2) add_exp2(part_sum[(j >> 1) & 1], v[i].get(j), v[i].get(j + 1), log2e, minus_c);
    if (first_round) {
      publish();
      __syncthreads();
    }
    const float least = bound();
    if (mx >= least) {
#pragma unroll
      for (int i = 0; i < kN; ++i)
        if (vm[i] >= least) {
          const int at = atomicAdd(&sh.n, 1);
          if (at < kVecs) sh.vec[at] = v[i].raw(), sh.id[at] = v0 + i * kThreads;
        }
    }
  };
  constexpr int kRound = NV * kThreads;
  W va[NV], vb[NV];
  int v0 = c.va + tid;
  chained_start();  // (nothing of the call's memory has been touched)
  auto load = [&](W (&v)[NV], int from) {
#pragma unroll
    for (int i = 0; i < NV; ++i) c.load(v[i], from + i * kThreads);
  };
  load(va, v0);
  const int rounds = max(1, (c.vb - c.va + kRound - 1) / kRound);
#pragma unroll 1
  for (int r = 0; r < rounds; r += 2, v0 += 2 * kRound) {
    if (r + 1 < rounds) load(vb, v0 + kRound);
    work(va, v0, r == 0);
    if (r + 1 >= rounds) break;
    if (r + 2 < rounds) load(va, v0 + 2 * kRound);
    work(vb, v0 + kRound, false);
    if (((r + 2) & (r + 1)) == 0) publish();  // after 2, 4, 8, .. rounds
  }
  if (warp == 0 && (c.head || c.tail)) {  // the row's ends: lane 0 and lane 1
    W end[1];
    const int v = lane == 0 ? c.va - 1 : c.vb;
    if (lane < 2) c.load_end(end[0], v);
    else end[0].clear();
    work(end, v, false);
  }
  publish();
  const uint32_t warp_top = __reduce_max_sync(0xffffffffu, order32(top));
  if (lane == 0) sh.w_max[warp] = warp_top;
  __syncthreads();

  // ---- the chunk's sum
  uint32_t k_most = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) k_most = max(k_most, sh.w_max[i]);
  const float most = value32(k_most), least = bound();
  float sum;
  {
    float s[4];
    asm("mov.b64 {%0, %1}, %2;" : "=f"(s[0]), "=f"(s[1]) : "l"(part_sum[0]));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(s[2]), "=f"(s[3]) : "l"(part_sum[1]));
    sum = (s[0] + s[1]) + (s[2] + s[3]);
    sum *= ex2_approx(fmaf(-most, kLog2e, -low(minus_c)));
  }
  sum = block_sum(sum, sh.w_sum);
  if (!(sum < INFINITY) || fabsf(most) > kMaxLogit) {
    __syncthreads();
    sum = most > -INFINITY ? slow_sum(c, most) : 0.f;
    sum = block_sum(sum, sh.w_sum);
  }

  // ---- its M largest values, in order
  const long long out = row * p.S + part;
  uint2* best = p.best + out * p.M;
  int n = sh.n;
  if (n > kVecs) {
    n = slow_list(c, least, p.M, sh);
  } else {
#pragma unroll 1
    for (int i = tid; i < n * W::N; i += kThreads) {  // a thread an element
      const float y = to_float(reinterpret_cast<const T*>(sh.vec)[i]);
      if (y >= least) {
        const int at = atomicAdd(&sh.n2, 1);
        if (at < kList) sh.key[at] = list_key(y, c.first(sh.id[i / W::N]) + i % W::N), sh.rank[at] = 0;
      }
    }
    __syncthreads();
    n = sh.n2;
    if (n > kList) n = slow_list(c, least, p.M, sh);
  }
  auto put = [&](int rank, unsigned long long key) {
    if (rank < p.M) best[rank] = make_uint2(__float_as_uint(value32((uint32_t)(key >> 32))), 0xffffffffu - (uint32_t)key);
  };
  if (n <= kDirect) {
    if (tid < n) {
      const unsigned long long key = sh.key[tid];
      int rank = 0;
#pragma unroll 8
      for (int j = 0; j < n; ++j) rank += sh.key[j] > key;
      put(rank, key);
    }
  } else {
    count_before<false>(sh, n);
#pragma unroll 1
    for (int i = tid; i < n; i += kThreads) put(sh.rank[i], sh.key[i]);
  }
  for (int r = n + tid; r < p.M; r += kThreads) best[r] = make_uint2(0xff800000u, 0xffffffffu);
  if (tid == 0) p.stats[out] = make_float2(most, sum);

  // ---- the CTA that counts last has every chunk of the sequence before it
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

// Chunks: one a row if that gives every SM its four CTAs or nearly; else as many as do, of 16 KB at least (shorter ones
// cost the last CTA more than they save), and where beams and candidates are many no more than give it 1024 values to
// look through.  More rows than places: a third of the GPU's places each, so that the last ones are short.  152 SMs are
// GB300's: the workspace's size follows from the cut and does not ask the device.
struct SelectPlan {
  int NV, S, chunk;
};
SelectPlan select_plan(long long rows, int K, int M, int V, int elem) {
  constexpr long long kPlaces = 4 * 152;
  // whole 16-byte vectors of a row, which may start anywhere in one (at most; its ends are apart); a vector a thread
  const long long vecs = (long long)V * elem / 16, pieces = vecs > 0 ? (vecs + kThreads - 1) / kThreads : 1;
  long long S = rows > kPlaces ? (3 * kPlaces + rows - 1) / rows : kPlaces / rows;
  const long long most = rows > kPlaces ? (pieces + 7) / 8 : (pieces + 3) / 4, lists = 1024 / ((long long)K * M);
  if (S > most) S = most;
  if (S > 2 && S > lists) S = lists > 2 ? lists : 2;
  if (S < 1) S = 1;
  const long long per = (pieces + S - 1) / S;
  return {per >= 4 ? 4 : per >= 2 ? 2 : 1, (int)((pieces + per - 1) / per), (int)(per * kThreads)};
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
  const SelectPlan plan = select_plan((long long)a.num_seqs * a.num_beams, a.num_beams, a.num_candidates, a.vocab, sizeof(T));
  size_t o_stats, o_best;
  select_layout((size_t)a.num_seqs * a.num_beams * plan.S, a.num_candidates, &o_stats, &o_best);
  SelectParams p;
  p.K = a.num_beams;
  p.V = a.vocab;
  p.M = a.num_candidates;
  p.S = plan.S;
  p.chunk = plan.chunk;
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
  auto kern = plan.NV == 4 ? select_kernel<T, 4> : plan.NV == 2 ? select_kernel<T, 2> : select_kernel<T, 1>;
  return launch_chained(kern, grid, kThreads, 0, s, p);
}

// ================================================================================ reordering
// Beam j of a sequence goes on from parent p_j.  Of its L cached tokens rank r holds L_r: columns before
// L_r / 16 are full pages, shared by table; the page being filled belongs to one beam, so its L_r mod 16 rows are
// copied from the parent's to beam j's own.
//
// A beam's own page may be another's source, so nothing is written before all that it replaces has been read: a
// thread owns one 16-byte place of the page (row, vector), loads it from the K parents' pages and stores it to the
// K beams' pages, K loads in flight at once, then takes the next place.  The tables go the same way, a
// thread a column.  Tables that are replaced in place wait for the pages' copies in a launch of their own.
// Bound: the launch and one chain of dependent loads (length, table entry, rows: 2300 cycles to the first row, then about 2000
// a place).  64 x 8 beams of 64 .. 2048 tokens, 8 heads of 128, two ranks, bf16: 9.5 us (54% of the copy); 24 layers of 6 x 5
// beams: 12.2; one sequence 2.8.  Not kept: two places at a time (14.8 us for the layers), a loop without its divisions (14.6: the
// loads then meet in the same banks of memory more often), blocks of 64 threads, more or fewer CTAs an SM.
struct ReorderParams {
  int B, K, cp, I, max_blocks, Hkv, layers2, ctas;    // layers2: pools of K and of V; ctas: of a (sequence, rank)'s pages
  int row_vecs, head_vecs, tail_at, tail_words;       // 16-byte vectors of a row and of a head's page; 4-bit records: place and words a row of the scales
  long long pool, layer_vecs;
  const int32_t *parents, *seq_lens, *tables_in, *own;
  int32_t* tables_out;  // null: pages only
  uint4 *k, *v;         // null: tables only
  int32_t* err;
};

// 1-D grid: (sequence, rank) slowest; within it the tables' CTA, then those that share the places of all pools.  As many as
// the GPU takes at once: before its first place each goes through a chain of dependent loads (length, parents, tables).
constexpr int kReorderThreads = 128;
constexpr int reorder_ctas(int kmax) { return kmax <= 4 ? 8 : kmax <= 8 ? 5 : kmax <= 16 ? 3 : 2; }  // on an SM
template <int KMAX>
__global__ void __launch_bounds__(kReorderThreads, reorder_ctas(KMAX)) reorder_kernel(const ReorderParams p) {
  __shared__ int s_parent[KMAX], s_own[KMAX];        // -1: none
  __shared__ long long s_src[KMAX], s_dst[KMAX];     // 16-byte vectors from the pool's start; -1: nothing to copy
  const int tables = p.tables_out != nullptr ? 1 : 0;
  const unsigned per = (unsigned)(tables + (p.k != nullptr ? p.ctas : 0));
  const unsigned unit = blockIdx.x / per, job = blockIdx.x % per;
  const int b = (int)(unit / (unsigned)p.cp), r = (int)(unit % (unsigned)p.cp);
  chained_start();
  const int L = ld(p.seq_lens + b);
  int parent = threadIdx.x < p.K ? ld(p.parents + (long long)b * p.K + threadIdx.x) : -1;
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
  const int cta = (int)job - tables, places = p.Hkv * fill * p.row_vecs;  // of a pool
  if (!first && (long long)cta * kReorderThreads >= (long long)places * p.layers2) return;  // (few tokens in the page)
  if (threadIdx.x < p.K) {
    const int j = threadIdx.x;
    if (parent < 0 || parent >= p.K) {
      if (first) report(p.err, CP_ERR_DEVICE_BOUNDS);
      parent = -1;
    }
    int src = -1, dst = -1;
    if (parent >= 0 && col < p.max_blocks) {
      dst = ld(p.own + (row0 + j) * p.max_blocks + col);
      if (fill > 0) src = ld(p.tables_in + (row0 + parent) * p.max_blocks + col);
      if (dst < 0 || dst >= p.pool) {
        if (first) report(p.err, CP_ERR_DEVICE_BOUNDS);
        dst = -1;
      } else if (fill > 0 && (src < 0 || src >= p.pool)) {
        if (first) report(p.err, CP_ERR_DEVICE_BOUNDS);
        src = -1;
      }
    }
    const long long page = (long long)p.Hkv * p.head_vecs;
    const bool moves = src >= 0 && dst >= 0 && src != dst;
    s_parent[j] = parent;
    s_own[j] = dst;
    s_src[j] = moves ? src * page : -1;
    s_dst[j] = dst * page;
  }
  __syncthreads();

  if (tables && job == 0) {
    for (int c = threadIdx.x; c <= col && c < p.max_blocks; c += kReorderThreads) {
      int32_t id[KMAX];
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if (j < p.K && s_parent[j] >= 0)
          id[j] = c == col && s_own[j] >= 0 ? s_own[j] : ld(p.tables_in + (row0 + s_parent[j]) * p.max_blocks + c);
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if (j < p.K && s_parent[j] >= 0) p.tables_out[(row0 + j) * p.max_blocks + c] = id[j];
    }
    return;
  }
  // head h of page 0 of pool i
  auto head = [&](int i, int h) -> uint4* {
    return ((i & 1) ? p.v : p.k) + (i >> 1) * p.layer_vecs + ((long long)r * p.pool * p.Hkv + h) * p.head_vecs;
  };
  // what place j of the K pages is replaced by, all of it read first
  auto move = [&](auto* place, int scale) {
    std::remove_reference_t<decltype(*place)> x[KMAX];
#pragma unroll
    for (int j = 0; j < KMAX; ++j)
      if (j < p.K && s_src[j] >= 0) x[j] = place[s_src[j] * scale];
#pragma unroll
    for (int j = 0; j < KMAX; ++j)
      if (j < p.K && s_src[j] >= 0) place[s_dst[j] * scale] = x[j];
  };
#pragma unroll 1
  for (long long at = (long long)cta * kReorderThreads + threadIdx.x; at < (long long)places * p.layers2; at += p.ctas * kReorderThreads) {
    const int pool = (int)(at / places), i = (int)(at - (long long)pool * places), q = i / p.row_vecs, h = q / fill;
    move(head(pool, h) + (q - h * fill) * p.row_vecs + (i - q * p.row_vecs), 1);
  }
  if (p.tail_words > 0) {  // 4-bit records: the rows' scales and minima
    const int words = p.Hkv * fill * p.tail_words;
#pragma unroll 1
    for (long long at = (long long)cta * kReorderThreads + threadIdx.x; at < (long long)words * p.layers2; at += p.ctas * kReorderThreads) {
      const int pool = (int)(at / words), i = (int)(at - (long long)pool * words), h = i / (fill * p.tail_words);
      move(reinterpret_cast<uint32_t*>(head(pool, h) + p.tail_at) + (i - h * fill * p.tail_words), 4);
    }
  }
}

cudaError_t reorder_launch(ReorderParams p, cudaStream_t s) {
  const int kmax = p.K <= 4 ? 4 : p.K <= 8 ? 8 : p.K <= 16 ? 16 : 32;
  const long long units = (long long)p.B * p.cp, slots = 152ll * reorder_ctas(kmax);  // (GB300's SMs; any number is right)
  const long long most = ((long long)p.Hkv * 15 * p.row_vecs * p.layers2 + kReorderThreads - 1) / kReorderThreads;
  const long long ctas = (slots + units - 1) / units;
  p.ctas = (int)(ctas < most ? ctas : most);
  const long long grid = units * ((p.tables_out != nullptr ? 1 : 0) + (p.k != nullptr ? p.ctas : 0));
  if (grid == 0) return cudaSuccess;
  if (grid >= (1ll << 31)) return cudaErrorInvalidConfiguration;
  auto kern = kmax == 4 ? reorder_kernel<4> : kmax == 8 ? reorder_kernel<8> : kmax == 16 ? reorder_kernel<16> : reorder_kernel<32>;
  return launch_chained(kern, dim3((unsigned)grid), kReorderThreads, 0, s, p);
}

}  // namespace
}  // namespace cpattn

// Enough for either type and for every smaller size: up to 4 * 152 rows there are at most so many chunks, beyond three
// times as many and one a row.
size_t cp_beam_select_bytes(int32_t num_seqs, int32_t num_beams, int32_t vocab, int32_t num_candidates) {
  const size_t rows = (size_t)num_seqs * num_beams;
  size_t a, b;
  (void)vocab;
  return cpattn::select_layout(rows > 4 * 152 ? rows + 3 * 4 * 152 : 4 * 152, num_candidates, &a, &b);
}
long long cp_beam_select_ctas(const cp_beam_select_args& a) {
  const long long rows = (long long)a.num_seqs * a.num_beams;
  return rows * cpattn::select_plan(rows, a.num_beams, a.num_candidates, a.vocab, a.dtype == CP_BF16 ? 2 : 4).S;
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
