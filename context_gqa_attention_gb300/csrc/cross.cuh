// What the kernels of cp_cross_attention share (internal): the launch's parameters, a sequence's bounds, and the
// meeting of the parts of items whose keys were cut: in a cluster's shared memory, or in the workspace.
#pragma once

#include "common.cuh"
#include "sm100.cuh"

namespace cpattn {
namespace {

using namespace sm100;

constexpr long long kBudget = 4000000000ll;  // SM cycles per wait (~2 s)
constexpr int kMaxCluster = 8;

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
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(mine)), "r"(rank));
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

// An item is `span` tokens of a sequence under the G query heads of a kv head: span * G query rows, row p being
// token p / G, head p mod G, which all see the same keys (or, with key_ranges, some of them).  Items n_whole ..
// of a launch are cut into split_k parts each, whose normalised rows and LSEs wait in the workspace.
struct CrossParams {
  int B, Hq, Hkv, G, Nq, Nkv, max_q, span, tiles;  // tiles: items of the longest sequence
  int n_whole, n_split, split_k, rows;             // rows: of an item in the workspace
  int ordered;                                     // items in the order of their keys (see cross_item)
  int cluster;                                     // many rows: parts of every item that meet in a cluster (1: none)
  float scale_log2;
  long long q_stride, k_stride, v_stride;
  const int32_t *cu_q, *cu_kv, *kv_lens, *ranges;
  const void *q, *k, *v;
  void* out;
  float* lse;  // or null
  float *ws_out, *ws_lse;
  int32_t* err;
};

struct CrossItem {
  int b, g, t0, tokens;  // the sequence, the kv head, its first token and how many there are (0: nothing to do)
  int q0, kv0, keys;     // first rows in q and k, v; keys of the sequence
};
// A sequence's rows and keys, as the tensors allow.
CP_DEV CrossItem cross_sequence(const CrossParams& p, int b, int& rows, bool& report_it) {
  CrossItem w;
  w.b = b;
  w.q0 = ld(p.cu_q + b);
  w.kv0 = ld(p.cu_kv + b);
  const int q1 = ld(p.cu_q + b + 1), kv1 = ld(p.cu_kv + b + 1), n = p.kv_lens != nullptr ? ld(p.kv_lens + b) : 0;
  const long long Tq = (long long)q1 - w.q0, Tkv = (long long)kv1 - w.kv0;
  w.keys = (int)Tkv;
  report_it = Tq > p.max_q;
  if (p.kv_lens != nullptr) {
    report_it = report_it || n < 0 || n > Tkv;
    w.keys = (int)max(0ll, min((long long)n, Tkv));
  }
  const bool bad = Tq < 0 || Tkv < 0 || w.q0 < 0 || w.kv0 < 0 || w.q0 + Tq > p.Nq || w.kv0 + Tkv > p.Nkv;
  report_it = report_it || bad;
  rows = bad ? 0 : (int)min(Tq, (long long)p.max_q);
  return w;
}
// The item of an index, once the last call is done with the memory (chained_start); every lane of a warp asks for the
// same.  reporter: one thread of the item's first CTA, which says
// what is wrong with the sequence.
//
// ordered (up to 32 sequences of different lengths, one a lane): the sequences with the most keys first, so that the last
// items are short, and indexes without rows behind all others.
CP_DEV CrossItem cross_item(const CrossParams& p, unsigned index, bool reporter) {
  CrossItem w;
  int rows;
  bool wrong;
  if (p.ordered) {
    chained_start();
    const int lane = (int)(threadIdx.x & 31), mine = min(lane, p.B - 1);
    w = cross_sequence(p, mine, rows, wrong);
    if (reporter && index == 0) {  // (thread 0 sees one sequence: it looks through the others)
      for (int b = 0; b < p.B; ++b) {
        int r;
        bool x;
        cross_sequence(p, b, r, x);
        if (x) report(p.err, CP_ERR_DEVICE_BOUNDS);
      }
    }
    __syncwarp();
    const int n = lane < p.B ? (rows + p.span - 1) / p.span : 0;
    int start = 0;  // items of the sequences before this one
    for (int j = 0; j < p.B; ++j) {
      const int k = __shfl_sync(0xffffffffu, w.keys, j), m = __shfl_sync(0xffffffffu, n, j);
      if (k > w.keys || (k == w.keys && j < lane)) start += m;
    }
    const unsigned u = index / (unsigned)p.Hkv;
    const uint32_t found = __ballot_sync(0xffffffffu, u >= (unsigned)start && u < (unsigned)(start + n));
    const int at = found != 0u ? __ffs(found) - 1 : 0;
    w.b = __shfl_sync(0xffffffffu, w.b, at);
    w.q0 = __shfl_sync(0xffffffffu, w.q0, at);
    w.kv0 = __shfl_sync(0xffffffffu, w.kv0, at);
    w.keys = __shfl_sync(0xffffffffu, w.keys, at);
    rows = __shfl_sync(0xffffffffu, rows, at);
    w.g = (int)(index % (unsigned)p.Hkv);
    w.t0 = (int)(u - (unsigned)__shfl_sync(0xffffffffu, start, at)) * p.span;
    w.tokens = found != 0u ? min(p.span, rows - w.t0) : 0;
    return w;
  }
  const unsigned tile = index % (unsigned)p.tiles, u = index / (unsigned)p.tiles;
  const int b = (int)(u / (unsigned)p.Hkv), g = (int)(u % (unsigned)p.Hkv), t0 = (int)tile * p.span;
  chained_start();
  w = cross_sequence(p, b, rows, wrong);
  w.g = g;
  w.t0 = t0;
  if (reporter && wrong && tile == 0 && w.g == 0) report(p.err, CP_ERR_DEVICE_BOUNDS);
  w.tokens = max(0, min(p.span, rows - w.t0));
  return w;
}
// The keys [lo, hi) of a token (within the sequence).
CP_DEV void cross_range(const CrossParams& p, const CrossItem& w, int token, int& lo, int& hi) {
  lo = 0, hi = w.keys;
  if (p.ranges != nullptr) {
    const int32_t* r = p.ranges + 2ll * (w.q0 + token);
    lo = max(0, ld(r));
    hi = min(w.keys, ld(r + 1));
    if (lo >= hi) lo = hi = 0;
  }
}

// Two sets of (reference in log2 units, sum, row) as one: the factor of a set whose reference is m.  (One of -inf saw
// no finite score: its sums are 0, or NaN.)
CP_DEV float factor(float m, float M) { return m == M || m == -INFINITY ? 1.f : exp2f(m - M); }
CP_DEV float natural_lse(float M, float L) {
  return L == 0.f ? -INFINITY : ((M == -INFINITY ? 0.f : M) + log2f(L)) * kLn2;
}

// Parts -> rows: out = sum_k e_k out_k / sum_k e_k with e_k = exp(lse_k - max lse); a part without a key has the
// LSE -inf and its row is not read, another one's is, even for a weight that underflows: 0 times what is not finite is NaN.
// A warp takes a row, its lanes the dims.
template <typename T, int D>
__global__ void __launch_bounds__(256) cross_merge_kernel(const CrossParams p) {
  constexpr int E = D / 32;
  const CrossItem w = cross_item(p, (unsigned)p.n_whole + blockIdx.x, false);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long part0 = (long long)blockIdx.x * p.split_k;
  for (int row = (int)blockIdx.y * 8 + warp; row < w.tokens * p.G; row += (int)gridDim.y * 8) {
    float M = -INFINITY;
    float x[4];  // LSEs in log2 units, 32 parts at a time across the lanes
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = lane + 32 * i;
      x[i] = k < p.split_k ? p.ws_lse[(part0 + k) * p.rows + row] * kLog2e : -INFINITY;
      M = fmaxf(M, x[i]);
    }
    M = warp_max(M);
    float sum = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (32 * i >= p.split_k) break;
      const float mine = x[i] == -INFINITY ? -1.f : exp2f(x[i] - (M == -INFINITY ? 0.f : M));  // (NaN stays; -1: no key)
      const int n = min(32, p.split_k - 32 * i);
#pragma unroll 4
      for (int j = 0; j < n; ++j) {
        const float e = __shfl_sync(0xffffffffu, mine, j);
        if (e < 0.f) continue;
        const float* src = p.ws_out + ((part0 + 32 * i + j) * p.rows + row) * D + lane * E;
        sum += e;
        if constexpr (E == 4) {
          const float4 v = *reinterpret_cast<const float4*>(src);
          acc[0] += e * v.x, acc[1] += e * v.y, acc[2] += e * v.z, acc[3] += e * v.w;
        } else {
          const float2 v = *reinterpret_cast<const float2*>(src);
          acc[0] += e * v.x, acc[1] += e * v.y;
        }
      }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const long long o = ((long long)w.q0 + w.t0 + row / p.G) * p.Hq + w.g * p.G + row % p.G;
    T* dst = static_cast<T*>(p.out) + o * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if constexpr (sizeof(T) == 2) dst[e] = __float2bfloat16_rn(acc[e] * inv);
      else dst[e] = acc[e] * inv;
    }
    if (lane == 0 && p.lse != nullptr)
      p.lse[o] = sum == 0.f ? -INFINITY : ((M == -INFINITY ? 0.f : M) + log2f(sum)) * kLn2;
  }
}
constexpr int kMaxParts = 128;

template <typename T, int D>
cudaError_t launch_merge(const CrossParams& p, cudaStream_t s) {
  // eight rows a CTA until there are plenty
  int y = (p.rows + 7) / 8;
  while (y > 1 && (long long)p.n_split * y > 2048) y = (y + 1) / 2;
  return launch_chained(cross_merge_kernel<T, D>, dim3((unsigned)p.n_split, (unsigned)y), 256, 0, s, p);
}

// Grid: items, each one's parts side by side (a cluster's are neighbours).
template <typename... K, typename... A>
cudaError_t launch_parts(void (*kern)(K...), long long items, int parts, int cluster, int threads, size_t smem,
                         cudaStream_t s, A... args) {
  if (items * parts >= (1ll << 31)) return cudaErrorInvalidConfiguration;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items * parts));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cluster;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace
}  // namespace cpattn

// How a launch is made of items and parts (host).
struct CrossPlan {
  int span, tiles, rows, ordered, cluster;
  long long items, n_split;
  int split_k;
  size_t bytes;
};
// Items of up to 64 rows: f32 (cross_f32.cu), and bf16 of up to 64 rows a kv head (cross_few.cu).  The tensor cores' tiles of
// 128 rows take the rest (cross.cu).
inline bool cp_cross_few(const cp_cross_args& a) {
  return a.dtype == CP_F32 || (long long)a.max_seqlen_q * (a.num_q_heads / a.num_kv_heads) <= 64;
}
// Tokens of an item: 64 rows of the kernels for few rows (or what there is), two row tiles of the other.
inline int cp_cross_span(const cp_cross_args& a) {
  const int G = a.num_q_heads / a.num_kv_heads;
  if (!cp_cross_few(a)) return 2 * (128 / G);
  return a.max_seqlen_q <= 0 ? 1 : a.max_seqlen_q < 64 / G ? a.max_seqlen_q : 64 / G;
}
inline int cp_cross_tiles(const cp_cross_args& a) {
  const int span = cp_cross_span(a);
  return a.max_seqlen_q > 0 ? (int)(((long long)a.max_seqlen_q + span - 1) / span) : 1;
}
CrossPlan cp_cross_plan_tc(const cp_cross_args& a, int sms);
CrossPlan cp_cross_plan_few(const cp_cross_args& a, int sms);
cudaError_t cp_launch_cross_tc(const cp_cross_args& a, float scale, void* ws, size_t ws_bytes, void* out, float* lse,
                               cudaStream_t s);
cudaError_t cp_launch_cross_few(const cp_cross_args& a, float scale, void* ws, size_t ws_bytes, void* out, float* lse,
                                cudaStream_t s);
inline void cp_cross_fill(cpattn::CrossParams& p, const cp_cross_args& a, const CrossPlan& plan, float scale, void* ws,
                          size_t ws_bytes, void* out, float* lse) {
  p.B = a.num_seqs;
  p.Hq = a.num_q_heads;
  p.Hkv = a.num_kv_heads;
  p.G = a.num_q_heads / a.num_kv_heads;
  p.Nq = a.total_q;
  p.Nkv = a.total_kv;
  p.max_q = a.max_seqlen_q;
  p.span = plan.span;
  p.tiles = plan.tiles;
  p.rows = plan.rows;
  p.ordered = plan.ordered;
  p.cluster = plan.cluster;
  p.scale_log2 = scale * cpattn::kLog2e;
  p.q_stride = a.q_stride;
  p.k_stride = a.k_stride;
  p.v_stride = a.v_stride;
  p.cu_q = a.cu_seqlens_q;
  p.cu_kv = a.cu_seqlens_kv;
  p.kv_lens = a.kv_lens;
  p.ranges = a.key_ranges;
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  p.out = out;
  p.lse = lse;
  p.err = a.err;
  const bool cut = plan.split_k > 1 && ws != nullptr && ws_bytes >= plan.bytes;
  p.n_split = cut ? (int)plan.n_split : 0;
  p.n_whole = (int)(plan.items - p.n_split);
  p.split_k = cut ? plan.split_k : 1;
  p.ws_out = static_cast<float*>(ws);
  p.ws_lse = cut ? p.ws_out + (size_t)plan.n_split * plan.split_k * plan.rows * a.head_dim : nullptr;
}
inline size_t cp_cross_parts_bytes(const CrossPlan& plan, int D) {
  return plan.split_k > 1 ? (size_t)plan.n_split * plan.split_k * plan.rows * (D + 1) * sizeof(float) : 0;
}
