// Cross attention (cp_cross_attention) of few query rows: the beams of a source in a decode step, a short prompt;
// and of any number of rows in f32.  No counterpart on the pages, whose attention is causal self-attention.
//
//   out_i = softmax over the keys j in [lo_i, hi_i) of scale q_i.k_j, times V
//
// The rows of an item (CrossParams) are all that a kv head's states are read for, so the time is that of the states:
// bytes, not operations.  Parts of the keys run at once and meet in a cluster's shared memory (up to eight), or in
// the workspace (cross_merge_kernel) where a few long items have to fill the GPU.
#include <cuda.h>

#include "cross.cuh"
#include "sm100.cuh"

namespace cpattn {
namespace {

using namespace sm100;

constexpr long long kBudget = 4000000000ll;  // SM cycles per wait (~2 s)
constexpr float kMaxGrowth = 8.f;            // log2 units the scores may exceed the running reference
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
// Two sets of (reference in log2 units, sum, row) as one: the factor of a set whose reference is m.  (One of -inf saw
// no finite score: its sums are 0, or NaN.)
CP_DEV float factor(float m, float M) { return m == M || m == -INFINITY ? 1.f : exp2f(m - M); }
CP_DEV float natural_lse(float M, float L) {
  return L == 0.f ? -INFINITY : ((M == -INFINITY ? 0.f : M) + log2f(L)) * kLn2;
}

// What W slices of the CTA's keys made of R rows, in shared memory: reference, sum, unnormalised row.
template <int D, int W, int R>
struct Slices {
  float o[W][R][D + 8];  // (rows 32 bytes apart in the banks)
  float m[W][R], l[W][R];
};

// Slices -> the CTA's part; parts -> result, or to the workspace.  cluster: parts that meet in shared memory (1: none).
template <typename T, int D, int W, int R>
CP_DEV void finish(const CrossParams& p, const CrossItem& w, Slices<D, W, R>& s, int cluster, int piece) {
  constexpr int V = D / 4;
  const int rows = w.tokens * p.G;
  auto out_row = [&](int row) -> long long {
    return ((long long)w.q0 + w.t0 + row / p.G) * p.Hq + w.g * p.G + row % p.G;
  };
  __syncthreads();
  for (int i = threadIdx.x; i < rows * V; i += blockDim.x) {
    const int row = i / V, dd = (i % V) * 4;
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) M = fmaxf(M, s.m[k][row]);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const float e = factor(s.m[k][row], M);
      const float4 x = *reinterpret_cast<const float4*>(&s.o[k][row][dd]);
      L += e * s.l[k][row];
      o.x += e * x.x, o.y += e * x.y, o.z += e * x.z, o.w += e * x.w;
    }
    if (cluster > 1) {
      *reinterpret_cast<float4*>(&s.o[0][row][dd]) = o;  // (only this thread read these)
      continue;
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    o.x *= inv, o.y *= inv, o.z *= inv, o.w *= inv;
    if (piece >= 0) {
      const long long at = (long long)piece * p.rows + row;
      *reinterpret_cast<float4*>(p.ws_out + at * D + dd) = o;
      if (dd == 0) p.ws_lse[at] = natural_lse(M, L);
    } else {
      put4<T>(p.out, out_row(row) * D + dd, o);
      if (dd == 0 && p.lse != nullptr) p.lse[out_row(row)] = natural_lse(M, L);
    }
  }
  if (cluster <= 1) return;
  __syncthreads();  // (the slices' references have been read)
  for (int row = threadIdx.x; row < rows; row += blockDim.x) {
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) M = fmaxf(M, s.m[k][row]);
#pragma unroll
    for (int k = 0; k < W; ++k) L += factor(s.m[k][row], M) * s.l[k][row];
    s.m[0][row] = M;
    s.l[0][row] = L;
  }
  cluster_sync();
  const int rank = (int)cluster_rank();
  for (int i = rank + cluster * (int)threadIdx.x; i < rows * V; i += cluster * (int)blockDim.x) {
    const int row = i / V, dd = (i % V) * 4;
    float m[kMaxCluster], l[kMaxCluster], M = -INFINITY, L = 0.f;
    float4 x[kMaxCluster], o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c) {
      m[c] = -INFINITY, l[c] = 0.f;
      if (c < cluster) {
        m[c] = peer_ld(peer_addr(&s.m[0][row], c));
        l[c] = peer_ld(peer_addr(&s.l[0][row], c));
        x[c] = peer_ld4(peer_addr(&s.o[0][row][dd], c));
      }
    }
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c) M = fmaxf(M, m[c]);
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c)
      if (c < cluster) {
        const float e = factor(m[c], M);
        L += e * l[c];
        o.x += e * x[c].x, o.y += e * x[c].y, o.z += e * x[c].z, o.w += e * x[c].w;
      }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    o.x *= inv, o.y *= inv, o.z *= inv, o.w *= inv;
    put4<T>(p.out, out_row(row) * D + dd, o);
    if (dd == 0 && p.lse != nullptr) p.lse[out_row(row)] = natural_lse(M, L);
  }
  cluster_sync();  // no CTA leaves while another reads its shared memory
}

// The keys that some row of the item sees, the CTA's part of them [first, end) in whole tiles, and the keys that every
// row sees.
struct Keys {
  int first, end, all_lo, all_hi;
};
template <bool RANGES>
CP_DEV Keys part_keys(const CrossParams& p, const CrossItem& w, int tile, int part, int parts, int (&s_range)[4]) {
  Keys k;
  int lo = 0, hi = w.keys;
  k.all_lo = 0, k.all_hi = w.keys;
  if constexpr (RANGES) {
    if (threadIdx.x == 0) s_range[0] = s_range[3] = 0x7fffffff, s_range[1] = s_range[2] = 0;
    __syncthreads();
    for (int t = threadIdx.x; t < w.tokens; t += blockDim.x) {
      int a, b;
      cross_range(p, w, w.t0 + t, a, b);
      if (a < b) {
        atomicMin(s_range, a);
        atomicMax(s_range + 1, b);
      }
      atomicMax(s_range + 2, a);
      atomicMin(s_range + 3, b);
    }
    __syncthreads();
    lo = s_range[0], hi = s_range[1], k.all_lo = s_range[2], k.all_hi = s_range[3];
  }
  const int every = lo < hi ? (hi - lo + tile - 1) / tile : 0;
  const int a = (int)((long long)every * part / parts), b = (int)((long long)every * (part + 1) / parts);
  k.first = every > 0 ? lo + a * tile : 0;
  k.end = a < b ? min(hi, lo + b * tile) : k.first;
  return k;
}

// ------------------------------------------------------------------------------ the kernel
// MMAs of 16 rows on the legacy tensor path: a 128-row tcgen05 tile would be padding.  A producer warp brings tiles of
// K and V through a ring (TMA, 128-byte swizzle); consumer warp (m, k) owns the 16 rows m and the k-th slice of every
// tile's keys, with a softmax reference of its own, so warps meet at the end only.  The reference moves when a score
// exceeds it by more than 2^8, which a vote of the warp finds; rows' sums stay in the lanes until the end.
//
// f32: each operand is the sum of three bf16 numbers (high, middle, low: 24 bits) and a product the sum of the six of
// theirs that count, in fp32.  (Three products of tf32 pairs took three times as long: 25 cycles of a sub-partition each
// against 8.4 for twice the work.  CUDA cores need 32 times fewer rows' worth of padding, but a shared-memory read for
// every four of their products.)
CP_DEV void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
CP_DEV void ldsm4_t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
CP_DEV void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
CP_DEV uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Halves that are infinite or NaN become 0; whether there were any.
CP_DEV bool clean(uint32_t& w) {
  const uint32_t bad = ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;  // an exponent of all ones carries
  w &= ~((bad >> 15) * 0xffffu);
  return bad != 0u;
}
// x and y = high + middle + low, as pairs of bf16.
CP_DEV void split(float x, float y, uint32_t& h, uint32_t& m, uint32_t& l) {
  h = pack2(x, y);
  x -= __uint_as_float(h << 16), y -= __uint_as_float(h & 0xffff0000u);
  m = pack2(x, y);
  x -= __uint_as_float(m << 16), y -= __uint_as_float(m & 0xffff0000u);
  l = pack2(x, y);
}
CP_DEV float as_float(float x) { return x; }
CP_DEV float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// The six products that count, the small ones first.
CP_DEV void mma_parts(float (&c)[4], const uint32_t (&ah)[4], const uint32_t (&am)[4], const uint32_t (&al)[4],
                      const uint32_t (&h)[2], const uint32_t (&m)[2], const uint32_t (&l)[2]) {
  mma_bf16(c, al, h[0], h[1]);
  mma_bf16(c, ah, l[0], l[1]);
  mma_bf16(c, am, m[0], m[1]);
  mma_bf16(c, am, h[0], h[1]);
  mma_bf16(c, ah, m[0], m[1]);
  mma_bf16(c, ah, h[0], h[1]);
}

template <typename T, int D, int MT>
struct Few {
  static constexpr bool kF32 = sizeof(T) == 4;
  static constexpr int kWK = MT == 4 || (kF32 && D == 128) ? 2 : 4;  // slices of a tile's keys
  static constexpr int kConsumers = MT * kWK;
  static constexpr int kThreads = 32 * (kConsumers + 1);
  static constexpr int kBytes = 16384;               // of a tile of K or of V
  static constexpr int kTile = kBytes / (D * (int)sizeof(T));  // keys
  static constexpr int kKeys = kTile / kWK;          // of a warp
  static constexpr int kMaxStep = kF32 ? 16 : 32;
  static constexpr int kStep = kKeys < kMaxStep ? kKeys : kMaxStep;
  static_assert(kStep % 16 == 0, "steps of the second product");
  static constexpr int kBoxCols = 128 / (int)sizeof(T), kBoxes = D / kBoxCols;
  // q as A fragments in registers (bf16, one row group), or in shared memory: rows 16 bytes apart in the banks; f32: the
  // three parts one behind the other
  static constexpr bool kQRegs = !kF32 && MT == 1;
  static constexpr int kQPitch = D * 2 + 16, kQPart = 16 * MT * kQPitch;
  static constexpr int kQBytes = kQRegs ? 0 : kQPart * (kF32 ? 3 : 1);
  using Parts = Slices<D, kWK, 16 * MT>;
  static constexpr int align16(int x) { return (x + 15) / 16 * 16; }
  static constexpr int smem_of(int stages) {
    const int work = stages * 2 * kBytes + kQBytes, parts = align16((int)sizeof(Parts));
    return (work > parts ? work : parts) + 16 * stages + 1024;  // (the base is rounded up to the swizzle atom)
  }
  static constexpr int ctas_of(int stages) { return 232448 / (smem_of(stages) + 1024); }
  // CTAs on an SM, and stages of the ring (three CTAs of two stages: 106 us for 64 sequences of 512 .. 4096 states and 8 kv
  // heads, two of three stages 98.6)
  static constexpr int kCtas = ctas_of(2) >= 2 ? 2 : 1;
  static constexpr int kStages = ctas_of(4) >= kCtas ? 4 : ctas_of(3) >= kCtas ? 3 : 2;
  static constexpr int kRing = kStages * 2 * kBytes, oQ = kRing;
  static constexpr int oBar = smem_of(kStages) - 1024 - 16 * kStages;
  static constexpr int kSmem = smem_of(kStages);
};

template <typename T, int D, int MT, bool RANGES>
__global__ void __launch_bounds__(Few<T, D, MT>::kThreads, Few<T, D, MT>::kCtas)
    few_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const CrossParams p,
               const int parts, const int cluster) {
  using F = Few<T, D, MT>;
  constexpr int NT = F::kStep / 8;
  constexpr bool kRestore = RANGES || F::kF32;  // V may be cleaned
  extern __shared__ uint8_t smem_raw[];
  __shared__ int s_range[4];
  __shared__ uint32_t s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* sbase = smem_raw + (base - raw);
  auto full = [&](int s) -> uint32_t { return base + (uint32_t)F::oBar + 16u * (uint32_t)s; };
  auto empty = [&](int s) -> uint32_t { return full(s) + 8u; };
  volatile uint32_t* abort_flag = &s_abort;
  const bool producer = warp == F::kConsumers;
  if (producer && lane == 0) {
    for (int s = 0; s < F::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), F::kConsumers);
    }
    s_abort = 0u;
    fence_mbar_init();
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
  }
  chained_start();
  const int part = (int)(blockIdx.x % (unsigned)parts);
  const CrossItem w = cross_item(p, blockIdx.x / (unsigned)parts, threadIdx.x == 0 && part == 0);
  if (w.tokens == 0) return;  // (as every CTA of the cluster does)
  const int piece = p.n_split > 0 ? (int)blockIdx.x : -1;
  const Keys key = part_keys<RANGES>(p, w, F::kTile, part, parts, s_range);
  const int ntiles = (key.end - key.first + F::kTile - 1) / F::kTile;
  const int rows = w.tokens * p.G;
  auto q_row = [&](int row) -> const T* {
    const int t = row / p.G;
    return static_cast<const T*>(p.q) + ((long long)w.q0 + w.t0 + t) * p.q_stride + (w.g * p.G + row - t * p.G) * D;
  };
  auto load = [&](int t) {  // tile t into its stage
    const int s = t % F::kStages;
    const uint32_t dst = base + (uint32_t)(s * 2 * F::kBytes);
    mbar_expect_tx(full(s), 2 * F::kBytes);
#pragma unroll
    for (int v = 0; v < 2; ++v)
#pragma unroll
      for (int kb = 0; kb < F::kBoxes; ++kb)
        tma_load_2d(dst + v * F::kBytes + kb * F::kTile * 128, v ? &map_v : &map_k, w.g * D + kb * F::kBoxCols,
                    w.kv0 + key.first + t * F::kTile, full(s));
  };
  // the first tiles are on their way while the other warps bring the rows of q
  const int early = min(ntiles, F::kStages);
  if (producer) {
    if (lane == 0)
      for (int t = 0; t < early; ++t) load(t);
    __syncwarp();
  } else if constexpr (!F::kQRegs) {
    for (int i = threadIdx.x; i < 16 * MT * (D / 8); i += 32 * F::kConsumers) {
      const int row = i / (D / 8), c = (i % (D / 8)) * 8;
      uint4* dst = reinterpret_cast<uint4*>(sbase + F::oQ + row * F::kQPitch + c * 2);
      uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
      if (row < rows) {
        const uint4* q = reinterpret_cast<const uint4*>(q_row(row) + c);
        x = q[0];
        if constexpr (F::kF32) y = q[1];
      }
      if constexpr (F::kF32) {
        uint4 h, m, l;
        split(__uint_as_float(x.x), __uint_as_float(x.y), h.x, m.x, l.x);
        split(__uint_as_float(x.z), __uint_as_float(x.w), h.y, m.y, l.y);
        split(__uint_as_float(y.x), __uint_as_float(y.y), h.z, m.z, l.z);
        split(__uint_as_float(y.z), __uint_as_float(y.w), h.w, m.w, l.w);
        dst[F::kQPart / 16] = m;
        dst[2 * F::kQPart / 16] = l;
        x = h;
      }
      *dst = x;
    }
  }
  __syncthreads();
  auto fail = [&]() {
    *abort_flag = 1u;
    report(p.err, CP_ERR_TIMEOUT);
  };

  const int gid = lane >> 2, tig = lane & 3;
  const int wm = warp / F::kWK, wk = warp % F::kWK;
  float o[D / 8][4];
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  if (producer) {
    // ---- producer
    if (lane == 0) {
      int issued = early;
      for (int t = early; t < ntiles; ++t) {
        if (!mbar_wait(empty(t % F::kStages), ((uint32_t)(t / F::kStages) & 1u) ^ 1u, abort_flag, kBudget)) {
          fail();
          break;
        }
        load(t);
        issued = t + 1;
      }
      // every copy has landed before the CTA goes on to use the ring
      for (int t = max(0, issued - F::kStages); t < issued; ++t)
        mbar_wait(full(t % F::kStages), (uint32_t)(t / F::kStages) & 1u, nullptr, kBudget);
    }
    __syncwarp();
  } else if (wm * 16 < rows) {
    // ---- a consumer's rows and their keys
    uint32_t qa[F::kQRegs ? D / 16 : 1][4];
    int lo[2] = {0, 0}, hi[2] = {w.keys, w.keys};
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = wm * 16 + gid + 8 * r;
      const bool real = row < rows;
      if constexpr (F::kQRegs) {
        const T* q = q_row(real ? row : 0);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          qa[k][r] = real ? *reinterpret_cast<const uint32_t*>(q + 16 * k + 2 * tig) : 0u;
          qa[k][r + 2] = real ? *reinterpret_cast<const uint32_t*>(q + 16 * k + 8 + 2 * tig) : 0u;
        }
      }
      if (RANGES && real) cross_range(p, w, w.t0 + row / p.G, lo[r], hi[r]);
    }
    // q's fragment of a step: matrices (rows 0-7, 8-15) x (its first, second 16 bytes)
    const uint32_t sq = base + (uint32_t)(F::oQ + (wm * 16 + (lane & 15)) * F::kQPitch + (lane >> 4) * 16);
    int u0 = 0x7fffffff, u1 = -1;  // steps whose V held infinities or NaN that were taken out
    const float sc = p.scale_log2;
    bool ok = true;
    for (int t = 0; t < ntiles; ++t) {
      const int s = t % F::kStages;
      ok = __all_sync(0xffffffffu, mbar_wait(full(s), (uint32_t)(t / F::kStages) & 1u, abort_flag, kBudget));
      if (!ok) break;
      const uint32_t sk = base + (uint32_t)(s * 2 * F::kBytes), sv = sk + (uint32_t)F::kBytes;
#pragma unroll 1
      for (int st = 0; st < F::kKeys / F::kStep; ++st) {
        const int r0 = wk * F::kKeys + st * F::kStep;  // first row of the tile
        const int k0 = key.first + t * F::kTile + r0;  // first key
        if (k0 >= key.end) break;
        float c[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i) c[i][0] = c[i][1] = c[i][2] = c[i][3] = 0.f;
        // S = Q K^T
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t a[F::kF32 ? 3 : 1][4];
          if constexpr (F::kQRegs) {
#pragma unroll
            for (int i = 0; i < 4; ++i) a[0][i] = qa[k][i];
          } else {
#pragma unroll
            for (int i = 0; i < (F::kF32 ? 3 : 1); ++i) ldsm4(a[i], sq + 32u * k + (uint32_t)(i * F::kQPart));
          }
          if constexpr (F::kF32) {
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              const int row = r0 + 8 * i + gid;
              uint32_t h[2], m[2], l[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {  // dims 16 k + 8 e + 2 tig and the next
                const int chunk = 4 * (k & 1) + 2 * e + (tig >> 1);
                const float2 x = *reinterpret_cast<const float2*>(sbase + (sk - base) + (k / 2) * F::kTile * 128 + row * 128 +
                                                                  ((chunk ^ (row & 7)) << 4) + (tig & 1) * 8);
                split(x.x, x.y, h[e], m[e], l[e]);
              }
              mma_parts(c[i], a[0], a[1], a[2], h, m, l);
            }
          } else {
#pragma unroll
            for (int i = 0; i < NT; i += 2) {  // a matrix is 8 keys' 16 bytes
              const int row = r0 + 8 * i + ((lane >> 4) << 3) + (lane & 7), chunk = 2 * (k & 3) + ((lane >> 3) & 1);
              uint32_t b[4];
              ldsm4(b, sk + (uint32_t)((k / 4) * F::kTile * 128 + row * 128) + (uint32_t)((chunk ^ (row & 7)) << 4));
              mma_bf16(c[i], a[0], b[0], b[1]);
              mma_bf16(c[i + 1], a[0], b[2], b[3]);
            }
          }
        }
        const bool whole = k0 + F::kStep <= key.end && (!RANGES || (k0 >= key.all_lo && k0 + F::kStep <= key.all_hi));
        if (!whole) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int a = max(lo[r], key.first) - k0, b = min(hi[r], key.end) - k0;
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int at = 8 * i + 2 * tig + e;
                if (at < a || at >= b) c[i][2 * r + e] = -INFINITY;
              }
          }
        }
        float top[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          top[r] = fmaxf(c[0][2 * r], c[0][2 * r + 1]);
#pragma unroll
          for (int i = 1; i < NT; ++i) top[r] = fmaxf(top[r], fmaxf(c[i][2 * r], c[i][2 * r + 1]));
          top[r] *= sc;
        }
        if (__any_sync(0xffffffffu, top[0] > m[0] + kMaxGrowth || top[1] > m[1] + kMaxGrowth)) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
            top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
            float alpha = 1.f;
            if (top[r] > m[r]) {
              alpha = m[r] == -INFINITY ? 1.f : ex2(m[r] - top[r]);  // (no key yet: sums of 0)
              m[r] = top[r];
            }
            l[r] *= alpha;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) o[i][2 * r] *= alpha, o[i][2 * r + 1] *= alpha;
          }
        }
        const float n0 = m[0] == -INFINITY ? 0.f : -m[0], n1 = m[1] == -INFINITY ? 0.f : -m[1];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          c[i][0] = ex2(fmaf(c[i][0], sc, n0)), c[i][1] = ex2(fmaf(c[i][1], sc, n0));
          c[i][2] = ex2(fmaf(c[i][2], sc, n1)), c[i][3] = ex2(fmaf(c[i][3], sc, n1));
          l[0] += c[i][0] + c[i][1];
          l[1] += c[i][2] + c[i][3];
        }
        if (k0 + F::kStep > key.end) {  // V rows that are no key of any row
          const int n = key.end - k0;
          for (int i = lane; i < F::kBoxes * F::kStep * 8; i += 32) {
            const int row = (i >> 3) % F::kStep, kb = i / (8 * F::kStep);
            if (row >= n)
              *reinterpret_cast<uint4*>(sbase + (sv - base) + kb * F::kTile * 128 + (r0 + row) * 128 + (i & 7) * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
          }
          __syncwarp();
        }
        // O += P V: the scores' fragments are the MMA's A operand as they lie
        bool bad = false;
#pragma unroll
        for (int i = 0; i < NT; i += 2) {
          if constexpr (F::kF32) {
            uint32_t ph[4], pm[4], pl[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              split(c[i + (e >> 1)][2 * (e & 1)], c[i + (e >> 1)][2 * (e & 1) + 1], ph[e], pm[e], pl[e]);
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
              uint32_t h[2], m[2], l[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {  // keys 2 tig + 8 e and the next, dim 8 n + gid
                float x[2];
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                  const int row = r0 + 8 * i + 8 * e + 2 * tig + f, chunk = 2 * (n & 3) + (gid >> 2);
                  x[f] = *reinterpret_cast<const float*>(sbase + (sv - base) + (n / 4) * F::kTile * 128 + row * 128 +
                                                         ((chunk ^ (row & 7)) << 4) + (gid & 3) * 4);
                }
                split(x[0], x[1], h[e], m[e], l[e]);
                // (an infinity's middle part would be NaN, and 0 times it is NaN)
                const uint32_t odd = ((h[e] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
                if (odd != 0u) {
                  const uint32_t keep = ~((odd >> 15) * 0xffffu);
                  h[e] &= keep, m[e] &= keep, l[e] &= keep;
                  bad = true;
                }
              }
              mma_parts(o[n], ph, pm, pl, h, m, l);
            }
          } else {
            const uint32_t pa[4] = {pack2(c[i][0], c[i][1]), pack2(c[i][2], c[i][3]), pack2(c[i + 1][0], c[i + 1][1]),
                                    pack2(c[i + 1][2], c[i + 1][3])};
            const int row = r0 + 8 * i + (((lane >> 3) & 1) << 3) + (lane & 7);
#pragma unroll
            for (int n = 0; n < D / 8; n += 2) {
              const int chunk = (n & 7) + (lane >> 4);
              uint32_t b[4];
              ldsm4_t(b, sv + (uint32_t)((n / 8) * F::kTile * 128 + row * 128) + (uint32_t)((chunk ^ (row & 7)) << 4));
              if (RANGES && !whole)
#pragma unroll
                for (int e = 0; e < 4; ++e) bad = clean(b[e]) || bad;
              mma_bf16(o[n], pa, b[0], b[1]);
              mma_bf16(o[n + 1], pa, b[2], b[3]);
            }
          }
        }
        if (kRestore && __any_sync(0xffffffffu, bad)) u0 = min(u0, k0), u1 = max(u1, k0 + F::kStep);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(s));
    }
    if (!ok && lane == 0) fail();
    if (kRestore && u1 >= 0) {
      // what was taken out of V for the rows that see it: p > 0 times it is itself, whatever p is.  The warp's keys
      // are one slice in kWK of every tile.
      const T* v = static_cast<const T*>(p.v) + (long long)w.kv0 * p.v_stride + w.g * D;
#pragma unroll
      for (int r = 0; r < 2; ++r)
        for (int j = max(u0, lo[r]); j < min(min(u1, hi[r]), key.end); ++j)
          if (((j - key.first) % F::kTile) / F::kKeys == wk)
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float x = as_float(v[j * p.v_stride + 8 * i + 2 * tig + e]);
                if (!isfinite(x)) o[i][2 * r + e] += x;
              }
    }
  } else {
    // a warp without rows keeps the ring going
    for (int t = 0; t < ntiles; ++t) {
      const int s = t % F::kStages;
      if (!__all_sync(0xffffffffu, mbar_wait(full(s), (uint32_t)(t / F::kStages) & 1u, abort_flag, kBudget))) {
        if (lane == 0) fail();
        break;
      }
      if (lane == 0) mbar_arrive(empty(s));
    }
  }
  __syncthreads();  // the ring is done with
  auto& slices = *reinterpret_cast<typename F::Parts*>(sbase);
  if (warp < F::kConsumers) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      const int row = wm * 16 + gid + 8 * r;
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        *reinterpret_cast<float2*>(&slices.o[wk][row][8 * i + 2 * tig]) = make_float2(o[i][2 * r], o[i][2 * r + 1]);
      if (tig == 0) slices.m[wk][row] = m[r], slices.l[wk][row] = l[r];
    }
  }
  finish<T>(p, w, slices, cluster, piece);
}

// ------------------------------------------------------------------------------ launches
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
  return cudaLaunchKernelEx(&cfg, kern, args..., parts, cluster);
}

// Parts that meet in a cluster, or (`cut`) in the workspace.
struct Meet {
  int parts, cluster;
};
Meet meet(const CrossPlan& plan, const CrossParams& p, int in_cluster) {
  if (p.n_split > 0) return {plan.split_k, 1};
  return {in_cluster, in_cluster};
}

template <typename T, int D, int MT>
cudaError_t launch_few(const CrossParams& p, const CUtensorMap& mk, const CUtensorMap& mv, long long items, Meet m,
                       cudaStream_t s) {
  using F = Few<T, D, MT>;
  auto kern = p.ranges != nullptr ? few_kernel<T, D, MT, true> : few_kernel<T, D, MT, false>;
  return launch_parts(kern, items, m.parts, m.cluster, F::kThreads, F::kSmem, s, mk, mv, p);
}

template <typename T, int D>
cudaError_t launch_t(const cp_cross_args& a, const CrossPlan& plan, Meet m, const CrossParams& p, cudaStream_t s) {
  CUtensorMap mk, mv;
  constexpr unsigned tile = Few<T, D, 1>::kTile;
  const unsigned long long cols = (unsigned long long)p.Hkv * D;
  const bool any = p.Nkv > 0;  // (no key: never loaded from)
  const unsigned long long n = any ? p.Nkv : 1, ks = any ? a.k_stride : cols, vs = any ? a.v_stride : cols;
  const auto make = sizeof(T) == 4 ? cp_make_f32_map_2d : cp_make_bf16_map_2d;
  if (!make(&mk, any ? p.k : p.q, cols, n, ks, tile) || !make(&mv, any ? p.v : p.q, cols, n, vs, tile))
    return cudaErrorInvalidValue;
  const cudaError_t e = plan.rows <= 16 ? launch_few<T, D, 1>(p, mk, mv, plan.items, m, s)
                        : plan.rows <= 32 ? launch_few<T, D, 2>(p, mk, mv, plan.items, m, s)
                                          : launch_few<T, D, 4>(p, mk, mv, plan.items, m, s);
  if (e != cudaSuccess || p.n_split == 0) return e;
  return launch_merge<T, D>(p, s);
}

// Keys of a tile, and CTAs that are resident at once.
int tile_of(const cp_cross_args& a) { return 16384 / (a.head_dim * (a.dtype == CP_F32 ? 4 : 2)); }
template <typename T, int D>
int ctas_of(int rows) {
  return rows <= 16 ? Few<T, D, 1>::kCtas : rows <= 32 ? Few<T, D, 2>::kCtas : Few<T, D, 4>::kCtas;
}
int slots_of(const cp_cross_args& a, int rows, int sms) {
  if (a.dtype == CP_F32) return sms * (a.head_dim == 64 ? ctas_of<float, 64>(rows) : ctas_of<float, 128>(rows));
  return sms * (a.head_dim == 64 ? ctas_of<__nv_bfloat16, 64>(rows) : ctas_of<__nv_bfloat16, 128>(rows));
}

// Parts of an item that meet in a cluster: as many as the GPU takes at once, each with a tile at least.  More items than
// that: parts of eight tiles or more until there are twice as many as the GPU takes, so that the last ones are short (64 sequences
// of 512 .. 4096 states, 8 kv heads, three CTAs on an SM: 101.5 us; 105.5 whole, 109 with four times as many).
int cluster_of(const cp_cross_args& a, const CrossPlan& c, int sms) {
  const int tile = tile_of(a);
  const long long key_tiles = ((long long)a.max_seqlen_kv + tile - 1) / tile, slots = slots_of(a, c.rows, sms);
  long long parts = slots / c.items;
  if (parts < 1) {
    parts = (2 * slots + c.items - 1) / c.items;
    if (parts > key_tiles / 8) parts = key_tiles / 8;
  }
  if (parts > key_tiles) parts = key_tiles;
  return (int)(parts < 1 ? 1 : parts > kMaxCluster ? kMaxCluster : parts);
}

}  // namespace
}  // namespace cpattn

CrossPlan cp_cross_plan_few(const cp_cross_args& a, int sms) {
  CrossPlan c;
  c.span = cp_cross_span(a);
  c.tiles = cp_cross_tiles(a);
  c.rows = c.span * (a.num_q_heads / a.num_kv_heads);
  c.items = (long long)a.num_seqs * a.num_kv_heads * c.tiles;
  c.n_split = 0;
  c.split_k = 1;
  c.ordered = 0;
  // more parts than a cluster takes, through the workspace: where eight leave most of the GPU idle and the keys are
  // many enough to pay for a second launch
  const int tile = cpattn::tile_of(a);
  const long long key_tiles = ((long long)a.max_seqlen_kv + tile - 1) / tile, slots = cpattn::slots_of(a, c.rows, sms);
  if (c.items * cpattn::kMaxCluster * 2 <= slots && key_tiles >= 8 * cpattn::kMaxCluster) {
    long long k = slots / c.items;
    if (k > key_tiles / 2) k = key_tiles / 2;
    if (k > cpattn::kMaxParts) k = cpattn::kMaxParts;
    c.split_k = (int)k;
    c.n_split = c.items;
  }
  c.bytes = cp_cross_parts_bytes(c, a.head_dim);
  return c;
}

cudaError_t cp_launch_cross_few(const cp_cross_args& a, float scale, void* ws, size_t ws_bytes, void* out, float* lse,
                                cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const CrossPlan plan = cp_cross_plan_few(a, sms);
  cpattn::CrossParams p;
  cp_cross_fill(p, a, plan, scale, ws, ws_bytes, out, lse);
  const cpattn::Meet m = cpattn::meet(plan, p, cpattn::cluster_of(a, plan, sms));
  if (a.dtype == CP_F32)
    return a.head_dim == 64 ? cpattn::launch_t<float, 64>(a, plan, m, p, s) : cpattn::launch_t<float, 128>(a, plan, m, p, s);
  return a.head_dim == 64 ? cpattn::launch_t<__nv_bfloat16, 64>(a, plan, m, p, s)
                          : cpattn::launch_t<__nv_bfloat16, 128>(a, plan, m, p, s);
}
