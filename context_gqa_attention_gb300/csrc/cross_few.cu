// Cross attention (cp_cross_attention) of few query rows in bf16: the beams of a source in a decode step, a short prompt.
// No counterpart on the pages, whose attention is causal self-attention.
//
//   out_i = softmax over the keys j in [lo_i, hi_i) of scale q_i.k_j, times V
//
// The rows of an item (CrossParams) are all that a kv head's states are read for, so the time is that of the states:
// bytes, not operations.  Parts of the keys run at once and meet in a cluster's shared memory (up to eight), or in
// the workspace (cross_merge_kernel) where a few long items have to fill the GPU.
#include "cross_few.cuh"

namespace cpattn {
namespace {

// ------------------------------------------------------------------------------ the kernel
// 64 sequences of 512 .. 4096 states, 4 beams of 32/8 heads, d = 128: 97.4 us (6.17 TB/s, 91% of the copy); one sequence of 1500
// states, 16 heads, d = 64: 6.2 us, latency of the launch, the first loads and the cluster's meeting.
//
// MMAs of 16 rows on the legacy tensor path: a 128-row tcgen05 tile would be padding.  A producer warp brings tiles of
// K and V through a ring (TMA, 128-byte swizzle); consumer warp (m, k) owns the 16 rows m and the k-th slice of every
// tile's keys, with a softmax reference of its own, so warps meet at the end only.  The reference moves when a score
// exceeds it by more than 2^8, which a vote of the warp finds; rows' sums stay in the lanes until the end.
// Halves that are infinite or NaN become 0; whether there were any.
CP_DEV bool clean(uint32_t& w) {
  const uint32_t bad = ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;  // an exponent of all ones carries
  w &= ~((bad >> 15) * 0xffffu);
  return bad != 0u;
}
template <int D, int MT>
struct Few {
  static constexpr int kWK = MT == 4 ? 2 : 4;        // slices of a tile's keys
  static constexpr int kConsumers = MT * kWK;
  static constexpr int kThreads = 32 * (kConsumers + 1);
  static constexpr int kBytes = 16384;               // of a tile of K or of V
  static constexpr int kTile = kBytes / (D * 2);  // keys
  static constexpr int kKeys = kTile / kWK;          // of a warp
  static constexpr int kStep = kKeys < 32 ? kKeys : 32;
  static_assert(kStep % 16 == 0, "steps of the second product");
  static constexpr int kBoxes = D / 64;
  // q as A fragments in registers (one row group), or in shared memory: rows 16 bytes apart in the banks
  static constexpr bool kQRegs = MT == 1;
  static constexpr int kQPitch = D * 2 + 16, kQBytes = kQRegs ? 0 : 16 * MT * kQPitch;
  using Parts = Slices<D, kWK, 16 * MT, 8>;
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

template <int D, int MT, bool RANGES>
__global__ void __launch_bounds__(Few<D, MT>::kThreads, Few<D, MT>::kCtas)
    few_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const CrossParams p,
               const int parts, const int cluster) {
  using F = Few<D, MT>;
  using T = __nv_bfloat16;
  constexpr int NT = F::kStep / 8;
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
    tma_load_3d(dst, &map_k, 0, w.kv0 + key.first + t * F::kTile, w.g * F::kBoxes, full(s));
    tma_load_3d(dst + F::kBytes, &map_v, 0, w.kv0 + key.first + t * F::kTile, w.g * F::kBoxes, full(s));
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
      uint4 x = make_uint4(0u, 0u, 0u, 0u);
      if (row < rows) x = *reinterpret_cast<const uint4*>(q_row(row) + c);
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
          uint32_t a[4];
          if constexpr (F::kQRegs) {
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = qa[k][i];
          } else {
            ldsm4(a, sq + 32u * k);
          }
#pragma unroll
          for (int i = 0; i < NT; i += 2) {  // a matrix is 8 keys' 16 bytes
            const int row = r0 + 8 * i + ((lane >> 4) << 3) + (lane & 7), chunk = 2 * (k & 3) + ((lane >> 3) & 1);
            uint32_t b[4];
            ldsm4(b, sk + (uint32_t)((k / 4) * F::kTile * 128 + row * 128) + (uint32_t)((chunk ^ (row & 7)) << 4));
            mma_bf16(c[i], a, b[0], b[1]);
            mma_bf16(c[i + 1], a, b[2], b[3]);
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
        if (RANGES && __any_sync(0xffffffffu, bad)) u0 = min(u0, k0), u1 = max(u1, k0 + F::kStep);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(s));
    }
    if (!ok && lane == 0) fail();
    if (RANGES && u1 >= 0) {
      // what was taken out of V for the rows that see it: p > 0 times it is itself, however small p.  The warp's keys
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
                const float x = __bfloat162float(v[j * p.v_stride + 8 * i + 2 * tig + e]);
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

// Parts that meet in a cluster, or (`cut`) in the workspace.
struct Meet {
  int parts, cluster;
};
Meet meet(const CrossPlan& plan, const CrossParams& p, int in_cluster) {
  if (p.n_split > 0) return {plan.split_k, 1};
  return {in_cluster, in_cluster};
}

template <int D, int MT>
cudaError_t launch_few(const CrossParams& p, const CUtensorMap& mk, const CUtensorMap& mv, long long items, Meet m,
                       cudaStream_t s) {
  using F = Few<D, MT>;
  auto kern = p.ranges != nullptr ? few_kernel<D, MT, true> : few_kernel<D, MT, false>;
  return launch_parts(kern, items, m.parts, m.cluster, F::kThreads, F::kSmem, s, mk, mv, p, m.parts, m.cluster);
}

template <int D>
cudaError_t launch_d(const cp_cross_args& a, const CrossPlan& plan, Meet m, const CrossParams& p, cudaStream_t s) {
  CUtensorMap mk, mv;
  if (!few_maps(a, p, Few<D, 1>::kTile, &mk, &mv)) return cudaErrorInvalidValue;
  const cudaError_t e = plan.rows <= 16 ? launch_few<D, 1>(p, mk, mv, plan.items, m, s)
                        : plan.rows <= 32 ? launch_few<D, 2>(p, mk, mv, plan.items, m, s)
                                          : launch_few<D, 4>(p, mk, mv, plan.items, m, s);
  if (e != cudaSuccess || p.n_split == 0) return e;
  return launch_merge<__nv_bfloat16, D>(p, s);
}

// 16 KB of keys (what the plan counts in), and CTAs that are resident at once.
int tile_of(const cp_cross_args& a) { return 16384 / (a.head_dim * (a.dtype == CP_F32 ? 4 : 2)); }
template <int D>
int ctas_of(int rows) {
  return rows <= 16 ? Few<D, 1>::kCtas : rows <= 32 ? Few<D, 2>::kCtas : Few<D, 4>::kCtas;
}
int slots_of(const cp_cross_args& a, int rows, int sms) {
  if (a.dtype == CP_F32) return sms * cp_cross_f32_ctas(rows);
  return sms * (a.head_dim == 64 ? ctas_of<64>(rows) : ctas_of<128>(rows));
}

// Parts of an item that meet in a cluster, by an estimate.  A CTA takes about 4.5 us and a time for each tile of its part;
// all together no less than the memory's rate allows (f32: or the tensor pipe's, for NB blocks of 8 rows).  If all run at
// once the longest decides, else the load of a place and most of the longest.  How far lengths differ is only known from
// the totals; of a padded batch they are taken to be about half of the longest.  (22 sequences of 674 .. 5392 states, 8 kv
// heads, 24 rows: 94 us whole, 72 in three; 64 of 512 .. 4096, 16 rows: 105.5 whole, 98.6 in two, 109 in four; 43 of up to
// 268, 4 kv heads: 6.6 whole, 11.2 in two; f32, 4 of up to 7668, 8 kv heads, 9 rows: 84 in three, 54 in eight.)
int cluster_of(const cp_cross_args& a, const CrossPlan& c, int sms) {
  const bool f32 = a.dtype == CP_F32;
  const double tile = tile_of(a), slots = slots_of(a, c.rows, sms), items = (double)c.items;
  const double longest = ceil(a.max_seqlen_kv / tile);
  const double usual = fmin(a.kv_lens != nullptr && a.num_seqs > 1 ? 0.55 * longest : longest, a.total_kv / (double)a.num_seqs / tile);
  const double each = f32 ? 1.1 : c.rows <= 16 ? 0.55 : 1.0;
  const double all = 3 + items * usual * fmax(0.0051, f32 ? 0.22 / sms * ceil(c.rows / 8.0) : 0.0);
  int best = 1;
  double least = 0;
  for (int k = 1; k <= kMaxCluster && (k == 1 || k <= longest); ++k) {
    const double ctas = items * k, most = 4.5 + each * ceil(longest / k);
    const double t = ctas <= slots ? fmax(most, all)
                                   : fmax(ctas / slots * (4.5 + each * usual / k), all + 3 * ctas / slots) + 0.75 * most;
    if (k == 1 || t < 0.97 * least) best = k, least = t;
  }
  return best;
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
  c.cluster = 1;  // (cluster_of says)
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
  if (a.dtype == CP_F32) return cp_launch_cross_f32(a, plan, m.parts, m.cluster, scale, ws, ws_bytes, out, lse, s);
  return a.head_dim == 64 ? cpattn::launch_d<64>(a, plan, m, p, s) : cpattn::launch_d<128>(a, plan, m, p, s);
}
