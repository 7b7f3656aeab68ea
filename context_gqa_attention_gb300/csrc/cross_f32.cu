// Cross attention (cp_cross_attention) in f32, of any number of query rows (items of up to 64): the beams of a source in a
// decode step above all.  No counterpart on the pages, whose attention is causal self-attention.
//
//   out_i = softmax over the keys j in [lo_i, hi_i) of scale q_i.k_j, times V
//
// Each operand is the sum of three bf16 numbers (high, middle, low: 24 bits) and a product the sum of the six of theirs
// that count, in fp32, on the legacy tensor path.  (Products of tf32 pairs, three of them: 25 cycles of a sub-partition each
// against 8.1 for a bf16 MMA, which has twice the work.)
//
// Bound: for up to 8 rows a kv head HBM once there is work for every SM (152 sequences of 2000 states, d = 128: 5.8 TB/s, 85%
// of the copy; d = 64: 5.2); for 16 rows 4.5 TB/s, for 32 the tensor pipe at 3.1.  8 sequences of 0 .. 900 states, 5 beams of
// 16 heads, d = 64: 15.4 us against 3.5 for their bytes: the start, the longest part, the cluster's meeting.
#include "cross_few.cuh"

namespace cpattn {
namespace {

// A transposed matrix of 8 x 8 16-bit elements (row lane / 4, two a lane).
CP_DEV uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// x and y = high + middle + low, as pairs of bf16.
CP_DEV void split(float x, float y, uint32_t& h, uint32_t& m, uint32_t& l) {
  h = pack2(x, y);
  x -= __uint_as_float(h << 16), y -= __uint_as_float(h & 0xffff0000u);
  m = pack2(x, y);
  x -= __uint_as_float(m << 16), y -= __uint_as_float(m & 0xffff0000u);
  l = pack2(x, y);
}

// A score that the parts' products left NaN, once more.  Where an element's bf16 is an infinity (the element is one, or a
// number above 3.39e38 that rounds to one) its lowest part is NaN, and so is every product of it: such a score is the sum of
// the elements' own products.  Others stay as they are.
template <int D>
__device__ __noinline__ float odd_score(const float* q, const float* k, float c) {
  float s = 0.f;
  bool odd = false;
  auto take = [&](float x, float y) {
    odd = odd || max(__float_as_uint(x) & 0x7fffffffu, __float_as_uint(y) & 0x7fffffffu) >= 0x7f7f8000u;
    s = fmaf(x, y, s);
  };
#pragma unroll 1
  for (int i = 0; i < D && !isnan(s); i += 4) {  // (a NaN stays: 300 rows of NaN over 8000 keys 0.78 ms, others 0.41)
    const float4 x = *reinterpret_cast<const float4*>(q + i), y = *reinterpret_cast<const float4*>(k + i);
    take(x.x, y.x), take(x.y, y.y), take(x.z, y.z), take(x.w, y.w);
  }
  return odd ? s : c;
}

// The products are taken transposed, S^T = K Q^T and O^T = V^T P^T: a tile of K or V is an MMA's 16 rows and the query rows
// are its 8 columns, so that 5 beams are padded to 8, and the many splits of K and V serve all query rows.  A producer warp
// brings tiles of 16 keys through a ring (TMA, 128-byte swizzle); consumer warp (m, g) takes every kGroups-th tile for the NB
// columns' blocks m, with a softmax reference of its own, so warps meet at the end only.  (Tiles of a warp's own, because
// what bounds a warp is the latency of its chains: six MMAs on each accumulator, 20 cycles each.  With the query rows as the
// MMA's 16 rows and warps on slices of the same tiles: 80 us where this takes 54, for 4 sequences of up to 7668 states, 9 rows, 8 kv
// heads.)
template <int D, int NB, int MW>
struct Fp32 {
  static constexpr int kRows = 8 * NB * MW;
  static constexpr int kTile = 16, kBytes = kTile * D * 4, kBoxes = D / 32;
  // CTAs on an SM, and warps that take turns at the tiles: as many as the registers allow (128, 168, 255 a thread)
  static constexpr int kCtas = NB <= 2 ? 2 : 1, kGroups = MW == 2 ? 3 : NB == 1 && D == 64 ? 7 : NB <= 2 ? 5 : 7;
  static constexpr int kConsumers = MW * kGroups, kThreads = 32 * (kConsumers + 1);
  // q as bf16, rows 16 bytes apart in the banks, the three parts one behind the other
  static constexpr int kQPitch = D * 2 + 16, kQPart = kRows * kQPitch;
  using Parts = Slices<D, kGroups, kRows, 4>;
  static constexpr int align16(int x) { return (x + 15) / 16 * 16; }
  static constexpr int smem_of(int stages) {
    const int work = stages * 2 * kBytes + 3 * kQPart, parts = align16((int)sizeof(Parts));
    return (work > parts ? work : parts) + 16 * stages + 1024;  // (the base is rounded up to the swizzle atom)
  }
  static constexpr int stages() {
    int n = 2;
    while (n < 12 && (smem_of(n + 1) + 1024) * kCtas <= 232448) ++n;
    return n;
  }
  static constexpr int kStages = stages();
  static constexpr int oQ = kStages * 2 * kBytes, oBar = smem_of(kStages) - 1024 - 16 * kStages;
  static constexpr int kSmem = smem_of(kStages);
};

template <int D, int NB, int MW, bool RANGES>
__global__ void __launch_bounds__(Fp32<D, NB, MW>::kThreads, Fp32<D, NB, MW>::kCtas)
    f32_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const CrossParams p,
               const int parts, const int cluster) {
  using F = Fp32<D, NB, MW>;
  constexpr int KS = D / 16;  // MMA steps over the dims
  constexpr int kChains = NB == 1 ? 2 : 1;  // accumulators that take turns in a dot product, for shorter chains
  extern __shared__ uint8_t smem_raw[];
  __shared__ int s_range[4];
  __shared__ uint32_t s_abort;
  __shared__ int s_issued;  // tiles whose copies have been issued
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
      mbar_init(empty(s), MW);
    }
    s_abort = 0u;
    s_issued = F::kStages;  // (or all)
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
  } else {
    for (int i = threadIdx.x; i < F::kRows * (D / 8); i += 32 * F::kConsumers) {
      const int row = i / (D / 8), c = (i % (D / 8)) * 8, t = row / p.G;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
      if (row < rows) {
        const float4* q = reinterpret_cast<const float4*>(
            static_cast<const float*>(p.q) + ((long long)w.q0 + w.t0 + t) * p.q_stride + (w.g * p.G + row - t * p.G) * D + c);
        x = q[0], y = q[1];
      }
      uint4 h, m, l;
      split(x.x, x.y, h.x, m.x, l.x);
      split(x.z, x.w, h.y, m.y, l.y);
      split(y.x, y.y, h.z, m.z, l.z);
      split(y.z, y.w, h.w, m.w, l.w);
      uint4* dst = reinterpret_cast<uint4*>(sbase + F::oQ + row * F::kQPitch + c * 2);
      dst[0] = h;
      dst[F::kQPart / 16] = m;
      dst[2 * F::kQPart / 16] = l;
    }
  }
  __syncthreads();
  auto fail = [&]() {
    *abort_flag = 1u;
    report(p.err, CP_ERR_TIMEOUT);
  };
  // Tile t is there.  A barrier's phases are told apart by parity alone, and a warp has not seen the tile that was in the stage
  // before: only once t has been issued is that one's phase over for certain.
  const uint32_t issued_at = smem_u32(&s_issued);
  auto arrived = [&](int t) -> bool {
    const long long t0 = clock64();
    for (uint32_t it = 1; t >= F::kStages; ++it) {
      int n;
      asm volatile("ld.acquire.cta.shared.b32 %0, [%1];" : "=r"(n) : "r"(issued_at) : "memory");
      if (n > t) break;
      if ((it & 31u) == 0 && (*abort_flag != 0u || clock64() - t0 > kBudget)) return false;
    }
    return mbar_wait(full(t % F::kStages), (uint32_t)(t / F::kStages) & 1u, abort_flag, kBudget);
  };

  const int gid = lane >> 2, tig = lane & 3;
  const int wm = warp / F::kGroups, group = warp % F::kGroups, row0 = wm * 8 * NB;
  // O^T: dims 16 i + gid (and + 8) of the query rows row0 + 8 n + 2 tig (and the next)
  float o[KS][NB][4], m[NB][2], l[NB][2];
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    m[n][0] = m[n][1] = -INFINITY;
    l[n][0] = l[n][1] = 0.f;
#pragma unroll
    for (int i = 0; i < KS; ++i) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
  }
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
        asm volatile("st.release.cta.shared.b32 [%0], %1;" ::"r"(issued_at), "r"(issued) : "memory");
      }
      // every copy has landed before the CTA goes on to use the ring
      for (int t = max(0, issued - F::kStages); t < issued; ++t)
        mbar_wait(full(t % F::kStages), (uint32_t)(t / F::kStages) & 1u, nullptr, kBudget);
    }
    __syncwarp();
  } else if (row0 < rows) {
    // ---- a consumer's rows and their keys
    int lo[NB][2], hi[NB][2];
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = row0 + 8 * n + 2 * tig + e;
        lo[n][e] = 0, hi[n][e] = w.keys;
        if (RANGES && row < rows) cross_range(p, w, w.t0 + row / p.G, lo[n][e], hi[n][e]);
      }
    // q's B fragments of 16 dims: matrices (dims 0-7, 8-15), and those of a second block of rows
    const uint32_t sq = base + (uint32_t)(F::oQ + (row0 + (lane & 7)) * F::kQPitch + ((lane >> 3) & 1) * 16);
    const uint32_t second = (uint32_t)((lane >> 4) * 8 * F::kQPitch);
    int u0 = 0x7fffffff, u1 = -1;  // steps whose V held infinities or NaN that were taken out
    const float sc = p.scale_log2;
    bool ok = true;
    for (int t = group; t < ntiles; t += F::kGroups) {
      const int s = t % F::kStages;
      ok = __all_sync(0xffffffffu, arrived(t));
      if (!ok) break;
      const uint8_t *pk = sbase + s * 2 * F::kBytes, *pv = pk + F::kBytes;
      const int k0 = key.first + t * F::kTile;  // first key
      // S^T = K Q^T: keys gid (and + 8), rows 2 tig (and the next)
      float c[NB][4], chain[kChains][NB][4];
#pragma unroll
      for (int i = 0; i < kChains; ++i)
#pragma unroll
        for (int n = 0; n < NB; ++n) chain[i][n][0] = chain[i][n][1] = chain[i][n][2] = chain[i][n][3] = 0.f;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t h[4], md[4], lw[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // key gid + 8 (e & 1), dims 16 k + 8 (e >> 1) + 2 tig and the next
          const int row = gid + 8 * (e & 1), chunk = 4 * (k & 1) + 2 * (e >> 1) + (tig >> 1);
          const float2 x = *reinterpret_cast<const float2*>(pk + (k / 2) * F::kTile * 128 + row * 128 +
                                                            ((chunk ^ (row & 7)) << 4) + (tig & 1) * 8);
          split(x.x, x.y, h[e], md[e], lw[e]);
        }
#pragma unroll
        for (int n = 0; n < NB; n += 2) {
          uint32_t bh[4], bm[4], bl[4];
          const uint32_t a = sq + (uint32_t)(8 * n * F::kQPitch) + 32u * k + (n + 1 < NB ? second : 0u);
          ldsm4(bh, a);
          ldsm4(bm, a + F::kQPart);
          ldsm4(bl, a + 2 * F::kQPart);
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            if (n + f >= NB) break;
            float(&d)[4] = chain[k % kChains][n + f];
            mma_bf16(d, lw, bh[2 * f], bh[2 * f + 1]);
            mma_bf16(d, h, bl[2 * f], bl[2 * f + 1]);
            mma_bf16(d, md, bm[2 * f], bm[2 * f + 1]);
            mma_bf16(d, md, bh[2 * f], bh[2 * f + 1]);
            mma_bf16(d, h, bm[2 * f], bm[2 * f + 1]);
            mma_bf16(d, h, bh[2 * f], bh[2 * f + 1]);
          }
        }
      }
      const bool whole = k0 + 16 <= key.end && (!RANGES || (k0 >= key.all_lo && k0 + 16 <= key.all_hi));
      float top[NB][2];
      bool moves = false, odd = false;
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          c[n][e] = chain[0][n][e], c[n][e + 2] = chain[0][n][e + 2];
          if (kChains > 1) c[n][e] += chain[kChains - 1][n][e], c[n][e + 2] += chain[kChains - 1][n][e + 2];
          if (!whole) {
            const int a = max(lo[n][e], key.first) - k0, b = min(hi[n][e], key.end) - k0;
            if (gid < a || gid >= b) c[n][e] = -INFINITY;
            if (gid + 8 < a || gid + 8 >= b) c[n][e + 2] = -INFINITY;
          }
          odd = odd || isnan(c[n][e]) || isnan(c[n][e + 2]);
        }
      if (odd) {  // (rare; a masked score is -inf, so a NaN is that of a key that the row sees)
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int row = row0 + 8 * n + 2 * tig + (e & 1), t = row / p.G;
            if (row < rows && isnan(c[n][e]))
              c[n][e] = odd_score<D>(
                  static_cast<const float*>(p.q) + ((long long)w.q0 + w.t0 + t) * p.q_stride + (w.g * p.G + row - t * p.G) * D,
                  static_cast<const float*>(p.k) + ((long long)w.kv0 + k0 + gid + 8 * (e >> 1)) * p.k_stride + w.g * D, c[n][e]);
          }
      }
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          top[n][e] = fmaxf(c[n][e], c[n][e + 2]) * sc;
          moves = moves || top[n][e] > m[n][e] + kMaxGrowth;
        }
      if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = top[n][e], alpha = 1.f;
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            if (x > m[n][e]) {
              alpha = m[n][e] == -INFINITY ? 1.f : ex2(m[n][e] - x);  // (no key yet: sums of 0)
              m[n][e] = x;
            }
            l[n][e] *= alpha;
#pragma unroll
            for (int i = 0; i < KS; ++i) o[i][n][e] *= alpha, o[i][n][e + 2] *= alpha;
          }
      }
      // P^T as B fragments (three parts), two keys a lane: the transposed scores' accumulators
      uint32_t ph[NB][2], pm[NB][2], pl[NB][2];
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        const float n0 = m[n][0] == -INFINITY ? 0.f : -m[n][0], n1 = m[n][1] == -INFINITY ? 0.f : -m[n][1];
#pragma unroll
        for (int e = 0; e < 4; ++e) c[n][e] = ex2(fmaf(c[n][e], sc, (e & 1) ? n1 : n0));
        l[n][0] += c[n][0] + c[n][2];
        l[n][1] += c[n][1] + c[n][3];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          split(c[n][2 * e], c[n][2 * e + 1], ph[n][e], pm[n][e], pl[n][e]);
          ph[n][e] = transposed(ph[n][e]), pm[n][e] = transposed(pm[n][e]), pl[n][e] = transposed(pl[n][e]);
        }
      }
      if (k0 + 16 > key.end) {  // V rows that are no key of any row
        const int z = key.end - k0;
        for (int i = lane; i < F::kBoxes * 16 * 8; i += 32) {
          const int row = (i >> 3) & 15, kb = i >> 7;
          if (row >= z)
            *reinterpret_cast<uint4*>(sbase + s * 2 * F::kBytes + F::kBytes + kb * F::kTile * 128 + row * 128 +
                                      (i & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        __syncwarp();
      }
      // O^T += V^T P^T
      bool bad = false;
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        uint32_t h[4], md[4], lw[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // dim 16 i + 8 (e & 1) + gid, keys 8 (e >> 1) + 2 tig and the next
          float x[2];
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            const int row = 8 * (e >> 1) + 2 * tig + f, chunk = 4 * (i & 1) + 2 * (e & 1) + (gid >> 2);
            x[f] = *reinterpret_cast<const float*>(pv + (i / 2) * F::kTile * 128 + row * 128 +
                                                   ((chunk ^ (row & 7)) << 4) + (gid & 3) * 4);
          }
          split(x[0], x[1], h[e], md[e], lw[e]);
          // (an infinity's middle part would be NaN, and 0 times it is NaN)
          const uint32_t odd = ((h[e] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
          if (odd != 0u) {
            const uint32_t keep = ~((odd >> 15) * 0xffffu);
            h[e] &= keep, md[e] &= keep, lw[e] &= keep;
            bad = true;
          }
        }
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          mma_bf16(o[i][n], lw, ph[n][0], ph[n][1]);
          mma_bf16(o[i][n], h, pl[n][0], pl[n][1]);
          mma_bf16(o[i][n], md, pm[n][0], pm[n][1]);
          mma_bf16(o[i][n], md, ph[n][0], ph[n][1]);
          mma_bf16(o[i][n], h, pm[n][0], pm[n][1]);
          mma_bf16(o[i][n], h, ph[n][0], ph[n][1]);
        }
      }
      if (__any_sync(0xffffffffu, bad)) u0 = min(u0, k0), u1 = max(u1, k0 + 16);
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(s));
    }
    if (!ok && lane == 0) fail();
    if (u1 >= 0) {
      // what was taken out of V for the rows that see it: p > 0 times it is itself, however small p
      const float* v = static_cast<const float*>(p.v) + (long long)w.kv0 * p.v_stride + w.g * D;
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          for (int j = max(u0, lo[n][e]); j < min(min(u1, hi[n][e]), key.end); ++j)
            if (((j - key.first) / F::kTile) % F::kGroups == group)
#pragma unroll
              for (int i = 0; i < KS; ++i)
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                  const float x = v[j * p.v_stride + 16 * i + 8 * f + gid];
                  if (!isfinite(x)) o[i][n][2 * f + e] += x;
                }
    }
  } else {
    // a warp without rows keeps the ring going
    for (int t = group; t < ntiles; t += F::kGroups) {
      if (!__all_sync(0xffffffffu, arrived(t))) {
        if (lane == 0) fail();
        break;
      }
      if (lane == 0) mbar_arrive(empty(t % F::kStages));
    }
  }
  __syncthreads();  // the ring is done with
  auto& slices = *reinterpret_cast<typename F::Parts*>(sbase);
  if (!producer) {
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = row0 + 8 * n + 2 * tig + e;
        float x = l[n][e];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
#pragma unroll
        for (int i = 0; i < KS; ++i)
          slices.o[group][row][16 * i + gid] = o[i][n][e], slices.o[group][row][16 * i + 8 + gid] = o[i][n][e + 2];
        if (gid == 0) slices.m[group][row] = m[n][e], slices.l[group][row] = x;
      }
  }
  finish<float>(p, w, slices, cluster, piece);
}

template <int D, int NB, int MW>
cudaError_t launch_f32(const CrossParams& p, const CUtensorMap& mk, const CUtensorMap& mv, long long items, int parts,
                       int cluster, cudaStream_t s) {
  using F = Fp32<D, NB, MW>;
  auto kern = p.ranges != nullptr ? f32_kernel<D, NB, MW, true> : f32_kernel<D, NB, MW, false>;
  return launch_parts(kern, items, parts, cluster, F::kThreads, F::kSmem, s, mk, mv, p, parts, cluster);
}
template <int D>
cudaError_t launch_d(const cp_cross_args& a, const CrossPlan& plan, int parts, int cluster, const CrossParams& p,
                     cudaStream_t s) {
  CUtensorMap mk, mv;
  if (!few_maps(a, p, Fp32<D, 1, 1>::kTile, &mk, &mv)) return cudaErrorInvalidValue;
  const cudaError_t e = plan.rows <= 8    ? launch_f32<D, 1, 1>(p, mk, mv, plan.items, parts, cluster, s)
                        : plan.rows <= 16 ? launch_f32<D, 2, 1>(p, mk, mv, plan.items, parts, cluster, s)
                        : plan.rows <= 24 ? launch_f32<D, 3, 1>(p, mk, mv, plan.items, parts, cluster, s)
                        : plan.rows <= 32 ? launch_f32<D, 4, 1>(p, mk, mv, plan.items, parts, cluster, s)
                                          : launch_f32<D, 4, 2>(p, mk, mv, plan.items, parts, cluster, s);
  if (e != cudaSuccess || p.n_split == 0) return e;
  return launch_merge<float, D>(p, s);
}

}  // namespace
}  // namespace cpattn

int cp_cross_f32_ctas(int rows) { return rows <= 16 ? cpattn::Fp32<64, 1, 1>::kCtas : cpattn::Fp32<64, 4, 1>::kCtas; }
cudaError_t cp_launch_cross_f32(const cp_cross_args& a, const CrossPlan& plan, int parts, int cluster, float scale, void* ws,
                                size_t ws_bytes, void* out, float* lse, cudaStream_t s) {
  cpattn::CrossParams p;
  cp_cross_fill(p, a, plan, scale, ws, ws_bytes, out, lse);
  return a.head_dim == 64 ? cpattn::launch_d<64>(a, plan, parts, cluster, p, s)
                          : cpattn::launch_d<128>(a, plan, parts, cluster, p, s);
}
