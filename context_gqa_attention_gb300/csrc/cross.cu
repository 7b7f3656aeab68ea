// Cross attention (cp_cross_attention) of many query rows on the 5th-generation tensor cores: bf16 in, f32
// accumulate.  No counterpart on the pages, whose attention is causal self-attention.
//
//   out_i = softmax over the keys j in [lo_i, hi_i) of scale q_i.k_j, times V
//
// Without causality every row of a sequence sees the same keys, so the G query heads of a kv head are packed: a
// tile of 128 rows is floor(128 / G) tokens under all G heads (one 3D box of q), whatever G is, and a CTA works
// on two consecutive tiles that share every K / V tile of 128 keys.  Warps:
//   0      TMA producer: both Q tiles once, then K and V tiles through a 4-slot ring
//   1      TMEM owner and MMA issuer (one thread): S = Q K^T, then O += P V with P read from TMEM; order
//          PV0(t) | QK0(t+1) | PV1(t) | QK1(t+1), so a tile's softmax overlaps the other's two MMAs
//   2-3    V guards: 0 times an infinity or a NaN is NaN, so they clear the V rows behind the last key, and with
//          key ranges (RANGES) every element that is not finite in tiles that some row sees in part
//   4-11   two softmax warpgroups, one a tile, a thread a row
// Parts: the keys of the last wave's items, or of all when they are few, are cut so that every SM has work; they meet in the
// shared memory of a cluster (CLUSTER), or in the workspace, where cross_merge_kernel joins them.
//
// Bound: the chain of a row tile, softmax - PV - QK^T, about 2780 cycles a key tile of two row tiles (d = 128) against 2150 of
// MMA: 8192 tokens over 6404 states, 16/2 heads, d = 128 take 292 to 315 us by the board (73 to 78% of the measured peak).  Short items: the
// start (about 4000 cycles: item, Q, first K tile and scores) and the way out (1700 to 3500).  9 prompts of 1 .. 447 tokens over
// 200 .. 1500 states, 16 heads, d = 64: 19.1 us; 3 texts of 600 .. 2500 tokens with ranges of 1025 of 3000 .. 8000 states, 32/8
// heads, d = 128: 113 us (33%: an eighth of the row tiles lies across two ranges and sees both).
//
// Every wait is bounded; on expiry the CTA raises CP_ERR_TIMEOUT, drains its copies and MMAs, frees TMEM and returns.
#include <cuda.h>

#include "cross.cuh"
#include "guard.cuh"
#include "rows.cuh"

namespace cpattn {
namespace {

constexpr int kThreads = 384;
constexpr int kSlots = 4;
constexpr int kRegsFirst = 72, kRegsSoftmax = 216, kRegsLaunch = 168;
static_assert(kRegsFirst + 2 * kRegsSoftmax <= 3 * kRegsLaunch, "register budgets exceed the launch");

template <int D, bool CLUSTER>
struct Smem {
  static constexpr int kQ = BM * D * 2;
  static constexpr int kKV = BN * D * 2;
  static constexpr int oQ = 0;
  static constexpr int oKV = 2 * kQ;
  static constexpr int oBar = oKV + kSlots * kKV;
  static constexpr int bQ = 0, bFull = 1, bEmpty = bFull + kSlots, bS = bEmpty + kSlots, bP = bS + 2, bO = bP + 2,
                       bFix = bO + 2, bLast = bFix + 2, bDone = bLast + 1, nBar = bDone + 1;
  static constexpr int oMisc = oBar + nBar * 8;  // TMEM base, abort flag, first / last unclean tile, keys of each row tile
  static constexpr int oM = oMisc + 48, oL = oM + 4 * 2 * BM;  // of a cluster: a row's reference and sum,
  static constexpr int oW = oL + 4 * 2 * BM;                    // and the parts' weights of this CTA's share of the rows
  static constexpr int kBytes = CLUSTER ? oW + 4 * kMaxCluster * BM : oM;
  // the base is rounded up to the 1 KB swizzle atom; never below 120 KB, so that one CTA (and its 512 TMEM
  // columns) has an SM to itself
  static constexpr int kAlloc = (kBytes + 1024) > 120 * 1024 ? (kBytes + 1024) : 120 * 1024;
  static_assert(kAlloc <= 232448, "dynamic shared memory beyond the 227 KB per-CTA limit");
};

// Columns outside [c0, c1), by bits, which become predicates several at a time.
CP_DEV uint32_t first_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }
CP_DEV void mask_columns(float (&v)[32], int c0, int c1) {
  const uint32_t seen = first_bits(c1) & ~first_bits(c0);
#pragma unroll
  for (int k = 0; k < 32; ++k) v[k] = (seen & (1u << k)) != 0u ? v[k] : -INFINITY;
}

template <int D, bool RANGES, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, 1)
    cross_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                 const __grid_constant__ CUtensorMap map_v, const CrossParams p) {
  using Sm = Smem<D, CLUSTER>;
  constexpr int KB = D / 64;
  extern __shared__ uint8_t smem_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* sbase = smem_raw + (base - raw);
  const uint32_t sQ = base + Sm::oQ, sKV = base + Sm::oKV;
  auto bar = [&](int i) -> uint32_t { return base + (uint32_t)Sm::oBar + 8u * (uint32_t)i; };
  int* misc = reinterpret_cast<int*>(sbase + Sm::oMisc);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(misc + 1);
  auto fail = [&]() {
    *abort_flag = 1u;
    report(p.err, CP_ERR_TIMEOUT);
  };
  // what needs nothing of the call's memory comes before the last call is waited for
  if (threadIdx.x == 0) {
    mbar_init(bar(Sm::bQ), 1);
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(bar(Sm::bFull + s), 1);
      mbar_init(bar(Sm::bEmpty + s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(Sm::bS + i), 1);
      mbar_init(bar(Sm::bP + i), 4);
      mbar_init(bar(Sm::bO + i), 1);
      mbar_init(bar(Sm::bFix + i), 2);
    }
    mbar_init(bar(Sm::bLast), 1);
    mbar_init(bar(Sm::bDone), 1);
    misc[1] = 0;
    misc[2] = 0x7fffffff;  // unclean tiles
    misc[3] = -1;
    for (int i = 4; i < 12; i += 4) {
      misc[i] = 0x7fffffff;  // [4, 5): keys that some row of tile 0 sees, [6, 7): that every row sees; then tile 1
      misc[i + 1] = 0;
      misc[i + 2] = 0;
      misc[i + 3] = 0x7fffffff;
    }
    fence_mbar_init();
    tma_prefetch_desc(&map_q);
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(misc), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)misc[0];

  // ---- the item, or the part of one
  int piece = -1, part = 0;
  unsigned index = blockIdx.x;
  if (CLUSTER) {
    part = (int)(index % (unsigned)p.cluster);
    index /= (unsigned)p.cluster;
  } else if ((int)index >= p.n_whole) {
    piece = (int)index - p.n_whole;
    part = piece % p.split_k;
    index = (unsigned)p.n_whole + (unsigned)(piece / p.split_k);
  }
  const CrossItem w = cross_item(p, index, threadIdx.x == 0 && part == 0);
  if (w.tokens == 0) {
    if (warp == 1) tmem_dealloc(tmem, 512);
    return;
  }
  const int per_tile = p.span / 2;  // tokens
  const int rows0 = min(w.tokens, per_tile) * p.G, rows1 = max(0, w.tokens - per_tile) * p.G;
  const bool two = rows1 > 0;
  if (threadIdx.x == 32) {  // (a copy takes its thread about 100 cycles; the producer's first ones go out meanwhile)
    mbar_expect_tx(bar(Sm::bQ), (two ? 2 : 1) * KB * per_tile * p.G * 128);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (i == 0 || two)
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
          tma_load_3d(sQ + i * Sm::kQ + kb * BM * 128, &map_q, kb * 64, w.g * p.G, w.q0 + w.t0 + i * per_tile,
                      bar(Sm::bQ));
  }
  if constexpr (RANGES) {  // a softmax warp a stretch of its row tile's tokens
    if (warp >= 4) {
      const int i = (warp - 4) >> 2, first = i * per_tile, n = min(per_tile, w.tokens - first);
      int lo = 0x7fffffff, hi = 0, all_lo = 0, all_hi = 0x7fffffff;
      for (int t = (int)threadIdx.x - 128 - 128 * i; t < n; t += 128) {
        int a, b;
        cross_range(p, w, w.t0 + first + t, a, b);
        if (a < b) lo = min(lo, a), hi = max(hi, b);
        all_lo = max(all_lo, a), all_hi = min(all_hi, b);
      }
      lo = __reduce_min_sync(0xffffffffu, lo), hi = __reduce_max_sync(0xffffffffu, hi);
      all_lo = __reduce_max_sync(0xffffffffu, all_lo), all_hi = __reduce_min_sync(0xffffffffu, all_hi);
      if (lane == 0) {
        int* m = misc + 4 + 4 * i;
        atomicMin(m, lo);
        atomicMax(m + 1, hi);
        atomicMax(m + 2, all_lo);
        atomicMin(m + 3, all_hi);
      }
    }
    __syncthreads();
  }
  // Key tiles of this CTA, counted from the first key that some row sees; each row tile works on those that one of its
  // rows sees.
  const int key_lo = RANGES ? min(misc[4], misc[8]) : 0, key_hi = RANGES ? max(misc[5], misc[9]) : w.keys;
  const int every = key_lo < key_hi ? (key_hi - key_lo + BN - 1) / BN : 0;
  int ta = 0, ntiles = every;
  if (CLUSTER || piece >= 0) {
    const int parts = CLUSTER ? p.cluster : p.split_k;
    ta = (int)((long long)every * part / parts);
    ntiles = (int)((long long)every * (part + 1) / parts) - ta;
  }
  const int k_first = key_lo + ta * BN;  // first key
  int t_lo[2], t_hi[2], all_lo[2], all_hi[2];  // a row tile's key tiles; the keys that all its rows see
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int lo = RANGES ? misc[4 + 4 * i] : 0, hi = RANGES ? misc[5 + 4 * i] : w.keys;
    const bool any = (i == 0 || two) && lo < hi;
    t_lo[i] = any ? min(ntiles, max(0, (lo - k_first) / BN)) : 0;
    t_hi[i] = any ? max(t_lo[i], min(ntiles, (hi - k_first + BN - 1) / BN)) : 0;
    all_lo[i] = RANGES ? misc[6 + 4 * i] : 0;
    all_hi[i] = RANGES ? misc[7 + 4 * i] : w.keys;
  }
  auto has = [&](int i, int t) -> bool { return t >= t_lo[i] && t < t_hi[i]; };
  auto in_part = [&](int t) -> bool {  // some row that works on key tile t sees only a part of it
    const int k0 = k_first + t * BN;
    bool r = false;
#pragma unroll
    for (int i = 0; i < 2; ++i) r = r || (has(i, t) && (k0 + BN > all_hi[i] || (RANGES && k0 < all_lo[i])));
    return r;
  };
  // keys of tile t that some row may see; 32 or fewer (a last tile) take a short way
  auto keys_in = [&](int t) -> int { return key_hi - k_first - t * BN; };
  // Without ranges the guards have only the last V tile to clean, if at all.  It lands at a barrier of its own: on the
  // ring's they would have to follow every phase, in step with the issuer.
  const bool clean_last = !RANGES && in_part(ntiles - 1);
  // where a row of tile i goes
  auto out_row = [&](int i, int row) -> long long {
    const int t = row / p.G;
    return ((long long)w.q0 + w.t0 + i * per_tile + t) * p.Hq + w.g * p.G + (row - t * p.G);
  };

  if (!CLUSTER && ntiles <= 0) {  // no key
    const int rows = rows0 + rows1;
    for (int r = threadIdx.x; r < rows; r += kThreads) {
      const int i = r >= rows0 ? 1 : 0, row = r - i * rows0;
      if (piece >= 0) {
        p.ws_lse[(long long)piece * p.rows + i * per_tile * p.G + row] = -INFINITY;
        continue;
      }
      const long long o = out_row(i, row);
      uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + o * D);
      for (int c = 0; c < D / 8; ++c) dst[c] = make_uint4(0u, 0u, 0u, 0u);
      if (p.lse != nullptr) p.lse[o] = -INFINITY;
    }
    if (threadIdx.x == 0) mbar_wait(bar(Sm::bQ), 0u, nullptr, kBudget);  // Q has landed before the CTA exits
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, 512);
    return;
  }

  if (warp < 4) {
    regs_dec<kRegsFirst>();
    if (warp == 0) {
      // ---------------------------------------------------------------- TMA producer
      if (lane == 0) {
        bool ok = true;
        int issued = 0;  // ring fills: K(t) is fill 2 t, V(t) fill 2 t + 1
        for (int i = 0; i < 2 * ntiles; ++i) {
          const int slot = i % kSlots;
          if (!mbar_wait(bar(Sm::bEmpty + slot), ((uint32_t)(i / kSlots) & 1u) ^ 1u, abort_flag, kBudget)) {
            ok = false;
            break;
          }
          const CUtensorMap* map = (i & 1) ? &map_v : &map_k;
          const uint32_t full = bar(clean_last && i == 2 * ntiles - 1 ? Sm::bLast : Sm::bFull + slot);
          mbar_expect_tx(full, Sm::kKV);
          tma_load_3d(sKV + slot * Sm::kKV, map, 0, w.kv0 + k_first + (i >> 1) * BN, w.g * KB, full);
          issued = i + 1;
        }
        if (!ok) fail();
        // every copy issued into this CTA's shared memory has landed before it exits
        mbar_wait(bar(Sm::bQ), 0u, nullptr, kBudget);
        for (int i = max(0, issued - kSlots); i < issued; ++i) {
          if (clean_last && i == 2 * ntiles - 1) mbar_wait(bar(Sm::bLast), 0u, nullptr, kBudget);
          else mbar_wait(bar(Sm::bFull + i % kSlots), (uint32_t)(i / kSlots) & 1u, nullptr, kBudget);
        }
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------------- MMA issuer
      if (lane == 0) {
        const uint32_t id_qk = idesc_bf16_f32(BM, BN, false, false);
        const uint32_t id_pv = idesc_bf16_f32(BM, D, false, true);
        // descriptors built once and advanced: this thread is on the critical path
        const uint64_t dq0 = desc_sw128(sQ, 16, 1024);
        const uint64_t dk0 = desc_sw128(sKV, 16, 1024);
        const uint64_t dv0 = desc_sw128(sKV, BN * 128, 1024);
        auto issue_qk = [&](int tile, int slot) {
          const uint64_t dq = desc_advance(dq0, (uint32_t)(tile * Sm::kQ));
          const uint64_t dk = desc_advance(dk0, (uint32_t)(slot * Sm::kKV));
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk / 4) * (BM * 128) + (kk % 4) * 32;
            mma_ss(tmem + (uint32_t)(tile * BN), desc_advance(dq, off), desc_advance(dk, off), id_qk, kk > 0);
          }
          mma_commit(bar(Sm::bS + tile));
        };
        auto issue_pv = [&](int tile, int slot, bool acc, bool few) {
          const uint64_t dv = desc_advance(dv0, (uint32_t)(slot * Sm::kKV));
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk) {
            if (kk == 2 && few) break;
            mma_ts(tmem + 256u + (uint32_t)(tile * D), tmem + (uint32_t)(tile * BN + kk * 8),
                   desc_advance(dv, kk * 16u * 128u), id_pv, acc || kk > 0);
          }
          mma_commit(bar(Sm::bO + tile));
        };
        bool ok = (CLUSTER && ntiles == 0) || (mbar_wait(bar(Sm::bQ), 0u, abort_flag, kBudget) &&
                                  mbar_wait(bar(Sm::bFull), 0u, abort_flag, kBudget));
        if (ok && (!CLUSTER || ntiles > 0)) {
          tc_fence_after();
          if (has(0, 0)) issue_qk(0, 0);
          if (has(1, 0)) issue_qk(1, 0);
          mma_commit(bar(Sm::bEmpty + 0));
        }
        for (int t = 0; ok && t < ntiles; ++t) {
          const int iv = 2 * t + 1, ik = 2 * t + 2, sv = iv % kSlots, sk = ik % kSlots;
          const bool few = keys_in(t) <= 32;
          // V(t), with ranges and in a last tile in part as the guards leave it
          if (!RANGES && clean_last && t == ntiles - 1) {
            ok = mbar_wait(bar(Sm::bFix), 0u, abort_flag, kBudget);
          } else {
            ok = mbar_wait(bar(Sm::bFull + sv), (uint32_t)(iv / kSlots) & 1u, abort_flag, kBudget);
            if (RANGES) ok = ok && mbar_wait(bar(Sm::bFix + (t & 1)), (uint32_t)(t >> 1) & 1u, abort_flag, kBudget);
          }
          if (has(0, t)) {
            ok = ok && mbar_wait(bar(Sm::bP + 0), (uint32_t)(t - t_lo[0]) & 1u, abort_flag, kBudget);
            if (!ok) break;
            tc_fence_after();
            issue_pv(0, sv, t > t_lo[0], few);
          }
          const bool more = t + 1 < ntiles;
          if (more) {
            ok = ok && mbar_wait(bar(Sm::bFull + sk), (uint32_t)(ik / kSlots) & 1u, abort_flag, kBudget);
            if (!ok) break;
            tc_fence_after();
            if (has(0, t + 1)) issue_qk(0, sk);
          }
          if (has(1, t)) {
            ok = ok && mbar_wait(bar(Sm::bP + 1), (uint32_t)(t - t_lo[1]) & 1u, abort_flag, kBudget);
            if (!ok) break;
            tc_fence_after();
            issue_pv(1, sv, t > t_lo[1], few);
          }
          if (!ok) break;
          mma_commit(bar(Sm::bEmpty + sv));
          if (more) {
            if (has(1, t + 1)) issue_qk(1, sk);
            mma_commit(bar(Sm::bEmpty + sk));
          }
        }
        if (!ok) fail();
        // every MMA issued by this thread has retired before TMEM is released
        mma_commit(bar(Sm::bDone));
        mbar_wait(bar(Sm::bDone), 0u, nullptr, kBudget);
      }
    } else {
      // ---------------------------------------------------------------- V guards
      // with ranges every tile, in step with the MMA issuer: a barrier's phases are told apart by parity alone
      for (int t = RANGES ? 0 : ntiles - 1; t < ntiles; ++t) {
        if (!RANGES && !clean_last) break;
        const int iv = 2 * t + 1, sv = iv % kSlots;
        const bool ok = __all_sync(0xffffffffu, RANGES ? mbar_wait(bar(Sm::bFull + sv), (uint32_t)(iv / kSlots) & 1u,
                                                                   abort_flag, kBudget)
                                                       : mbar_wait(bar(Sm::bLast), 0u, abort_flag, kBudget));
        if (!ok) {
          if (lane == 0) fail();
          break;
        }
        uint8_t* tile = sbase + Sm::oKV + sv * Sm::kKV;
        const int last = key_hi - k_first - t * BN;  // rows from here on are no key of any row
        if constexpr (RANGES) {
          if (in_part(t)) {
            if (guard_v<D, BN>(tile, last, (warp - 2) * 32 + lane)) {
              atomicMin(misc + 2, t);
              atomicMax(misc + 3, t);
            }
            fence_proxy_async_smem();  // the MMA reads what was written here
          }
        } else {
          for (int i = (warp - 2) * 32 + lane; i < Sm::kKV / 16; i += 64)
            if (((i >> 3) & (BN - 1)) >= last) reinterpret_cast<uint4*>(tile)[i] = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(Sm::bFix + (RANGES ? t & 1 : 0)));
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax, one warpgroup per tile
    regs_inc<kRegsSoftmax>();
    const int tile = (warp - 4) >> 2, q4 = warp & 3;
    const int row = q4 * 32 + lane, rows = tile == 0 ? rows0 : rows1;
    const int t0 = t_lo[tile], t1 = t_hi[tile];
    float* row_m = reinterpret_cast<float*>(sbase + Sm::oM) + tile * BM + row;  // (CLUSTER)
    float* row_l = reinterpret_cast<float*>(sbase + Sm::oL) + tile * BM + row;
    if (rows > 0 && t0 == t1) {  // no key for this tile's rows
      if (row < rows) {
        const long long o = out_row(tile, row);
        if constexpr (CLUSTER) {
          *row_m = -INFINITY, *row_l = 0.f;
        } else if (piece >= 0) {
          p.ws_lse[(long long)piece * p.rows + tile * per_tile * p.G + row] = -INFINITY;
        } else {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + o * D);
          for (int c = 0; c < D / 8; ++c) dst[c] = make_uint4(0u, 0u, 0u, 0u);
          if (p.lse != nullptr) p.lse[o] = -INFINITY;
        }
      }
    } else if (rows > 0) {
      const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
      const uint32_t tS = tmem + lane_off + (uint32_t)(tile * BN);
      const uint32_t tO = tmem + lane_off + 256u + (uint32_t)(tile * D);
      int lo = 0, hi = w.keys;
      if (RANGES && row < rows) cross_range(p, w, w.t0 + tile * per_tile + row / p.G, lo, hi);
      float m = -INFINITY, l = 0.f;
      bool ok = true;
      for (int t = t0; t < t1; ++t) {
        ok = __all_sync(0xffffffffu, mbar_wait(bar(Sm::bS + tile), (uint32_t)(t - t0) & 1u, abort_flag, kBudget));
        if (!ok) break;
        tc_fence_after();
        const int k0 = k_first + t * BN;
        float s0[32], s1[32], s2[32], s3[32];
        float alpha;
        if (keys_in(t) <= 32) {  // a last tile of few keys
          tmem_ld32(tS, s0);
          tmem_wait_ld(s0);
          mask_columns(s0, lo - k0, hi - k0);
          float mt = s0[0];
#pragma unroll
          for (int k = 1; k < 32; ++k) mt = fmaxf(mt, s0[k]);
          mt *= p.scale_log2;
          alpha = 1.f;
          if (mt > m + kRescaleThreshold) {
            alpha = ex2(m - mt);
            m = mt;
          }
          const float neg = m == -INFINITY ? 0.f : -m;
          uint64_t sum2 = f2(0.f, 0.f);
          exp_pack_tmem(s0, f2(p.scale_log2, p.scale_log2), f2(neg, neg), sum2, tS);
          tmem_wait_st();
          float a, b;
          f2u(sum2, a, b);
          l = l * alpha + (a + b);
        } else {
          load_row(tS, s0, s1, s2, s3);
          int lim = hi - 1 - k0;
          if constexpr (RANGES) {
            if (!__all_sync(0xffffffffu, lo <= k0 && hi >= k0 + BN)) {
              mask_columns(s0, lo - k0, hi - k0);
              mask_columns(s1, lo - k0 - 32, hi - k0 - 32);
              mask_columns(s2, lo - k0 - 64, hi - k0 - 64);
              mask_columns(s3, lo - k0 - 96, hi - k0 - 96);
            }
            lim = BN - 1;
          }
          alpha = row_max_update(s0, s1, s2, s3, lim, p.scale_log2, m);
          // S(t) complete implies PV(t-1) complete (it was issued before QK(t)): O is stable and the S columns may
          // take P(t)
          l = l * alpha + row_exp_tmem(s0, s1, s2, s3, p.scale_log2, m, tS);
        }
        if (t > t0) rescale_o<D>(tO, alpha);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(Sm::bP + tile));
      }
      if (ok)
        ok = __all_sync(0xffffffffu, mbar_wait(bar(Sm::bO + tile), (uint32_t)(t1 - t0 - 1) & 1u, abort_flag, kBudget));
      // (with ranges a row tile may be done before the other, whose operands lie where it would stage its rows)
      if (RANGES && ok) ok = __all_sync(0xffffffffu, mbar_wait(bar(Sm::bDone), 0u, abort_flag, kBudget));
      if (ok) {
        tc_fence_after();
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const float lse = l == 0.f ? -INFINITY : ((m == -INFINITY ? 0.f : m) + log2f(l)) * kLn2;
        // what the guards took out of V and this row sees: p > 0 times it is itself, however small p
        if constexpr (RANGES) {
          const int u0 = *(volatile int*)(misc + 2), u1 = *(volatile int*)(misc + 3);
          if (u1 >= 0) {
            const int r0 = max(lo, k_first + u0 * BN), r1 = min(hi, k_first + (u1 + 1) * BN);
            const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.v) + (long long)w.kv0 * p.v_stride;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              float o[32];
              tmem_ld32(tO + c, o);
              tmem_wait_ld(o);
              if (row < rows) restore<D>(o, v, p.v_stride, w.g * D + c, r0, r1);
              __syncwarp();
              tmem_st32(tO + c, o);
            }
            tmem_wait_st();
          }
        }
        // Rows go out through shared memory, one whole row an instruction: tile 0 over the Q tiles (free: its last
        // PV came after the other tile's last QK), tile 1 over the ring (its last PV is the CTA's last MMA)
        const int mine = min(32, rows - q4 * 32);  // rows of this warp
        const bool f32 = CLUSTER || piece >= 0;
        const uint32_t sb = (tile == 0 ? sQ : sKV) + (uint32_t)(q4 * 32 * D * (f32 ? 4 : 2));
        if constexpr (CLUSTER) {
          stage_rows_f32<D>(tO, 1.f, sb, lane);
          *row_m = m, *row_l = l;
        } else if (piece >= 0) {
          stage_rows_f32<D>(tO, inv, sb, lane);
          __syncwarp();
          const long long r0 = (long long)piece * p.rows + tile * per_tile * p.G + q4 * 32;
          if (mine == 32) {
            store_staged_f32<D>(sb, lane, p.ws_out + r0 * D, D);
          } else if (mine > 0) {
            for (int r = 0; r < mine; ++r)
              for (int c = lane; c < D; c += 32) {
                float x;
                asm volatile("ld.shared.f32 %0, [%1];"
                             : "=f"(x)
                             : "r"(sb + (uint32_t)((c / 32) * 4096 + r * 128) +
                                   ((uint32_t)(((c % 32) / 4) ^ (r & 7)) << 4) + (uint32_t)(c % 4) * 4u));
                p.ws_out[(r0 + r) * D + c] = x;
              }
          }
          if (lane < mine) p.ws_lse[r0 + lane] = lse;
        } else if (mine > 0) {
          stage_rows_bf16<D>(tO, inv, sb, lane);
          __syncwarp();
          const long long o = out_row(tile, min(row, rows - 1));
          constexpr int kLanes = D / 8, kAt = 32 / kLanes;  // lanes of a row, 16 bytes each, and rows at a time
          const int c = lane % kLanes;
          const uint32_t a0 = sb + (uint32_t)((c / 8) * 4096);
#pragma unroll 8
          for (int r0 = 0; r0 < 32; r0 += kAt) {
            const int r = r0 + lane / kLanes;
            const long long at = __shfl_sync(0xffffffffu, o, r) * D + 8 * c;
            if (r0 >= mine) break;
            if (r < mine) {
              uint4 x;
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                           : "r"(a0 + (uint32_t)(r * 128) + ((uint32_t)((c & 7) ^ (r & 7)) << 4)));
              *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + at) = x;
            }
          }
          if (lane < mine && p.lse != nullptr) p.lse[o] = lse;
        }
      } else if (lane == 0) {
        fail();
      }
    }
    if constexpr (CLUSTER) {
      // ---- the parts' rows as one: CTA r takes the r-th share of them
      __syncwarp();
      cluster_sync();
      const int n = rows0 + rows1, rank = (int)cluster_rank(), k = p.cluster;
      const int r0 = n * rank / k, mine = n * (rank + 1) / k - r0, tid = (int)threadIdx.x - 128;
      float* weight = reinterpret_cast<float*>(sbase + Sm::oW);
      auto slot = [&](int r) { return r < rows0 ? r : BM + r - rows0; };  // of a row of the item among those of both tiles
      if (tid < mine) {
        const uint32_t at = 4u * (uint32_t)slot(r0 + tid);
        float ms[kMaxCluster], ls[kMaxCluster], M = -INFINITY, L = 0.f;
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {
          ms[c] = c < k ? peer_ld(peer_addr(sbase + Sm::oM, c) + at) : -INFINITY;
          ls[c] = c < k ? peer_ld(peer_addr(sbase + Sm::oL, c) + at) : 0.f;
          M = fmaxf(M, ms[c]);
        }
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {
          ms[c] = ls[c] == 0.f ? 0.f : factor(ms[c], M);
          L += ms[c] * ls[c];
        }
        const float inv = L == 0.f ? 0.f : 1.f / L;
        // (-1: a part without keys, whose rows are not read; a weight of 0 times what is not finite is NaN)
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) weight[c * BM + tid] = ls[c] == 0.f ? -1.f : ms[c] * inv;
        if (p.lse != nullptr) p.lse[r0 + tid < rows0 ? out_row(0, r0 + tid) : out_row(1, r0 + tid - rows0)] = natural_lse(M, L);
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
      for (int i = tid; i < mine * (D / 4); i += 256) {
        const int r = i / (D / 4), c4 = i % (D / 4), s = slot(r0 + r), row32 = s & 31;
        const uint32_t at = (uint32_t)((s >> 7) * 2 * Sm::kQ + (s & 127) / 32 * (32 * D * 4) + (c4 / 8) * 4096 + row32 * 128) +
                            ((uint32_t)((c4 & 7) ^ (row32 & 7)) << 4);
        float4 x[kMaxCluster], o = make_float4(0.f, 0.f, 0.f, 0.f);
        float e[kMaxCluster];
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {
          e[c] = c < k ? weight[c * BM + r] : -1.f;
          if (!(e[c] < 0.f)) x[c] = peer_ld4(peer_addr(sbase, c) + at);
        }
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c)
          if (!(e[c] < 0.f)) o.x += e[c] * x[c].x, o.y += e[c] * x[c].y, o.z += e[c] * x[c].z, o.w += e[c] * x[c].w;
        const long long to = (r0 + r < rows0 ? out_row(0, r0 + r) : out_row(1, r0 + r - rows0)) * D + 4 * c4;
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + to) = make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
      }
      __syncwarp();
      cluster_sync();  // no CTA leaves while another reads its shared memory
    }
  }
  if (CLUSTER && warp < 4) {
    __syncwarp();
    cluster_sync();
    cluster_sync();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch(const cp_cross_args& a, const CrossPlan& plan, float scale, void* ws, size_t ws_bytes, void* out,
                   float* lse, cudaStream_t s) {
  CrossParams p;
  cp_cross_fill(p, a, plan, scale, ws, ws_bytes, out, lse);
  CUtensorMap mq, mk, mv;
  const unsigned per_tile = (unsigned)p.span / 2;
  if (!cp_make_bf16_map_3d(&mq, a.q, D, (unsigned long long)p.Hq, (unsigned long long)p.Nq,
                           (unsigned long long)a.q_stride, (unsigned)p.G, per_tile))
    return cudaErrorInvalidValue;
  if (p.Nkv > 0) {
    const unsigned long long blocks = (unsigned long long)p.Hkv * (D / 64), rows = (unsigned long long)p.Nkv;
    if (!cp_make_columns_map(&mk, a.k, 2, blocks, rows, (unsigned long long)a.k_stride, BN, D / 64) ||
        !cp_make_columns_map(&mv, a.v, 2, blocks, rows, (unsigned long long)a.v_stride, BN, D / 64))
      return cudaErrorInvalidValue;
  } else {
    mk = mv = mq;  // (no key: never loaded from)
  }
  const long long grid = p.n_whole + (long long)p.n_split * p.split_k;
  if (grid * p.cluster >= (1ll << 31)) return cudaErrorInvalidConfiguration;
  auto kern = a.key_ranges != nullptr ? cross_kernel<D, true, false>
              : p.cluster > 1         ? cross_kernel<D, false, true>
                                      : cross_kernel<D, false, false>;
  // the warpgroups' register budgets assume the registers a thread of this launch gets; a build that gave the
  // kernel another count would leave an increase waiting, so refuse it
  cudaFuncAttributes fa;
  cudaError_t e = cudaFuncGetAttributes(&fa, kern);
  if (e != cudaSuccess) return e;
  if (fa.numRegs != kRegsLaunch) return cudaErrorInvalidKernelImage;
  const int smem = p.cluster > 1 ? Smem<D, true>::kAlloc : Smem<D, false>::kAlloc;
  e = launch_parts(kern, grid, p.cluster, p.cluster, kThreads, smem, s, mq, mk, mv, p);
  if (e != cudaSuccess || p.n_split == 0) return e;
  return launch_merge<__nv_bfloat16, D>(p, s);
}

}  // namespace
}  // namespace cpattn

// Time of an item: about 2.5 us and 1.75 a key tile (d = 64: 3 and 1.3), one on an SM.  Its keys are cut in one of two ways.
// Parts that meet in the workspace take 3 us more to write their fp32 rows, and the merge about 3 us and 0.05 a part; of items
// that are all alike, those of whole waves stay whole and the rest are cut.  Parts of every item that meet in a cluster (up
// to eight CTAs) take 4 us more (d = 128: 6 to 8, the fewer parts the more), and pay only where all clusters run at once: the
// clusters of k CTAs that find k free SMs in one group are 76, 46, 36, 28, 23, 15 and 15 for k = 2 .. 8 by the occupancy query, some
// fewer here, since other GPUs have other SMs switched off.  (8 items of 2000 states, d = 64: 13.1 us through the workspace, 12.0
// in clusters of eight; 16: 16.1 and 13.3 in clusters of six, 22.4 of eight, which take turns; 32: 17.9 and 14.5 of four.)
// Not for rows with ranges, whose keys are fewer than the totals say.
// Where items differ, how many there are and how long can only be guessed from the totals: the load of an SM and half of the
// longest item decide.
CrossPlan cp_cross_plan_tc(const cp_cross_args& a, int sms) {
  CrossPlan c;
  const double B = a.num_seqs;
  c.span = cp_cross_span(a);
  c.tiles = cp_cross_tiles(a);
  c.rows = c.span * (a.num_q_heads / a.num_kv_heads);
  c.items = (long long)a.num_seqs * a.num_kv_heads * c.tiles;
  c.n_split = 0;
  c.split_k = 1;
  const bool alike = a.key_ranges == nullptr && a.kv_lens == nullptr &&
                     (a.num_seqs == 1 || (B * a.max_seqlen_q <= a.total_q && B * a.max_seqlen_kv <= a.total_kv));
  c.ordered = !alike && a.num_seqs > 1 && a.num_seqs <= 32;
  const double most = ceil(a.max_seqlen_kv / (double)cpattn::BN);
  const double usual = alike ? most : fmin(most, ceil(a.total_kv / B / cpattn::BN));
  const double live = alike ? (double)c.items
                            : fmin((double)c.items, a.num_kv_heads * ((double)a.total_q / c.span + 0.5 * B));
  const double fixed = a.head_dim == 64 ? 3 : 2.5, tile = a.head_dim == 64 ? 1.3 : 1.75;
  const double waves = alike ? floor(live / sms) : 0, rest = live - waves * sms;
  double best = 0;
  for (int k = 1; k <= 32 && k <= most && (k == 1 || rest * k <= 4.0 * sms); ++k) {
    const double set_up = k > 1 ? fixed + 3 : fixed;
    const double part = set_up + tile * ceil(usual / k), longest = set_up + tile * ceil(most / k);
    double t = alike ? ceil(rest * k / sms) * part : fmax(rest * k * part / sms + 0.5 * longest, longest);
    if (k > 1) t += 3 + 0.05 * rest * k;
    if (k == 1 || t < 0.97 * best) {
      best = t;
      c.split_k = k;
    }
  }
  c.cluster = 1;
  constexpr int kAtOnce[cpattn::kMaxCluster + 1] = {0, 0, 72, 44, 34, 26, 22, 14, 14};  // of 152 SMs
  for (int k = 2; k <= cpattn::kMaxCluster && k <= most && a.key_ranges == nullptr; ++k) {
    if (live * 152 > kAtOnce[k] * sms) break;
    const double t = fixed + (a.head_dim == 64 ? 3.4 + 2.4 / k : 4.8 + 6.0 / k) + tile * ceil(most / k);
    if (t < 0.97 * best) {
      best = t;
      c.cluster = k;
    }
  }
  if (c.cluster > 1) c.split_k = 1;
  if (c.split_k > 1) c.n_split = alike ? (long long)rest : c.items;
  if (c.n_split == 0) c.split_k = 1;
  c.bytes = cp_cross_parts_bytes(c, a.head_dim);
  return c;
}

cudaError_t cp_launch_cross_tc(const cp_cross_args& a, float scale, void* ws, size_t ws_bytes, void* out, float* lse,
                               cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const CrossPlan plan = cp_cross_plan_tc(a, sms);
  return a.head_dim == 64 ? cpattn::launch<64>(a, plan, scale, ws, ws_bytes, out, lse, s)
                          : cpattn::launch<128>(a, plan, scale, ws, ws_bytes, out, lse, s);
}
