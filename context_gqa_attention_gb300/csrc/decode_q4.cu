// Decode over a round-robin paged cache held in 4 bits (cp_decode_attention_q4), one query token per
// sequence, bf16 queries; scores may be modified as in decode_mod.cu.
//
// "Add utility functions to enable pass-kv prefill and allgather decode" (vLLM PR 26059),
// Purpose: decode KV stays on the CP ranks round-robin, each rank attends the new query over its
// own tokens and the partials are combined.  The 4-bit format is this library's (include/cpattn.h).
//
// Work unit and MMA shapes as in decode_mod.cu: S^T = K Q^T with the tokens, O^T = V^T P^T with the
// head's dims as the M dimension, 8 query heads as N.  Per token and group of 64 dims the value is
// minimum + scale n, so
//   q.k   = sum over groups of  scale (q.n) + minimum (sum of q)
//   out_d = sum over tokens of  (p scale) n_d + p minimum
// and the MMAs see the bare codes n; everything else is a few fp32 operations per score.
//
// What bounds it: a page costs the same instructions whether its rows have 256 or 64 bytes, so at a
// quarter of the traffic the instruction pipes are as near as HBM.  Hence
//  * a code becomes an MMA operand by one AND for two values (f16 subnormals, see codes());
//  * the running reference of the softmax moves only when a score exceeds it by 2^8;
//  * whole records (9 d bytes are contiguous) go to a ring of each warp's own in shared memory by the
//    copy engine, an iteration or two ahead; loads into registers left the warps waiting for DRAM two
//    thirds of the time (64 sequences of 1024..32768 tokens, 32/8 heads: 349 us), 16-byte cp.async
//    stopped at 83% of the copy bandwidth and took a tenth of the instructions (277 us);
//  * several independent pages per iteration keep a warp issuing (Q4Shape): 263 us, and with up to four heads to
//    a kv head two of them share a tile of scores: 243 us, 81% of the copy bandwidth (76% with five to eight
//    heads).  What is left is instructions: without its arithmetic the same kernel runs at 95%.
#include <cuda_fp16.h>

#include "decode_mod.cuh"
#include "q4.cuh"

namespace cpattn {
namespace {

CP_DEV void mma16816_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Pairs (j, j + 4), j = 0..3, of a word's codes as an f16x2 operand without any arithmetic: a code in
// the low bits of an f16 is the subnormal n 2^-24 (16 n 2^-24 for the upper nibble of a byte, j odd),
// exact in the MMA.  One logic operation for two values, and one shift for four.
template <int J>
CP_DEV uint32_t codes(uint32_t w) {
  return (J < 2 ? w : w >> 8) & (J % 2 == 0 ? 0x000f000fu : 0x00f000f0u);
}
constexpr float kCodeUnit = 16777216.f;  // 2^24: what a code's subnormal is multiplied by
constexpr long long kBudget = 4000000000ll;  // SM cycles per wait (~2 s)
constexpr float kMaxFactor = 16384.f;    // f16 factors p scale stay below this many units

// floor(log2 x) of a normal x > 0, and 2^e for e within [-126, 127] (the nearer end outside).
CP_DEV int exponent(float x) { return (int)(__float_as_uint(x) >> 23) - 127; }
CP_DEV float pow2(int e) { return __uint_as_float((uint32_t)(min(max(e, -126), 127) + 127) << 23); }

// `bytes` (a multiple of 16) from global to shared memory by the copy engine, completing on an mbarrier.
CP_DEV void bulk_load(uint32_t dst, const uint8_t* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
CP_DEV uint4 lds128(uint32_t a) {
  uint4 x;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(a));
  return x;
}
CP_DEV uint2 lds64(uint32_t a) {
  uint2 x;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "r"(a));
  return x;
}
CP_DEV uint32_t lds32(uint32_t a) {
  uint32_t x;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x) : "r"(a));
  return x;
}

// Tokens and the MMA.  Row r of S^T (r = gid, and gid + 8) is token row_token(r) of the page: K's pieces
// of eight neighbouring lanes then lie in rows of both parities (no bank conflict), and V's rows of one
// load (tid = 0..3) are four neighbours.
CP_DEV int row_token(int r) { return (r >> 1) ^ ((r & 1) * 5); }

// NT: tiles of 8 query heads.  NP: pages per iteration of a warp.  Independent pages next to each other
// are what keeps a warp issuing: four on 12 warps per SM beat two on 16 and one on 16 (d = 128, the batch
// of 64: 263, 277 and 314 us; d = 64: 189, 193).  Two with a second tile of heads (147 against 163 us).
template <int D, int NT>
struct Q4Shape {
  static constexpr int NP = NT == 1 ? 4 : 2;
  static constexpr int kStages = NP == 4 ? 2 : 3;
  static constexpr int kCtas = NT == 1 ? 3 : 2;  // per SM
  static constexpr int kRec = 9 * D;
  static constexpr int kStage = NP * 2 * kRec;              // per warp: [page][K, V]
  static constexpr int kRing = kStages * kWarps * kStage;   // [stage][warp]
  static constexpr int kQRow = 2 * (D / 16) + 4;            // words of q operands per lane, padded
  static constexpr int kQBytes = NT * 32 * kQRow * 4 + 8 * NT * (D / kQ4Group + 1) * 4;
  static constexpr int kParts = (int)sizeof(WarpParts<D, 8 * NT>);
  static constexpr int kBytes = kRing > kParts ? kRing : kParts;
  static_assert(kQBytes <= kWarps * kStage, "the q operands take the last stage before the loop");
};

// PK: pages that share a tile of scores.  With up to four heads a page's scores fill half of a tile's eight
// columns, so the tile's other half takes another page's: Q's heads stand in both halves, of each page's
// product a thread keeps the columns that are its page's, and everything between the products (scales,
// exponentials, factors, transposes) is done once for two pages.  P V takes the halves in turn, the other
// one zero; the halves keep sums of their own, joined at the end.  (The batch of 64, d = 128, 4 heads to a kv
// head: 263 -> 247 us; with a cap and a bias 339 -> 292.)
template <int D, int NT, int PK, bool MOD>
__global__ void __launch_bounds__(kWarps * 32, (Q4Shape<D, NT>::kCtas)) decode_q4_kernel(const ModParams p) {
  using T = __nv_bfloat16;
  using Sh = Q4Shape<D, NT>;
  constexpr int NP = Sh::NP, ST = Sh::kStages, REC = Sh::kRec;
  constexpr int HR = 8 * NT;
  constexpr int GR = D / kQ4Group;
  constexpr int KS = D / 16;  // MMAs of each product
  constexpr int NS = NP / PK;  // score tiles per iteration
  static_assert(PK == 1 || NT == 1, "only a group that fills half a tile shares it");
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(8) unsigned long long s_bar[kWarps][Sh::kStages];  // a stage's records have landed
  WarpParts<D, HR>& parts = *reinterpret_cast<WarpParts<D, HR>*>(smem);  // over the ring, at the end
  Unit u;
  if (!take_unit<T, D, HR>(p, parts, u)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tid = lane & 3;
  const int mine = PK == 2 ? tid >> 1 : 0;  // which of a tile's pages this thread's columns belong to
  const uint32_t ring = sm100::smem_u32(smem) + (uint32_t)(warp * Sh::kStage);
  auto stage_at = [&](int st) -> uint32_t { return ring + (uint32_t)(st * (kWarps * Sh::kStage)); };

  // ---- this warp's iterations: k covers pages pg0 + (k kWarps + warp) NP + i.  Table entries 32 at a
  // time (lane j holds the j-th page's), a batch ahead.
  const int32_t* trow = p.tables + ((long long)u.r * p.B + u.b) * p.max_blocks;
  const int pg0 = u.l0 / kPage, pg1 = (u.l1 + kPage - 1) / kPage;
  const int iters = (pg1 - pg0 - warp * NP + kWarps * NP - 1) / (kWarps * NP);
  auto fetch_ids = [&](int j0) -> int {
    const int j = j0 + lane, pg = pg0 + (j / NP * kWarps + warp) * NP + j % NP;
    int id = -1;
    if (pg < pg1 && pg < p.max_blocks) id = ld(trow + pg);
    return id >= 0 && id < p.pool ? id : -1;
  };
  int ids = fetch_ids(0), ids_next = fetch_ids(32);
  const int page_stride = p.Hkv * REC;  // Hkv <= 65535: below 2^31
  const long long unit_base = (long long)u.r * p.pool * page_stride + (long long)u.g * REC;
  const uint8_t* const kb = p.kc + unit_base;
  const uint8_t* const vb = p.vc + unit_base;
  const uint32_t bars = sm100::smem_u32(&s_bar[warp][0]);
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < ST; ++i) sm100::mbar_init(bars + 8u * i, 1);
    sm100::fence_mbar_init();
  }
  __syncwarp();
  uint32_t there = 0u;  // bit stage * NP + i: the page is in the pool (and is copied)
  auto issue = [&](int k, int st) {
    if (k < iters) {
      if ((k * NP & 31) == 0 && k > 0) {
        ids = ids_next;
        ids_next = fetch_ids(k * NP + 32);
      }
      int id[NP], n = 0;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        id[i] = __shfl_sync(0xffffffffu, ids, (k * NP + i) & 31);
        const uint32_t bit = 1u << (st * NP + i);
        there = id[i] >= 0 ? there | bit : there & ~bit;
        n += id[i] >= 0;
      }
      const uint32_t bar = bars + 8u * (uint32_t)st;
      if (lane == 0) {
        sm100::mbar_expect_tx(bar, (uint32_t)(n * 2 * REC));  // (arrives; 0 bytes when no page is there)
#pragma unroll
        for (int i = 0; i < NP; ++i)
          if (id[i] >= 0) {
            const long long at = (long long)id[i] * page_stride;
            const uint32_t dst = stage_at(st) + (uint32_t)(i * 2 * REC);
            bulk_load(dst, kb + at, REC, bar);
            bulk_load(dst + REC, vb + at, REC, bar);
          }
      }
    }
  };
#pragma unroll
  for (int k = 0; k < ST - 1; ++k) issue(k, k);

  // ---- Q^T as the B operand of S^T = K Q^T, arranged in shared memory by the whole CTA (8 dims, one
  // word of codes, are 4 operand words of one lane).  Codes are f16, so q is too, scaled by a power of
  // two per head to a largest component in [2^8, 2^9): its 8 significant bits stay exact down to
  // 2^-12 of that, with the odd pairs' 1 / 16 in.  Also q's sum over each group, and the factor back.
  uint32_t(*const q_ops)[32][Sh::kQRow] =
      reinterpret_cast<uint32_t(*)[32][Sh::kQRow]>(smem + (ST - 1) * kWarps * Sh::kStage);
  float(*const q_sums)[GR] = reinterpret_cast<float(*)[GR]>(q_ops + NT);
  float* const q_back = &q_sums[HR][0];
  constexpr int TPH = D / 8;  // threads per head
#pragma unroll
  for (int i0 = 0; i0 < HR * TPH; i0 += kWarps * 32) {
    const int i = i0 + (int)threadIdx.x, head = i / TPH, c = i % TPH;
    const int from = PK == 2 ? head & 3 : head;
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (from < p.G)
      x = ld(reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) +
                                               ((long long)u.b * p.Hq + (long long)u.g * p.G + from) * D) + c);
    const float f[8] = {bf16_lo(x.x), bf16_hi(x.x), bf16_lo(x.y), bf16_hi(x.y),
                        bf16_lo(x.z), bf16_hi(x.z), bf16_lo(x.w), bf16_hi(x.w)};
    float mx = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(f[e]));
#pragma unroll
    for (int o = 1; o < TPH; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const int ex = mx > 0.f && isfinite(mx) ? max(exponent(mx) - 8, -100) : 0;
    const float down = pow2(-ex);
    uint32_t h[4];
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {  // pairs (e, e + 4), as codes() brings them
      const float part = e % 2 == 0 ? down : down * 0.0625f;
      const __half2 v = __floats2half2_rn(f[e] * part, f[e + 4] * part);
      h[e] = *reinterpret_cast<const uint32_t*>(&v);
      sum += f[e] * down + f[e + 4] * down;
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (head < HR) {
      *reinterpret_cast<uint4*>(&q_ops[head / 8][(head % 8) * 4 + (c % 8) / 2][(c / 8) * 8 + (c % 2) * 4]) =
          make_uint4(h[0], h[1], h[2], h[3]);
      if (c % 8 == 0) q_sums[head][c / 8] = sum / kCodeUnit;
      if (c == 0) q_back[head] = pow2(ex) * kCodeUnit;
    }
  }
  __syncthreads();
  uint32_t qb[NT][KS][2];
  float qsum[NT][GR][2], qscale[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int w = 0; w < KS / 2; ++w) {
      const uint4 x = *reinterpret_cast<const uint4*>(&q_ops[nt][lane][4 * w]);
      qb[nt][2 * w][0] = x.x, qb[nt][2 * w][1] = x.y, qb[nt][2 * w + 1][0] = x.z, qb[nt][2 * w + 1][1] = x.w;
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int head = 8 * nt + 2 * tid + c;
      qscale[nt][c] = p.scale * kLog2e * q_back[head];
#pragma unroll
      for (int gr = 0; gr < GR; ++gr) qsum[nt][gr][c] = q_sums[head][gr];
    }
  }
  // the ring's last stage is free, and the copy engine writes it next: ordinary stores and loads of shared
  // memory are ordered before its own by a proxy fence of every thread that made them
  sm100::fence_proxy_async_smem();
  __syncthreads();
  const Mods<NT> mods(p, u, PK == 2 ? tid & 1 : tid);

  // Per head of this thread's columns (2 tid, 2 tid + 1): reference m (log2; neg = -m, 0 before the
  // first score; limit: the score past which it moves, in the scores' units) and the sum of this
  // thread's tokens; per group the sum of P minimum (this thread's tokens) and the unit 1 / inv of the
  // f16 factors P scale that o is in (a power of two; 2^-126 before the first one, so that any factor
  // worth keeping moves it).
  float m[NT][2], neg[NT][2], limit[NT][2], l[NT][2], pm[NT][GR][2], inv[NT][GR][2], o[NT][KS][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      m[nt][c] = -INFINITY, neg[nt][c] = 0.f, limit[nt][c] = -INFINITY, l[nt][c] = 0.f;
#pragma unroll
      for (int gr = 0; gr < GR; ++gr) pm[nt][gr][c] = 0.f, inv[nt][gr][c] = 8.507059173023462e37f;  // 2^126
    }
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
  }

  // this thread's places within a record: K pieces of tokens row_token(gid) and 8 on, V pieces of
  // tokens tid, tid ^ 5 and 8 on, scales of tokens row_token(gid) and 8 on
  const int tok = row_token(gid);
  constexpr uint32_t kRow = D / 2;
  uint32_t k_at, v0_at, v1_at;
  if constexpr (D == 128) {
    k_at = (uint32_t)tok * kRow + tid * 16u;
    v0_at = (uint32_t)tid * kRow + gid * 8u;
    v1_at = (uint32_t)(tid ^ 5) * kRow + gid * 8u;
  } else {
    k_at = (uint32_t)tok * kRow + tid * 8u;
    v0_at = (uint32_t)tid * kRow + gid * 4u;
    v1_at = (uint32_t)(tid ^ 5) * kRow + gid * 4u;
  }
  const uint32_t s_at = 8u * D + (uint32_t)tok * (D / 16);
  auto load_scales = [&](uint32_t rec, int h, uint32_t (&w)[GR]) {
    if constexpr (GR == 2) {
      const uint2 x = lds64(rec + s_at + (uint32_t)(h * (D / 2)));
      w[0] = x.x, w[GR - 1] = x.y;
    } else {
      w[0] = lds32(rec + s_at + (uint32_t)(h * (D / 2)));
    }
  };

  bool bad = false;
  int st = 0;           // k mod ST
  uint32_t phase = 0u;  // k / ST mod 2
  for (int k = 0; k < iters; ++k) {
    issue(k + ST - 1, st == 0 ? ST - 1 : st - 1);  // the stage that the last iteration read
    if (!__all_sync(0xffffffffu, sm100::mbar_wait(bars + 8u * (uint32_t)st, phase, nullptr, kBudget))) {
      if (lane == 0) report(p.err, CP_ERR_TIMEOUT);
      // what was issued has another chance to land before the shared memory is given up
      for (int j = k; j < min(k + ST, iters); ++j)
        sm100::mbar_wait(bars + 8u * (uint32_t)(j % ST), (uint32_t)(j / ST) & 1u, nullptr, kBudget);
      break;
    }
    const uint32_t base = stage_at(st);
    const int page0 = pg0 + (k * kWarps + warp) * NP;
    // some token of the iteration's pages is not visible
    const bool edge = (there >> (st * NP) & ((1u << NP) - 1u)) != (1u << NP) - 1u || page0 * kPage < u.a ||
                      (page0 + NP) * kPage > u.l1;
    auto token = [&](int j, int h) { return (page0 + PK * j + mine) * kPage + tok + 8 * h; };
    auto visible = [&](int j, int h) {
      const int t = token(j, h);
      return (there >> (st * NP + PK * j + mine) & 1u) && t >= u.a && t < u.l1;
    };

    // ---- S^T: rows = tokens row_token(gid), 8 on; columns = heads 2 tid, 2 tid + 1 (of page `mine`)
    float s[NS][NT][4];  // [token half * 2 + head], log2 units (MOD) or to be multiplied by qscale
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      float c[PK][NT][GR][4];
#pragma unroll
      for (int i = 0; i < PK; ++i) {
        const uint32_t rec = base + (uint32_t)((PK * j + i) * 2 * REC);
        uint32_t w[2][2 * GR];  // [token half][word]: the groups' words in turn
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if constexpr (D == 128) {
            const uint4 x = lds128(rec + k_at + (uint32_t)h * 8u * kRow);
            w[h][0] = x.x, w[h][1] = x.y, w[h][2 * GR - 2] = x.z, w[h][2 * GR - 1] = x.w;
          } else {
            const uint2 x = lds64(rec + k_at + (uint32_t)h * 8u * kRow);
            w[h][0] = x.x, w[h][1] = x.y;
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int gr = 0; gr < GR; ++gr)
#pragma unroll
            for (int e = 0; e < 4; ++e) c[i][nt][gr][e] = 0.f;
#pragma unroll
        for (int wi = 0; wi < 2; ++wi)
#pragma unroll
          for (int gr = 0; gr < GR; ++gr) {
            const uint32_t w0 = w[0][wi * GR + gr], w1 = w[1][wi * GR + gr];
            const int ks = gr * 4 + wi * 2;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma16816_f16(c[i][nt][gr], codes<0>(w0), codes<0>(w1), codes<1>(w0), codes<1>(w1), qb[nt][ks][0], qb[nt][ks][1]);
              mma16816_f16(c[i][nt][gr], codes<2>(w0), codes<2>(w1), codes<3>(w0), codes<3>(w1), qb[nt][ks + 1][0],
                           qb[nt][ks + 1][1]);
            }
          }
      }
      uint32_t sm[2][GR];
      const uint32_t rec = base + (uint32_t)((PK * j + mine) * 2 * REC);
      load_scales(rec, 0, sm[0]);
      load_scales(rec, 1, sm[1]);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float v = bf16_hi(sm[h][0]) * qsum[nt][0][e];
            v = fmaf(bf16_lo(sm[h][0]), mine == 0 ? c[0][nt][0][2 * h + e] : c[PK - 1][nt][0][2 * h + e], v);
            if constexpr (GR == 2) {
              v = fmaf(bf16_hi(sm[h][GR - 1]), qsum[nt][GR - 1][e], v);
              v = fmaf(bf16_lo(sm[h][GR - 1]), mine == 0 ? c[0][nt][GR - 1][2 * h + e] : c[PK - 1][nt][GR - 1][2 * h + e], v);
            }
            s[j][nt][2 * h + e] = MOD ? v * qscale[nt][e] : v;
          }
      if constexpr (MOD) mods.apply(s[j], p, u, token(j, 0));
    }
    if (edge) {
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        bad |= !(there >> (st * NP + PK * j + mine) & 1u) && (page0 + PK * j + mine) * kPage < u.l1;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (!visible(j, h)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) s[j][nt][2 * h] = s[j][nt][2 * h + 1] = -INFINITY;
          }
      }
    }
    bool grow = false;
    float mx[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        mx[nt][h] = fmaxf(s[0][nt][h], s[0][nt][2 + h]);
#pragma unroll
        for (int i = 1; i < NS; ++i) mx[nt][h] = fmaxf(mx[nt][h], fmaxf(s[i][nt][h], s[i][nt][2 + h]));
        grow |= mx[nt][h] > limit[nt][h];
      }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float before = m[nt][h];
          const float alpha = new_reference(MOD ? mx[nt][h] : mx[nt][h] * qscale[nt][h], m[nt][h], neg[nt][h]);
          limit[nt][h] = MOD ? m[nt][h] + kMaxGrowth : (m[nt][h] + kMaxGrowth) / qscale[nt][h];
          l[nt][h] *= alpha;
          // What o holds shrinks, and its unit with it, so that later factors do not meet a unit set by tokens
          // that no longer count: by whole powers of two of the reference itself, which o in units then leaves
          // where it was to a factor of 2 however often the reference moves.  (alpha 0: nothing is left in o.)
          const int down = alpha == 0.f ? 256 : m[nt][h] == before ? 0 : (int)(floorf(m[nt][h]) - floorf(before));
#pragma unroll
          for (int gr = 0; gr < GR; ++gr) {
            pm[nt][gr][h] *= alpha;
            const int e = min(down, 126 - exponent(inv[nt][gr][h]));
            const float keep = alpha * pow2(e);
            inv[nt][gr][h] = pow2(exponent(inv[nt][gr][h]) + e);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              o[nt][gr * 4 + j][h] *= keep;
              o[nt][gr * 4 + j][2 + h] *= keep;
            }
          }
        }
    }

    // ---- P in place of the scores; its sums, and those of P minimum, keep 32 bits.  P scale goes to
    // the tensor cores as f16 (11 bits, the codes' type) in units that keep it below kMaxFactor.
    uint32_t vs[NS][2][GR];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const uint32_t rec = base + (uint32_t)(((PK * i + mine) * 2 + 1) * REC);
      load_scales(rec, 0, vs[i][0]);
      load_scales(rec, 1, vs[i][1]);
    }
    if (edge) {  // scales of masked rows may be anything: 0
#pragma unroll
      for (int i = 0; i < NS; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int gr = 0; gr < GR; ++gr) vs[i][h][gr] = visible(i, h) ? vs[i][h][gr] : 0u;
    }
#pragma unroll
    for (int i = 0; i < NS; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          s[i][nt][e] = sm100::ex2(fmaf(s[i][nt][e], MOD ? 1.f : qscale[nt][e & 1], neg[nt][e & 1]));
        l[nt][0] += s[i][nt][0] + s[i][nt][2];
        l[nt][1] += s[i][nt][1] + s[i][nt][3];
#pragma unroll
        for (int gr = 0; gr < GR; ++gr)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float mn = bf16_hi(vs[i][h][gr]);
            pm[nt][gr][0] = fmaf(s[i][nt][2 * h], mn, pm[nt][gr][0]);
            pm[nt][gr][1] = fmaf(s[i][nt][2 * h + 1], mn, pm[nt][gr][1]);
          }
      }
    uint32_t pb[NS][NT][GR][2];
    auto factors = [&]() -> bool {  // true: one is too large for its unit
      __half2 top = __float2half2_rn(0.f);
#pragma unroll
      for (int i = 0; i < NS; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int gr = 0; gr < GR; ++gr)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float sc = bf16_lo(vs[i][h][gr]);
              const __half2 f = __floats2half2_rn(s[i][nt][2 * h] * sc * inv[nt][gr][0],
                                                  s[i][nt][2 * h + 1] * sc * inv[nt][gr][1]);
              top = __hmax2(top, f);
              pb[i][nt][gr][h] = *reinterpret_cast<const uint32_t*>(&f);
            }
      return !__hble2(top, __float2half2_rn(kMaxFactor));
    };
    if (__any_sync(0xffffffffu, factors())) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int gr = 0; gr < GR; ++gr)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float f = 0.f;
#pragma unroll
            for (int i = 0; i < NS; ++i)
#pragma unroll
              for (int h = 0; h < 2; ++h) f = fmaxf(f, s[i][nt][2 * h + c] * bf16_lo(vs[i][h][gr]));
            f = fmaxf(f, __shfl_xor_sync(0xffffffffu, f, 4));
            f = fmaxf(f, __shfl_xor_sync(0xffffffffu, f, 8));
            f = fmaxf(f, __shfl_xor_sync(0xffffffffu, f, 16));
            if (f * inv[nt][gr][c] > kMaxFactor) {  // the largest factor becomes at most 1 unit
              const float unit = pow2(-1 - exponent(f));
              const float alpha = pow2(exponent(unit) - exponent(inv[nt][gr][c]));
              inv[nt][gr][c] = unit;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                o[nt][gr * 4 + j][c] *= alpha;
                o[nt][gr * 4 + j][2 + c] *= alpha;
              }
            }
          }
      factors();
    }

    // ---- O^T: rows = dims 8 gid + j and 8 gid + 4 + j of the group, columns = heads (of the pages' halves)
#pragma unroll
    for (int j = 0; j < NS; ++j) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int gr = 0; gr < GR; ++gr)
#pragma unroll
          for (int h = 0; h < 2; ++h) pb[j][nt][gr][h] = transpose8x8(pb[j][nt][gr][h]);
#pragma unroll
      for (int i = 0; i < PK; ++i) {
        const uint32_t rec = base + (uint32_t)(((PK * j + i) * 2 + 1) * REC);
        const bool on = PK == 1 || (gid >> 2) == i;
        uint32_t x[4][GR];  // tokens tid, tid ^ 5, and 8 on
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint32_t at = rec + (t & 1 ? v1_at : v0_at) + (uint32_t)(t >> 1) * 8u * kRow;
          if constexpr (GR == 2) {
            const uint2 y = lds64(at);
            x[t][0] = y.x, x[t][GR - 1] = y.y;
          } else {
            x[t][0] = lds32(at);
          }
        }
#pragma unroll
        for (int gr = 0; gr < GR; ++gr) {
          const uint32_t ab0 = low_halves(x[0][gr], x[1][gr]), ab1 = high_halves(x[0][gr], x[1][gr]);
          const uint32_t cd0 = low_halves(x[2][gr], x[3][gr]), cd1 = high_halves(x[2][gr], x[3][gr]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float(&op)[KS][4] = o[nt];
            const uint32_t b0 = on ? pb[j][nt][gr][0] : 0u, b1 = on ? pb[j][nt][gr][1] : 0u;
            mma16816_f16(op[gr * 4 + 0], codes<0>(ab0), codes<0>(ab1), codes<0>(cd0), codes<0>(cd1), b0, b1);
            mma16816_f16(op[gr * 4 + 1], codes<1>(ab0), codes<1>(ab1), codes<1>(cd0), codes<1>(cd1), b0, b1);
            mma16816_f16(op[gr * 4 + 2], codes<2>(ab0), codes<2>(ab1), codes<2>(cd0), codes<2>(cd1), b0, b1);
            mma16816_f16(op[gr * 4 + 3], codes<3>(ab0), codes<3>(ab1), codes<3>(cd0), codes<3>(cd1), b0, b1);
          }
        }
      }
    }
    __syncwarp();  // every lane has read the stage
    st = st + 1 == ST ? 0 : st + 1;
    if (st == 0) phase ^= 1u;
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) report(p.err, CP_ERR_DEVICE_BOUNDS);

  // ---- this warp's part: sums over the lanes that share a column, output rows per head; two pages' halves
  // of a tile (columns 4 apart, in lanes tid ^ 2) become one
  __syncthreads();  // every copy has landed and been read: the ring is free
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float sum = column_sum(l[nt][h]), ref = m[nt][h], keep = 1.f, add = 0.f;
      if constexpr (PK == 2) {
        const float m2 = __shfl_xor_sync(0xffffffffu, ref, 2), l2 = __shfl_xor_sync(0xffffffffu, sum, 2);
        ref = fmaxf(m[nt][h], m2);
        // (a reference of -inf: no finite score, sums of 0 or NaN)
        keep = m[nt][h] == ref || m[nt][h] == -INFINITY ? 1.f : exp2f(m[nt][h] - ref);
        add = m2 == ref || m2 == -INFINITY ? 1.f : exp2f(m2 - ref);
        sum = sum * keep + l2 * add;
      }
      const int head = 8 * nt + 2 * tid + h;
      const bool write = PK == 1 || mine == 0;
      if (gid == 0 && write) {
        parts.m[warp][head] = ref;
        parts.l[warp][head] = sum;
      }
#pragma unroll
      for (int gr = 0; gr < GR; ++gr) {  // MMA j: codes j and j + 4 of word gid, times 16 for j odd
        const float y = column_sum(pm[nt][gr][h]), unit = pow2(-exponent(inv[nt][gr][h]));
        auto val = [&](int j, int e) {
          const float x = fmaf(o[nt][gr * 4 + j][e] * (j % 2 == 0 ? kCodeUnit : kCodeUnit / 16.f), unit, y);
          return PK == 1 ? x : x * keep + __shfl_xor_sync(0xffffffffu, x, 2) * add;
        };
        const float4 a = make_float4(val(0, h), val(1, h), val(2, h), val(3, h));
        const float4 b = make_float4(val(0, 2 + h), val(1, 2 + h), val(2, 2 + h), val(3, 2 + h));
        if (write) {
          float4* const at = reinterpret_cast<float4*>(&parts.o[warp][head][64 * gr + 8 * gid]);
          at[0] = a;
          at[1] = b;
        }
      }
    }
  finish<T, D, HR>(p, parts, u.b, u.g, u.part, u.live);
}

template <int D, int NT, int PK>
cudaError_t launch_q4(const ModParams& p, bool mod, cudaStream_t s) {
  auto kern = mod ? decode_q4_kernel<D, NT, PK, true> : decode_q4_kernel<D, NT, PK, false>;
  constexpr int bytes = Q4Shape<D, NT>::kBytes;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  return e == cudaSuccess ? launch_decode(kern, p, bytes, Q4Shape<D, NT>::kCtas, s) : e;
}
template <int D>
cudaError_t launch_d(const ModParams& p, bool mod, cudaStream_t s) {
  if (p.G <= 4) return launch_q4<D, 1, 2>(p, mod, s);
  return p.G <= 8 ? launch_q4<D, 1, 1>(p, mod, s) : launch_q4<D, 2, 1>(p, mod, s);
}

}  // namespace
}  // namespace cpattn

cudaError_t cp_launch_decode_q4(const cp_decode_args& a, const cp_score_mod& mod, float scale,
                                const CpDecodeWorkspace* ws, void* out, float* out_lse, cudaStream_t s) {
  using namespace cpattn;
  const ModParams p = decode_mod_params(a, mod, scale, ws, out, out_lse);
  const bool m = changes_scores(mod);
  return a.head_dim == 64 ? launch_d<64>(p, m, s) : launch_d<128>(p, m, s);
}
