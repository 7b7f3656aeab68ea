// What the tcgen05 prefill kernels do with the rows of a tile (internal): the softmax of a thread's row of scores
// in TMEM, the rescaling of its output row, and the rows' way out through shared memory.
#pragma once

#include "common.cuh"
#include "sm100.cuh"

namespace cpattn {
namespace {

using namespace sm100;

constexpr int BM = 128;          // query rows per tile (TMEM lanes)
constexpr int BN = 128;          // keys per tile
constexpr float kRescaleThreshold = 8.f;     // log2 units

CP_DEV uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

CP_DEV void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}

// A warp's 32 staged rows (the boxes stage_rows_* wrote at sb) written out one row per store
// instruction: lane l carries columns [E l, E l + E), E = d / 32, so each warp-wide store covers
// a whole contiguous output row.  dst: row 0 of the warp; consecutive rows are `stride` elements
// apart.
template <int D>
CP_DEV void store_staged_f32(uint32_t sb, int lane, float* dst, long long stride) {
  constexpr int E = D / 32;
  const int col = E * lane, cin = col % 32;
  const uint32_t a0 = sb + (uint32_t)((col / 32) * 4096 + (cin % 4) * 4);
  const int chunk = cin / 4;
#pragma unroll 8
  for (int r = 0; r < 32; ++r) {
    const uint32_t a = a0 + (uint32_t)(r * 128) + ((uint32_t)(chunk ^ (r & 7)) << 4);
    float* g = dst + r * stride + col;
    if constexpr (E == 4) {
      float4 v;
      asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
      *reinterpret_cast<float4*>(g) = v;
    } else {
      float2 v;
      asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a));
      *reinterpret_cast<float2*>(g) = v;
    }
  }
}
template <int D>
CP_DEV void store_staged_bf16(uint32_t sb, int lane, __nv_bfloat16* dst, long long stride) {
  constexpr int E = D / 32;
  const int col = E * lane, cin = col % 64;
  const uint32_t a0 = sb + (uint32_t)((col / 64) * 4096 + (cin % 8) * 2);
  const int chunk = cin / 8;
#pragma unroll 8
  for (int r = 0; r < 32; ++r) {
    const uint32_t a = a0 + (uint32_t)(r * 128) + ((uint32_t)(chunk ^ (r & 7)) << 4);
    __nv_bfloat16* g = dst + r * stride + col;
    if constexpr (E == 4) {
      uint2 v;
      asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
      *reinterpret_cast<uint2*>(g) = v;
    } else {
      uint32_t v;
      asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
      *reinterpret_cast<uint32_t*>(g) = v;
    }
  }
}

// ---------------------------------------------------------------------------------- row softmax
// Packed two-lane fp32 arithmetic (f32x2 instructions of the sm_100 family) and 3-input max.
CP_DEV uint64_t f2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
CP_DEV void f2u(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
CP_DEV uint64_t ffma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
CP_DEV uint64_t fadd2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
CP_DEV float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The 128 scores of this thread's row (its TMEM lane), one TMEM round trip.
CP_DEV void load_row(uint32_t tS, float (&v0)[32], float (&v1)[32], float (&v2)[32],
                     float (&v3)[32]) {
  tmem_ld32(tS, v0);
  tmem_ld32(tS + 32, v1);
  tmem_ld32(tS + 64, v2);
  tmem_ld32(tS + 96, v3);
  tmem_wait_ld(v0);
  tmem_wait_ld(v1);
  tmem_wait_ld(v2);
  tmem_wait_ld(v3);
}

// Four independent packed partial sums keep the additions off one serial dependency chain.
CP_DEV void exp_chunk(float (&a)[32], uint64_t sc2, uint64_t n2, uint64_t& sum2) {
  uint64_t acc[4] = {f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
  for (int k = 0; k < 32; k += 2) {
    float x0, x1;
    f2u(ffma2(f2(a[k], a[k + 1]), sc2, n2), x0, x1);
    a[k] = ex2(x0);
    a[k + 1] = ex2(x1);
    acc[(k >> 1) & 3] = fadd2(acc[(k >> 1) & 3], f2(a[k], a[k + 1]));
  }
  sum2 = fadd2(sum2, fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3])));
}

// Row max of four 32-column chunks with four independent accumulators.
CP_DEV float max4x32(const float (&v0)[32], const float (&v1)[32], const float (&v2)[32],
                     const float (&v3)[32]) {
  float m0 = -INFINITY, m1 = -INFINITY, m2 = -INFINITY, m3 = -INFINITY;
#pragma unroll
  for (int k = 0; k < 32; k += 2) {
    m0 = fmax3(m0, v0[k], v0[k + 1]);
    m1 = fmax3(m1, v1[k], v1[k + 1]);
    m2 = fmax3(m2, v2[k], v2[k + 1]);
    m3 = fmax3(m3, v3[k], v3[k + 1]);
  }
  return fmaxf(fmaxf(m0, m1), fmaxf(m2, m3));
}

// Online-softmax step of one row over a 128-key tile: columns > lim are masked (skipped when
// every row of the warp sees the whole tile), the running max m (log2 units) moves only when
// the tile max exceeds it by more than 2^8, and the scores become p = 2^(s*sc - m) in place.
// Returns alpha, the factor the row's O accumulator must be scaled by (l is updated here).
CP_DEV float row_softmax(float (&v0)[32], float (&v1)[32], float (&v2)[32], float (&v3)[32],
                         int lim, float sc, float& m, float& l) {
  if (!__all_sync(0xffffffffu, lim >= BN - 1)) {
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      v0[k] = k <= lim ? v0[k] : -INFINITY;
      v1[k] = k + 32 <= lim ? v1[k] : -INFINITY;
      v2[k] = k + 64 <= lim ? v2[k] : -INFINITY;
      v3[k] = k + 96 <= lim ? v3[k] : -INFINITY;
    }
  }
  const float m_tile = max4x32(v0, v1, v2, v3) * sc;
  float alpha = 1.f;
  if (m_tile > m + kRescaleThreshold) {  // first visible tile, or the max grew a lot
    alpha = ex2(m - m_tile);
    m = m_tile;
  }
  const float neg = (m == -INFINITY) ? 0.f : -m;
  const uint64_t sc2 = f2(sc, sc), n2 = f2(neg, neg);
  uint64_t sum2 = f2(0.f, 0.f);
  exp_chunk(v0, sc2, n2, sum2);
  exp_chunk(v1, sc2, n2, sum2);
  exp_chunk(v2, sc2, n2, sum2);
  exp_chunk(v3, sc2, n2, sum2);
  float s_lo, s_hi;
  f2u(sum2, s_lo, s_hi);
  l = l * alpha + (s_lo + s_hi);
  return alpha;
}

// Split form of row_softmax for kernels whose P buffer is already free when the scores
// arrive: mask + max + running-max update first (returns alpha) ...
CP_DEV float row_max_update(float (&v0)[32], float (&v1)[32], float (&v2)[32], float (&v3)[32],
                            int lim, float sc, float& m) {
  if (!__all_sync(0xffffffffu, lim >= BN - 1)) {
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      v0[k] = k <= lim ? v0[k] : -INFINITY;
      v1[k] = k + 32 <= lim ? v1[k] : -INFINITY;
      v2[k] = k + 64 <= lim ? v2[k] : -INFINITY;
      v3[k] = k + 96 <= lim ? v3[k] : -INFINITY;
    }
  }
  const float m_tile = max4x32(v0, v1, v2, v3) * sc;
  float alpha = 1.f;
  if (m_tile > m + kRescaleThreshold) {
    alpha = ex2(m - m_tile);
    m = m_tile;
  }
  return alpha;
}

// Exponentials of a row packed as bf16 pairs into the first 64 columns of its S buffer in TMEM
// (the A operand of a tensor-memory PV MMA), 16 columns per store; returns the row sum of p.
CP_DEV void exp_pack_tmem(float (&a)[32], uint64_t sc2, uint64_t n2, uint64_t& sum2, uint32_t taddr) {
  exp_chunk(a, sc2, n2, sum2);
  uint32_t pk[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) pk[k] = pack_bf16(a[2 * k], a[2 * k + 1]);
  tmem_st16(taddr, pk);
}
CP_DEV float row_exp_tmem(float (&v0)[32], float (&v1)[32], float (&v2)[32], float (&v3)[32],
                          float sc, float m, uint32_t tS) {
  const float neg = (m == -INFINITY) ? 0.f : -m;
  const uint64_t sc2 = f2(sc, sc), n2 = f2(neg, neg);
  uint64_t sum2 = f2(0.f, 0.f);
  exp_pack_tmem(v0, sc2, n2, sum2, tS);
  exp_pack_tmem(v1, sc2, n2, sum2, tS + 16);
  exp_pack_tmem(v2, sc2, n2, sum2, tS + 32);
  exp_pack_tmem(v3, sc2, n2, sum2, tS + 48);
  tmem_wait_st();
  float lo, hi;
  f2u(sum2, lo, hi);
  return lo + hi;
}

// P row (bf16) into a 128x128 P tile stored as two 64-column blocks in the 128-byte-swizzled
// K-major layout the MMA reads: 16-byte chunk c of row r sits at chunk c ^ (r % 8).
CP_DEV void store_p_row(uint32_t sP, int row, const float (&v0)[32], const float (&v1)[32],
                        const float (&v2)[32], const float (&v3)[32]) {
  const uint32_t prow = sP + row * 128;
  const uint32_t sw = (uint32_t)(row & 7);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const float* a = c == 0 ? v0 : c == 1 ? v1 : c == 2 ? v2 : v3;
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const int col = c * 32 + h * 8;
      const uint32_t blk = (uint32_t)(col / 64), ch = (uint32_t)((col % 64) / 8);
      st_shared_v4(prow + blk * (BM * 128) + ((ch ^ sw) << 4), pack_bf16(a[h * 8], a[h * 8 + 1]),
                   pack_bf16(a[h * 8 + 2], a[h * 8 + 3]), pack_bf16(a[h * 8 + 4], a[h * 8 + 5]),
                   pack_bf16(a[h * 8 + 6], a[h * 8 + 7]));
    }
  }
}

// O row *= alpha in TMEM (warp-collective; nothing to do when no lane of the warp needs it).
template <int D>
CP_DEV void rescale_o(uint32_t tO, float alpha) {
  if (!__any_sync(0xffffffffu, alpha != 1.f)) return;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    float o[32];
    tmem_ld32(tO + c * 32, o);
    tmem_wait_ld(o);
#pragma unroll
    for (int k = 0; k < 32; ++k) o[k] *= alpha;
    tmem_st32(tO + c * 32, o);
  }
  tmem_wait_st();
}

// Final O row / l -> the partial output (f32) and its natural-log LSE (warp-collective).
template <int D>
CP_DEV void write_row(uint32_t tO, float m, float l, bool row_valid, float* dst, float* lse_dst) {
  const float inv_l = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    float o[32];
    tmem_ld32(tO + c * 32, o);
    tmem_wait_ld(o);
    if (row_valid && l > 0.f) {
#pragma unroll
      for (int k = 0; k < 32; k += 4)
        *reinterpret_cast<float4*>(dst + c * 32 + k) =
            make_float4(o[k] * inv_l, o[k + 1] * inv_l, o[k + 2] * inv_l, o[k + 3] * inv_l);
    }
  }
  if (row_valid) *lse_dst = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

// Final O row / l -> bf16 output (round to nearest even) and its LSE (warp-collective).
template <int D>
CP_DEV void write_row_bf16(uint32_t tO, float m, float l, bool row_valid, __nv_bfloat16* dst,
                           float* lse_dst) {
  const float inv_l = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    float o[32];
    tmem_ld32(tO + c * 32, o);
    tmem_wait_ld(o);
    if (row_valid) {
#pragma unroll
      for (int k = 0; k < 32; k += 8)
        *reinterpret_cast<uint4*>(dst + c * 32 + k) = make_uint4(
            pack_bf16(o[k] * inv_l, o[k + 1] * inv_l), pack_bf16(o[k + 2] * inv_l, o[k + 3] * inv_l),
            pack_bf16(o[k + 4] * inv_l, o[k + 5] * inv_l), pack_bf16(o[k + 6] * inv_l, o[k + 7] * inv_l));
    }
  }
  if (row_valid) *lse_dst = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

// Final O rows of one warp (its 32 TMEM lanes = 32 query rows, scaled by 1/l) staged in shared
// memory as 128-byte-swizzled boxes: f32 boxes of 32 columns x 32 rows (4 KB each, 16-byte chunk
// j of row r at chunk j ^ (r % 8)), or bf16 boxes of 64 columns.  A thread writes its own row,
// store_staged_* read them back a row per warp instruction; the swizzle keeps both directions
// free of bank conflicts.
template <int D>
CP_DEV void stage_rows_f32(uint32_t tO, float inv_l, uint32_t sbase, int lane) {
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    float o[32];
    tmem_ld32(tO + c * 32, o);
    tmem_wait_ld(o);
    const uint32_t rb = sbase + (uint32_t)(c * 4096 + lane * 128);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      st_shared_v4(rb + ((uint32_t)(j ^ (lane & 7)) << 4), __float_as_uint(o[4 * j] * inv_l),
                   __float_as_uint(o[4 * j + 1] * inv_l), __float_as_uint(o[4 * j + 2] * inv_l),
                   __float_as_uint(o[4 * j + 3] * inv_l));
  }
}
template <int D>
CP_DEV void stage_rows_bf16(uint32_t tO, float inv_l, uint32_t sbase, int lane) {
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    float o[32];
    tmem_ld32(tO + c * 32, o);
    tmem_wait_ld(o);
    const uint32_t rb = sbase + (uint32_t)((c >> 1) * 4096 + lane * 128);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      st_shared_v4(rb + ((uint32_t)(((c & 1) * 4 + j) ^ (lane & 7)) << 4),
                   pack_bf16(o[8 * j] * inv_l, o[8 * j + 1] * inv_l),
                   pack_bf16(o[8 * j + 2] * inv_l, o[8 * j + 3] * inv_l),
                   pack_bf16(o[8 * j + 4] * inv_l, o[8 * j + 5] * inv_l),
                   pack_bf16(o[8 * j + 6] * inv_l, o[8 * j + 7] * inv_l));
  }
}

}  // namespace
}  // namespace cpattn
