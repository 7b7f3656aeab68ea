// Prefill attention with modified scores (cp_attn_prefill_mod) on the 5th-generation tensor cores:
// bf16 in, f32 accumulate, contiguous K / V.
//
// "Add utility functions to enable pass-kv prefill and allgather decode" (vLLM PR 26059),
// Purpose: pass-KV prefill and the combination of a Q row's partials (folded in: no partials).
//
//   s_ij = scale q_i.k_j;  s_ij = cap tanh(s_ij / cap);  s_ij -= slope |i - j|   (each optional)
//   out_i = softmax over the keys j in [lo_i, hi_i) of s_ij, times V
//
// One CTA works on two "tiles" of 128 query rows that share every K / V tile of 128 keys: two
// query heads of a kv group (even group), or two consecutive row tiles of one head.  Warps:
//   0     TMA producer: both Q tiles once, then K and V tiles through a 4-slot ring
//   1     TMEM owner and MMA issuer (one thread): S = Q K^T into the tile's TMEM columns, then
//         O += P V with P read from TMEM; order PV0(t) | QK0(t+1) | PV1(t) | QK1(t+1), so a tile's
//         softmax overlaps the other tile's two MMAs
//   2-3   V guards: in a key tile that some row sees only in part they clear what must not reach
//         the MMA (0 times an infinity is NaN), see below
//   4-19  four softmax warpgroups, two per tile: a thread owns half of a query row's 128 scores
// The keys a CTA walks are the union [key_lo, key_hi) of its rows' ranges, so windows and short
// documents load their own keys only; tiles start at key_lo, not at a multiple of 128.
//
// Bound: the chain of a tile's softmax, PV and next QK (3.3k cycles a key tile, 3.7k with a cap, against
// the tensor pipe's 2.05k), so everything on it is kept short: four softmax warpgroups rather than
// two, PV started by halves of P, and the cap a polynomial on the packed fp32 pipe wherever a warp's
// scores allow it (tanh(y) / y in y^2, own least-maximum fits), only else 1 - 2 / (1 + e^2y), two
// special-function operations per score.  8192 tokens, 16/2 heads, d = 128, in the calls' device time: 236 us with
// cap 50 (61% of the measured bf16 peak), 314 with cap 5 and 401 with cap 1 (scores past the polynomials' range),
// 205 without, 220 with a distance bias, 305 with both; 16384 tokens in a window of 4096 with cap 30: 421.
#include <cuda.h>

#include "common.cuh"
#include "guard.cuh"
#include "sm100.cuh"

namespace cpattn {
namespace {

using namespace sm100;

constexpr int BM = 128;  // query rows per tile (TMEM lanes)
constexpr int BN = 128;  // keys per tile
constexpr int BH = BN / 2;  // scores of a row per softmax thread
constexpr int kThreads = 640;
constexpr int kSlots = 4;                    // K / V ring
constexpr long long kBudget = 4000000000ll;  // SM cycles per wait (~2 s)
constexpr float kMaxGrowth = 8.f;            // log2 units the scores may exceed the running reference

struct PrefillModParams {
  int Hq, Hkv, G, Nq, Nkv, window, tiles;  // Nq, Nkv: rows; tiles: row tiles (items) of the longest sequence
  float scale_log2, softcap, cap_in;  // cap_in = scale / cap: y = cap_in q.k
  const int32_t* cu_q;
  const int32_t* cu_kv;  // null: the query rows
  const int32_t* kv_start;
  const int32_t* prefix;
  const float* slopes;
  const __nv_bfloat16* v;  // for the rows of a tile that held infinities or NaN
  __nv_bfloat16* out;
  float* lse;
  int32_t* err;
};

template <int D>
struct Smem {
  static constexpr int kQ = BM * D * 2;
  static constexpr int kKV = BN * D * 2;
  static constexpr int oQ = 0;
  static constexpr int oKV = 2 * kQ;
  static constexpr int oBar = oKV + kSlots * kKV;
  static constexpr int bQ = 0, bFull = 1, bEmpty = bFull + kSlots, bS = bEmpty + kSlots, bP = bS + 2,
                       bO = bP + 4, bFix = bO + 2, bDone = bFix + 2, nBar = bDone + 1;
  static constexpr int oMisc = oBar + nBar * 8;  // TMEM base, abort flag, first / last unclean tile
  static constexpr int kBytes = oMisc + 16;
  // the base is rounded up to the 1 KB swizzle atom; never below 120 KB, so that one CTA (and its
  // 512 TMEM columns) has an SM to itself
  static constexpr int kAlloc = (kBytes + 1024) > 120 * 1024 ? (kBytes + 1024) : 120 * 1024;
  static_assert(kAlloc <= 232448, "dynamic shared memory beyond the 227 KB per-CTA limit");
};

// ------------------------------------------------------------------------------ packed fp32
CP_DEV uint64_t f2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
CP_DEV void f2u(uint64_t v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
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
CP_DEV uint64_t fmul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
CP_DEV float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
CP_DEV uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// A thread's 64 scores: two chunks of 32 TMEM columns.
constexpr int kChunks = BH / 32;
struct Row {
  float c[kChunks][32];
};
CP_DEV float chunk_max(const float (&a)[32]) {
  float m[2] = {-INFINITY, -INFINITY};
#pragma unroll
  for (int k = 0; k < 32; k += 4)
#pragma unroll
    for (int i = 0; i < 2; ++i) m[i] = fmax3(m[i], a[k + 2 * i], a[k + 2 * i + 1]);
  return fmaxf(m[0], m[1]);
}
CP_DEV float row_abs_max(const Row& v) {
  float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int k = 0; k < 32; k += 4)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      m[i] = fmaxf(fmaxf(m[i], fabsf(v.c[i >> 1][k + 2 * (i & 1)])), fabsf(v.c[i >> 1][k + 2 * (i & 1) + 1]));
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// The lowest n of 64 bits (none for n <= 0, all for n >= 64).
CP_DEV uint64_t first_bits(int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull; }

// cap tanh(y) in log2 units from y = cap_in * (q.k): polynomials of tanh(y) / y in y^2 for |y| <= kCapNear and
// kCapFar (relative errors 5.5e-7 and 6.3e-7, least-maximum fits to tanh), beyond 1 - 2 / (1 + e^2y) (absolute
// error about 2^-22 of the cap).  y_max: the row's largest |cap_in s|.
//
// In a tile that all 32 rows see (`whole`) the warp's largest score chooses the form for all of them, but for large
// caps, whose 2^-22 a small score would feel.  In one that some see in part, each score takes the form that its own
// size asks for: keys that a row does not see can then only make it wait for both.
constexpr float kCapNear = 0.5f, kCapFar = 1.25f;
constexpr float kCapSmall = 128.f;  // log2 units: 2^-22 of it is below the rounding of the products' sums
template <int N, typename Put>
CP_DEV void cap_poly(const Row& v, float cap_in, float cap_log2, const float (&a)[N + 1], Put put) {
  const uint64_t in2 = f2(cap_in, cap_in);
  uint64_t c[N + 1];
#pragma unroll
  for (int i = 0; i <= N; ++i) c[i] = f2(a[i] * cap_log2, a[i] * cap_log2);
#pragma unroll
  for (int i = 0; i < kChunks; ++i)
#pragma unroll
    for (int k = 0; k < 32; k += 2) {
      const uint64_t y = fmul2(f2(v.c[i][k], v.c[i][k + 1]), in2), u = fmul2(y, y);
      uint64_t r = c[N];
#pragma unroll
      for (int j = N - 1; j >= 0; --j) r = ffma2(r, u, c[j]);
      put(i, k, y, fmul2(r, y));
    }
}
CP_DEV void cap_scores(Row& v, float cap_in, float cap_log2, float y_max, bool whole) {
  const float near[4] = {0.999999463558197f, -0.33326318860054016f, 0.13190296292304993f, -0.04440222680568695f};
  const float mid[7] = {0.9999994039535522f, -0.3332934081554413f, 0.1329064816236496f, -0.052205443382263184f,
                        0.018229125067591667f, -0.004626906011253595f, 0.0005844940315000713f};
  auto far = [&](float y) { return cap_log2 - __fdividef(2.f * cap_log2, 1.f + ex2(y * (2.f * kLog2e))); };
  auto put = [&](int i, int k, uint64_t, uint64_t x) { f2u(x, v.c[i][k], v.c[i][k + 1]); };
  if (whole && __all_sync(0xffffffffu, y_max <= kCapNear)) {
    cap_poly<3>(v, cap_in, cap_log2, near, put);
  } else if (__all_sync(0xffffffffu, y_max <= kCapFar)) {
    cap_poly<6>(v, cap_in, cap_log2, mid, put);
  } else if (whole && cap_log2 <= kCapSmall) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
#pragma unroll
      for (int k = 0; k < 32; ++k) v.c[i][k] = far(v.c[i][k] * cap_in);
  } else {
    cap_poly<6>(v, cap_in, cap_log2, mid, [&](int i, int k, uint64_t y, uint64_t x) {
      float y0, y1, x0, x1;
      f2u(y, y0, y1);
      f2u(x, x0, x1);
      v.c[i][k] = fabsf(y0) <= kCapFar ? x0 : far(y0);  // (NaN: far, and NaN)
      v.c[i][k + 1] = fabsf(y1) <= kCapFar ? x1 : far(y1);
    });
  }
}

// A capped score is bounded, |x| <= min(|y|, 1) cap log2(e).  Where that says that none of a row's tile can exceed
// the row's reference by more than the growth that every reference is allowed, which both halves of the row ask at
// one barrier, the row's maximum need not be known; and if all lie in the near form's range, P follows from the
// score in one chain, the polynomial's packed FMAs under the exponentials' special-function time.
// The folded coefficients, up to scale (scale / cap)^6, and s^2, up to (cap / 2 scale)^2, stay normal numbers.
inline bool cap_folds(float scale, float softcap) {
  const double y = (double)scale / softcap, c = scale * y * y * y * y * y * y;
  return y >= 1e-5 && c >= 1e-30 && c <= 1e30;
}

struct CapCoefficients {
  // x = s (c0 + u (c1 + u (c2 + u c3))), u = s^2, for |cap_in s| <= kCapNear (relative error 5.5e-7)
  uint64_t c[4];
};
CP_DEV CapCoefficients cap_coefficients(float cap_in, float scale_log2) {
  const float a[4] = {0.999999463558197f, -0.33326318860054016f, 0.13190296292304993f, -0.04440222680568695f};
  CapCoefficients r;
  float k = scale_log2;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.c[i] = f2(a[i] * k, a[i] * k);
    k *= cap_in * cap_in;
  }
  return r;
}
// P = 2^(x - ref) of 32 columns, packed as bf16 pairs over the row's own S columns in TMEM (the A
// operand of the PV MMA; bf16 is the tensor core's operand type), the sum kept in fp32.
// exponent(s): x - ref of a pair of columns, whose scores are s, in order.
template <typename Exponent>
CP_DEV float exp_columns(const float (&a)[32], uint32_t taddr, Exponent exponent) {
  uint64_t acc[4] = {f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f)};
  uint32_t pk[16];
#pragma unroll
  for (int k = 0; k < 32; k += 2) {
    float x, y;
    f2u(exponent(f2(a[k], a[k + 1])), x, y);
    x = ex2(x);
    y = ex2(y);
    acc[(k >> 1) & 3] = fadd2(acc[(k >> 1) & 3], f2(x, y));
    pk[k >> 1] = pack_bf16(x, y);
  }
  tmem_st16(taddr, pk);
  float lo, hi;
  f2u(fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3])), lo, hi);
  return lo + hi;
}

// A distance bias that is linear over a chunk (every key at or before the query) goes into the
// exponent's FMA, and the reference takes the bound max(s) + bias at the chunk's last key, at most 31
// slopes above its largest score: with slopes (log2 units) up to kMaxFold / 31 no P that matters is
// lost, since fp32 and bf16 hold 2^-126.  Steeper slopes are added to the scores first.
constexpr float kMaxFold = 40.f;

// 8 TMEM columns of this lane's row to registers (complete on return), and back.
CP_DEV void tmem_ld8(uint32_t taddr, float (&v)[8]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3]), "=&r"(r[4]), "=&r"(r[5]), "=&r"(r[6]), "=&r"(r[7])
      : "r"(taddr)
      : "memory");
}
CP_DEV void tmem_st8(uint32_t taddr, const float (&v)[8]) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// COLS columns of an O row *= alpha in TMEM (nothing to do when no lane of the warp needs it).
template <int COLS>
CP_DEV void rescale_o(uint32_t tO, float alpha) {
  if (!__any_sync(0xffffffffu, alpha != 1.f)) return;
#pragma unroll
  for (int c = 0; c < COLS; c += 8) {  // few at a time: the row's scores are live in registers
    float o[8];
    tmem_ld8(tO + c, o);
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] *= alpha;
    tmem_st8(tO + c, o);
  }
  tmem_wait_st();
}

// The two warps that hold the halves of the same 32 rows meet at a named barrier of their own.
CP_DEV void pair_sync(int id) { asm volatile("barrier.cta.sync %0, 64;" ::"r"(id) : "memory"); }
CP_DEV bool pair_any(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"((uint32_t)x)
      : "memory");
  return r != 0u;
}

// ------------------------------------------------------------------------------ kernel
// TT: the two tiles are two row tiles of one head.  CAP: scores with nothing but a cap, most of whose
// tiles take a short way.
template <int D, bool TT, bool CAP>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_mod_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v, const PrefillModParams p) {
  using Sm = Smem<D>;
  constexpr int KB = D / 64;
  constexpr int SPAN = TT ? 2 * BM : BM;  // query rows of an item
  extern __shared__ uint8_t smem_raw[];
  __shared__ int s_range[kThreads / 32][4];
  __shared__ float s_rows[2][2][BM];  // [tile][half][row]: what the halves of a row tell each other
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  chained_start();

  // ---- the item: heads fastest, then row tiles (the last, longest one first), then sequences
  const int h0 = blockIdx.x * (TT ? 1 : 2), b = blockIdx.z;
  const int q0 = ld(p.cu_q + b), Tq = ld(p.cu_q + b + 1) - q0;
  int kv0 = q0, Tkv = Tq;
  if (p.cu_kv != nullptr) {
    kv0 = ld(p.cu_kv + b);
    Tkv = ld(p.cu_kv + b + 1) - kv0;
  }
  const int prefix = p.prefix != nullptr ? ld(p.prefix + b) : 0;
  const int q_lo = (p.tiles - 1 - (int)blockIdx.y) * SPAN;
  if (blockIdx.y == 0 && threadIdx.x == 0 && Tq - q_lo > SPAN) report(p.err, CP_ERR_DEVICE_BOUNDS);  // max_seqlen_q
  if (q_lo >= Tq) return;
  const int q_hi = min(q_lo + SPAN, Tq);
  const int C = Tkv - Tq;  // cached tokens before the new ones
  // fewer kv tokens than new queries, or rows that the tensors do not have: flagged, the item is skipped
  if (C < 0 || q0 < 0 || kv0 < 0 || (long long)q0 + Tq > p.Nq || (long long)kv0 + Tkv > p.Nkv) {
    if (threadIdx.x == 0) report(p.err, CP_ERR_DEVICE_BOUNDS);
    return;
  }
  const int pre = min(prefix, Tkv);
  // keys [lo, hi) of a row of the sequence
  auto lo_of = [&](int row) -> int {
    int lo = 0;
    if (p.window > 0 && C + row >= p.window) lo = C + row - p.window + 1;
    if (p.kv_start != nullptr) lo = max(lo, ld(p.kv_start + q0 + row));
    return min(lo, Tkv);
  };
  auto hi_of = [&](int row) -> int { return max(C + row + 1, pre); };
  // ---- barriers, Q and TMEM, while the rows' ranges come in
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* sbase = smem_raw + (base - raw);
  const uint32_t sQ = base + Sm::oQ, sKV = base + Sm::oKV;
  auto bar = [&](int i) -> uint32_t { return base + (uint32_t)Sm::oBar + 8u * (uint32_t)i; };
  uint32_t* misc = reinterpret_cast<uint32_t*>(sbase + Sm::oMisc);
  volatile uint32_t* abort_flag = misc + 1;
  int* unclean = reinterpret_cast<int*>(misc + 2);  // first, last key tile whose V was unclean
  auto fail = [&]() {
    *abort_flag = 1u;
    report(p.err, CP_ERR_TIMEOUT);
  };

  if (threadIdx.x == 0) {
    mbar_init(bar(Sm::bQ), 1);
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(bar(Sm::bFull + s), 1);
      mbar_init(bar(Sm::bEmpty + s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(Sm::bS + i), 1);
      mbar_init(bar(Sm::bP + 2 * i), 8);
      mbar_init(bar(Sm::bP + 2 * i + 1), 8);
      mbar_init(bar(Sm::bO + i), 1);
      mbar_init(bar(Sm::bFix + i), 2);
    }
    mbar_init(bar(Sm::bDone), 1);
    misc[1] = 0u;
    unclean[0] = 0x7fffffff;
    unclean[1] = -1;
    fence_mbar_init();
    tma_prefetch_desc(&map_q);
    mbar_expect_tx(bar(Sm::bQ), 2 * Sm::kQ);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
        tma_load_2d(sQ + i * Sm::kQ + kb * BM * 128, &map_q, (h0 + (TT ? 0 : i)) * D + kb * 64,
                    q0 + q_lo + (TT ? i * BM : 0), bar(Sm::bQ));
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(misc), 512);
    tmem_relinquish();
  }

  // union of the rows' ranges and the range that every row sees
  int key_lo, key_hi, all_lo, all_hi;
  if (p.kv_start == nullptr) {
    key_lo = lo_of(q_lo);
    key_hi = hi_of(q_hi - 1);
    all_lo = lo_of(q_hi - 1);
    all_hi = hi_of(q_lo);
    if (q_hi - q_lo < SPAN) all_hi = -1;  // rows past the sequence see nothing
  } else {
    int v[4] = {0x7fffffff, 0, 0, 0x7fffffff};
    for (int i = (int)threadIdx.x - 128; i >= 0 && i < SPAN; i += kThreads - 128) {  // (warps 0 and 1 set up)
      const int row = q_lo + i;
      const int lo = row < q_hi ? lo_of(row) : 1, hi = row < q_hi ? hi_of(row) : 0;
      if (lo < hi) {
        v[0] = min(v[0], lo);
        v[1] = max(v[1], hi);
        v[2] = max(v[2], lo);
        v[3] = min(v[3], hi);
      } else {  // a row without keys: no tile is seen by every row
        v[3] = -1;
      }
    }
    v[0] = __reduce_min_sync(0xffffffffu, v[0]);
    v[1] = __reduce_max_sync(0xffffffffu, v[1]);
    v[2] = __reduce_max_sync(0xffffffffu, v[2]);
    v[3] = __reduce_min_sync(0xffffffffu, v[3]);
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) s_range[warp][i] = v[i];
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  if (p.kv_start != nullptr) {
    key_lo = 0x7fffffff, key_hi = 0, all_lo = 0, all_hi = 0x7fffffff;
    for (int w = 0; w < kThreads / 32; ++w) {
      key_lo = min(key_lo, s_range[w][0]);
      key_hi = max(key_hi, s_range[w][1]);
      all_lo = max(all_lo, s_range[w][2]);
      all_hi = min(all_hi, s_range[w][3]);
    }
  }
  const int ntiles = key_lo < key_hi ? (key_hi - key_lo + BN - 1) / BN : 0;
  // With a distance bias the key tiles are walked from the last to the first: the bias is largest next to the
  // query, so the running reference is met at once and stays (walking up, it moved at every tile of a steep
  // head: 8192 tokens, 16/2 heads took 263 us, now 220).
  const bool down = !CAP && p.slopes != nullptr;
  auto key_tile = [&](int t) -> int { return down ? ntiles - 1 - t : t; };
  auto in_part = [&](int kt) -> bool {  // some row of the CTA sees only a part of key tile kt
    const int k0 = key_lo + kt * BN;
    return k0 < all_lo || k0 + BN > all_hi;
  };

  if (ntiles == 0) {  // no row sees a key
    for (int i = threadIdx.x; i < (q_hi - q_lo) * (TT ? 1 : 2); i += kThreads) {
      const long long row = (long long)(q0 + q_lo + (TT ? i : i >> 1)) * p.Hq + h0 + (TT ? 0 : i & 1);
      for (int c = 0; c < D; c += 8) *reinterpret_cast<uint4*>(p.out + row * D + c) = make_uint4(0u, 0u, 0u, 0u);
      p.lse[row] = -INFINITY;
    }
    if (threadIdx.x == 0) mbar_wait(bar(Sm::bQ), 0u, nullptr, kBudget);  // Q has landed before the CTA exits
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, 512);
    return;
  }

  const int g = h0 / p.G;

  if (warp < 4) {
    regs_dec<64>();  // 128 x 64 + 512 x 104 = the 640 x 96 registers of the launch: the rows' scores in registers,
                     // with 32 (d = 64: 52) bytes of spills beside them in the capped forms, 8 in the others of d = 64
    if (warp == 0) {
      // ---------------------------------------------------------------- TMA producer
      if (lane == 0) {
        tma_prefetch_desc(&map_k);
        tma_prefetch_desc(&map_v);
        bool ok = true;
        int issued = 0;  // ring fills: K(t) is fill 2 t, V(t) fill 2 t + 1
        for (int i = 0; i < 2 * ntiles; ++i) {
          const int slot = i % kSlots;
          if (!mbar_wait(bar(Sm::bEmpty + slot), ((uint32_t)(i / kSlots) & 1u) ^ 1u, abort_flag, kBudget)) {
            ok = false;
            break;
          }
          const CUtensorMap* map = (i & 1) ? &map_v : &map_k;
          mbar_expect_tx(bar(Sm::bFull + slot), Sm::kKV);
#pragma unroll
          for (int kb = 0; kb < KB; ++kb)
            tma_load_2d(sKV + slot * Sm::kKV + kb * BN * 128, map, g * D + kb * 64, kv0 + key_lo + key_tile(i >> 1) * BN,
                        bar(Sm::bFull + slot));
          issued = i + 1;
        }
        if (!ok) fail();
        // every copy issued into this CTA's shared memory has landed before it exits
        mbar_wait(bar(Sm::bQ), 0u, nullptr, kBudget);
        for (int i = max(0, issued - kSlots); i < issued; ++i)
          mbar_wait(bar(Sm::bFull + i % kSlots), (uint32_t)(i / kSlots) & 1u, nullptr, kBudget);
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
        };
        // O += P V of the tile: chunk c of both halves as soon as its P is there (each half's P lies over
        // the front of its own scores)
        auto pv_of = [&](int tile, int t, int slot) -> bool {
          const uint64_t dv = desc_advance(dv0, (uint32_t)(slot * Sm::kKV));
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            if (!mbar_wait(bar(Sm::bP + 2 * tile + c), (uint32_t)t & 1u, abort_flag, kBudget)) return false;
            tc_fence_after();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int half = i >> 1, kk = 2 * c + (i & 1);  // 16-key step of the half
              mma_ts(tmem + 256u + (uint32_t)(tile * D), tmem + (uint32_t)(tile * BN + half * BH + kk * 8),
                     desc_advance(dv, (uint32_t)(half * (BH / 16) + kk) * 16u * 128u), id_pv, t > 0 || c > 0 || i > 0);
            }
          }
          mma_commit(bar(Sm::bO + tile));
          return true;
        };
        bool ok = mbar_wait(bar(Sm::bQ), 0u, abort_flag, kBudget) &&
                  mbar_wait(bar(Sm::bFull), 0u, abort_flag, kBudget);
        if (ok) {
          tc_fence_after();
          issue_qk(0, 0);
          mma_commit(bar(Sm::bS + 0));
          issue_qk(1, 0);
          mma_commit(bar(Sm::bS + 1));
          mma_commit(bar(Sm::bEmpty + 0));
        }
        for (int t = 0; ok && t < ntiles; ++t) {
          const int iv = 2 * t + 1, ik = 2 * t + 2, sv = iv % kSlots, sk = ik % kSlots;
          // V(t) as the guards leave it (they have seen it land)
          ok = mbar_wait(bar(Sm::bFix + (t & 1)), (uint32_t)(t >> 1) & 1u, abort_flag, kBudget) &&
               mbar_wait(bar(Sm::bFull + sv), (uint32_t)(iv / kSlots) & 1u, abort_flag, kBudget);
          if (!ok) break;
          ok = pv_of(0, t, sv);
          if (!ok) break;
          const bool more = t + 1 < ntiles;
          if (more) {
            ok = mbar_wait(bar(Sm::bFull + sk), (uint32_t)(ik / kSlots) & 1u, abort_flag, kBudget);
            if (!ok) break;
            tc_fence_after();
            issue_qk(0, sk);
            mma_commit(bar(Sm::bS + 0));
          }
          ok = pv_of(1, t, sv);
          if (!ok) break;
          mma_commit(bar(Sm::bEmpty + sv));
          if (more) {
            issue_qk(1, sk);
            mma_commit(bar(Sm::bS + 1));
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
      // every tile, in step with the MMA issuer: a barrier's phases are told apart by parity alone
      for (int t = 0; t < ntiles; ++t) {
        const int iv = 2 * t + 1, sv = iv % kSlots;
        const bool ok = __all_sync(0xffffffffu, mbar_wait(bar(Sm::bFull + sv), (uint32_t)(iv / kSlots) & 1u,
                                                          abort_flag, kBudget));
        if (!ok) {
          if (lane == 0) fail();
          break;
        }
        const int kt = key_tile(t);
        if (in_part(kt)) {
          if (guard_v<D, BN>(sbase + Sm::oKV + sv * Sm::kKV, key_hi - key_lo - kt * BN, (warp - 2) * 32 + lane)) {
            atomicMin(unclean, kt);
            atomicMax(unclean + 1, kt);
          }
          fence_proxy_async_smem();  // the MMA reads what was written here
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(Sm::bFix + (t & 1)));
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax, two warpgroups per tile
    regs_inc<104>();
    const int sw = warp - 4, tile = sw >> 3, half = (sw >> 2) & 1, q4 = warp & 3;
    const int pair = 1 + tile * 4 + q4;  // named barrier of the warps with the same rows
    const int row = q_lo + (TT ? tile * BM : 0) + q4 * 32 + lane;  // within the sequence
    const int head = h0 + (TT ? 0 : tile);
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const uint32_t tS = tmem + lane_off + (uint32_t)(tile * BN + half * BH);
    const uint32_t tO = tmem + lane_off + 256u + (uint32_t)(tile * D + half * (D / 2));
    float* const s_mine = &s_rows[tile][half][q4 * 32 + lane];
    float* const s_other = &s_rows[tile][half ^ 1][q4 * 32 + lane];
    const bool valid = row < q_hi;
    const int lo = valid ? lo_of(row) : 0, hi = valid ? hi_of(row) : 0;
    const bool cap = p.softcap > 0.f;
    const float cap_log2 = p.softcap * kLog2e;
    const bool biased = p.slopes != nullptr;
    const float slope = biased ? ld(p.slopes + head) * kLog2e : 0.f;
    // scores come out of cap and bias in log2 units; untouched ones are scaled within the exponent
    const float sc = CAP || cap || biased ? 1.f : p.scale_log2;
    float m = -INFINITY, l = 0.f;
    CapCoefficients coef;
    if constexpr (CAP) coef = cap_coefficients(p.cap_in, p.scale_log2);
    bool ok = true;
    // chunk i of this warp's P is in TMEM: its PV may start
    auto stored = [&](int i) {
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(Sm::bP + 2 * tile + i));
    };
    for (int t = 0; t < ntiles; ++t) {
      const int kt0 = key_lo + key_tile(t) * BN;
      ok = __all_sync(0xffffffffu, mbar_wait(bar(Sm::bS + tile), (uint32_t)t & 1u, abort_flag, kBudget));
      // a warp that gives up raises the abort flag; its partner gives up at its own wait, or where the
      // two meet within the tile
      if (!ok) {
        if (lane == 0) fail();
        __syncwarp();
        // the votes below, as the partner will meet them
        for (int i = 0; i < (CAP ? 3 : 2); ++i) pair_any(pair, true);
        break;
      }
      tc_fence_after();
      Row v;
#pragma unroll
      for (int i = 0; i < kChunks; ++i) tmem_ld32(tS + 32 * i, v.c[i]);
#pragma unroll
      for (int i = 0; i < kChunks; ++i) tmem_wait_ld(v.c[i]);
      const int k0 = kt0 + half * BH;        // this thread's first key
      const int c0 = lo - k0, c1 = hi - k0;  // visible columns [c0, c1)
      // S(t) complete implies PV(t-1) complete (issued before QK(t)): O is stable and the S columns may
      // take P(t)
      float y = 0.f;
      bool bounded = false, near = false;
      if constexpr (CAP) {
        y = row_abs_max(v) * p.cap_in;
        // (a partner that gave up says no, and then takes part in the votes below)
        bounded = !pair_any(pair, !(c0 <= 0 && c1 >= BH && fminf(y, 1.f) * cap_log2 <= m + kMaxGrowth));
        near = bounded && __all_sync(0xffffffffu, y <= kCapNear);
      }
      if (CAP && near) {
        const uint64_t n2 = f2(-m, -m);
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          l += exp_columns(v.c[i], tS + 16 * i, [&](uint64_t s) {
            const uint64_t u = fmul2(s, s);
            return ffma2(s, ffma2(ffma2(ffma2(coef.c[3], u, coef.c[2]), u, coef.c[1]), u, coef.c[0]), n2);
          });
          stored(i);
        }
        continue;
      }
      const bool whole = bounded || __all_sync(0xffffffffu, c0 <= 0 && c1 >= BH);
      if (CAP || cap) cap_scores(v, p.cap_in, cap_log2, CAP ? y : row_abs_max(v) * p.cap_in, whole);
      const float s0 = cap ? 1.f : p.scale_log2;
      const int behind = k0 - (C + row);  // this thread's first key, counted from the query
      bool fold = false;                  // the bias goes into the exponent
      if (!CAP && biased) {
        if (__any_sync(0xffffffffu, behind + BH - 1 > 0 && hi > C + row + 1 && k0 < hi)) {  // keys past the query
#pragma unroll
          for (int i = 0; i < kChunks; ++i)
#pragma unroll
            for (int k = 0; k < 32; ++k)
              v.c[i][k] = fmaf(-slope, fabsf((float)behind + (float)(32 * i + k)), v.c[i][k] * s0);
        } else if (slope >= 0.f && 31.f * slope <= kMaxFold) {
          fold = true;
        } else {
          // (the distance is stepped, exactly, not the bias: a steep one's roundings far away would otherwise stay
          // in it next to the query)
          const uint64_t s02 = f2(s0, s0), slope2 = f2(slope, slope), two = f2(2.f, 2.f);
#pragma unroll
          for (int i = 0; i < kChunks; ++i) {
            uint64_t at = f2((float)(behind + 32 * i), (float)(behind + 32 * i + 1));
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              f2u(ffma2(slope2, at, fmul2(f2(v.c[i][k], v.c[i][k + 1]), s02)), v.c[i][k], v.c[i][k + 1]);
              at = fadd2(at, two);
            }
          }
        }
      }
      if (!whole) {  // by bits, which become predicates seven at a time
        const uint64_t seen = first_bits(c1) & ~first_bits(c0);
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          const uint32_t w = (uint32_t)(seen >> (32 * i));
#pragma unroll
          for (int k = 0; k < 32; ++k) v.c[i][k] = (w & (1u << k)) != 0u ? v.c[i][k] : -INFINITY;
        }
      }
      if (!CAP || !bounded) {
        float mt = -INFINITY;  // the row's largest score here, or what bounds it
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          const float x = chunk_max(v.c[i]);
          mt = fmaxf(mt, !CAP && fold ? fmaf(x, s0, slope * (float)(behind + 32 * i + 31)) : x * sc);
        }
        // The reference, the same in both halves, moves only when a score exceeds it by more than 2^8: the
        // halves ask each other at one barrier, and exchange their maxima only then.  (The next write of s_mine
        // comes after another vote, that is after both have read here.)  CAP: by more than 2^4, so that a row
        // whose first tile shows it few keys does not keep a reference that bounds few tiles.
        constexpr float kGrowth = CAP ? kMaxGrowth / 2.f : kMaxGrowth;
        if (pair_any(pair, mt > m + kGrowth)) {
          *s_mine = mt;
          if (pair_any(pair, *abort_flag != 0u)) {  // both leave, or neither
            ok = false;
            break;
          }
          mt = fmaxf(mt, *s_other);
          float alpha = 1.f;
          if (mt > m + kGrowth) {
            alpha = m == -INFINITY ? 1.f : ex2(m - mt);  // (no key yet: O is 0, as it stays)
            m = mt;
          }
          l *= alpha;
          if (t > 0) rescale_o<D / 2>(tO, alpha);
        }
      }
      const float neg = m == -INFINITY ? 0.f : -m;
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        if (!CAP && fold) {
          const uint64_t s02 = f2(s0, s0), step = f2(2.f * slope, 2.f * slope);
          const float b0 = fmaf(slope, (float)(behind + 32 * i), neg);
          uint64_t bias = f2(b0, b0 + slope);
          l += exp_columns(v.c[i], tS + 16 * i, [&](uint64_t s) {
            const uint64_t x = ffma2(s, s02, bias);
            bias = fadd2(bias, step);
            return x;
          });
        } else {
          const uint64_t sc2 = f2(sc, sc), n2 = f2(neg, neg);
          l += exp_columns(v.c[i], tS + 16 * i, [&](uint64_t s) { return ffma2(s, sc2, n2); });
        }
        stored(i);
      }
    }
    if (ok)
      ok = __all_sync(0xffffffffu,
                      mbar_wait(bar(Sm::bO + tile), (uint32_t)(ntiles - 1) & 1u, abort_flag, kBudget));
    if (!ok && lane == 0) fail();
    ok = !pair_any(pair, !ok);
    if (ok) {
      tc_fence_after();
      *s_mine = l;
      pair_sync(pair);
      l += *s_other;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const long long orow = (long long)(q0 + row) * p.Hq + head;
      // keys of this row within the tiles whose V the guards changed (none, nearly always)
      const int u0 = *(volatile int*)unclean, u1 = *(volatile int*)(unclean + 1);
      const int r0 = u1 < 0 ? 0 : max(lo, key_lo + u0 * BN), r1 = u1 < 0 ? 0 : min(hi, key_lo + (u1 + 1) * BN);
      const bool whole = row - lane + 32 <= q_hi;  // all 32 rows of this warp are real
      // whole warps stage their half rows in shared memory (tile 0 over the Q tiles, free since its last
      // PV came after the other tile's last QK; tile 1 over the ring, its last PV being the CTA's last
      // MMA) and write them out 8 bytes a lane, whole half rows per instruction.  128-byte rows of
      // 64 columns, 16-byte pieces swizzled by the row; a half is a box of its own (d = 128) or half
      // of one.
      const uint32_t sb = (tile == 0 ? sQ : sKV) + (uint32_t)(q4 * 32 * D * 2 + (D == 128 ? half * 4096 : 0));
      constexpr int kPieces = D / 16;  // of a half row
      const int piece0 = D == 128 ? 0 : half * kPieces;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const int col = half * (D / 2) + c * 32;
        float o[32];
        tmem_ld32(tO + c * 32, o);
        tmem_wait_ld(o);
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] *= inv;
        if (r0 < r1) restore<D>(o, p.v + (long long)kv0 * p.Hkv * D, (long long)p.Hkv * D, g * D + col, r0, r1);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 x = make_uint4(pack_bf16(o[8 * j], o[8 * j + 1]), pack_bf16(o[8 * j + 2], o[8 * j + 3]),
                                     pack_bf16(o[8 * j + 4], o[8 * j + 5]), pack_bf16(o[8 * j + 6], o[8 * j + 7]));
          if (whole)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                             sb + (uint32_t)(lane * 128) + ((uint32_t)((piece0 + c * 4 + j) ^ (lane & 7)) << 4)),
                         "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w)
                         : "memory");
          else if (valid)
            *reinterpret_cast<uint4*>(p.out + orow * D + col + 8 * j) = x;
        }
      }
      if (whole) {
        __syncwarp();
        constexpr int LR = 2 * kPieces, RI = 32 / LR;  // lanes per half row, rows per instruction
        const int e8 = lane % LR;
        __nv_bfloat16* dst = p.out + ((long long)(q0 + row - lane) * p.Hq + head) * D + half * (D / 2) + 4 * e8;
#pragma unroll 8
        for (int i = 0; i < 32; i += RI) {
          const int r = i + lane / LR;
          uint2 x;
          asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                       : "=r"(x.x), "=r"(x.y)
                       : "r"(sb + (uint32_t)(r * 128) + ((uint32_t)((piece0 + e8 / 2) ^ (r & 7)) << 4) + (e8 & 1) * 8u));
          *reinterpret_cast<uint2*>(dst + (long long)r * p.Hq * D) = x;
        }
      }
      if (valid && half == 0) p.lse[orow] = l == 0.f ? -INFINITY : ((m == -INFINITY ? 0.f : m) + log2f(l)) * kLn2;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch(const cp_prefill_args& a, const cp_score_mod& mod, float scale, void* out, float* lse,
                   cudaStream_t s) {
  const unsigned long long hq = (unsigned long long)a.num_q_heads * D, hkv = (unsigned long long)a.num_kv_heads * D;
  const unsigned long long nkv = a.cu_seqlens_kv ? (unsigned long long)a.total_kv : (unsigned long long)a.total_q;
  CUtensorMap mq, mk, mv;
  if (!cp_make_bf16_map_2d(&mq, a.q, hq, (unsigned long long)a.total_q, hq, BM) ||
      !cp_make_bf16_map_2d(&mk, a.k, hkv, nkv, hkv, BN) || !cp_make_bf16_map_2d(&mv, a.v, hkv, nkv, hkv, BN))
    return cudaErrorInvalidValue;
  PrefillModParams p;
  p.Hq = a.num_q_heads;
  p.Hkv = a.num_kv_heads;
  p.G = a.num_q_heads / a.num_kv_heads;
  p.Nq = a.total_q;
  p.Nkv = (int)nkv;
  p.window = mod.window;
  p.scale_log2 = scale * kLog2e;
  p.softcap = mod.softcap;
  p.cap_in = mod.softcap > 0.f ? scale / mod.softcap : 0.f;
  const bool folds = mod.softcap > 0.f && cap_folds(scale, mod.softcap) && mod.alibi_slopes == nullptr;
  p.cu_q = a.cu_seqlens_q;
  p.cu_kv = a.cu_seqlens_kv;
  p.kv_start = mod.kv_start;
  p.prefix = mod.prefix_lens;
  p.slopes = mod.alibi_slopes;
  p.v = static_cast<const __nv_bfloat16*>(a.v);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.err = a.err;
  const bool tt = p.G % 2 != 0;  // odd groups: two row tiles of one head share the K / V tiles
  const int span = tt ? 2 * BM : BM;
  // at least one, which reports a sequence that is longer than a max_seqlen_q of 0
  p.tiles = a.max_seqlen_q > 0 ? (a.max_seqlen_q + span - 1) / span : 1;
  if (p.tiles > 65535 || a.num_seqs > 65535) return cudaErrorInvalidConfiguration;
  const dim3 grid(tt ? a.num_q_heads : a.num_q_heads / 2, p.tiles, a.num_seqs);
  auto kern = tt ? (folds ? prefill_mod_kernel<D, true, true> : prefill_mod_kernel<D, true, false>)
                 : (folds ? prefill_mod_kernel<D, false, true> : prefill_mod_kernel<D, false, false>);
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kAlloc);
  if (e != cudaSuccess) return e;
  return launch_chained(kern, grid, kThreads, Smem<D>::kAlloc, s, mq, mk, mv, p);
}

}  // namespace
}  // namespace cpattn

cudaError_t cp_launch_prefill_mod(const cp_prefill_args& a, const cp_score_mod& mod, float scale, void* out,
                                  float* out_lse, cudaStream_t s) {
  return a.head_dim == 64 ? cpattn::launch<64>(a, mod, scale, out, out_lse, s)
                          : cpattn::launch<128>(a, mod, scale, out, out_lse, s);
}
