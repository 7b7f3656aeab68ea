// The paged round-robin K/V cache's own traffic: cp_rope_kv_cache_write (rotate q and k by their
// positions and append k and v, as rows of the cache's type or as 4-bit records) and
// cp_kv_cache_read (positions of a sequence back to contiguous rows).
//
// "Add utility functions to enable pass-kv prefill and allgather decode" (vLLM PR 26059),
// Purpose: KV kept round-robin on the CP ranks; "[Feature] Prefill Context Parallel (PCP) basic
// support" (PR 28718), Purpose: per-rank block tables.
//
// Both are bound by HBM: every input row is read once, every output row written once, 16 bytes a
// thread (2 x 32768 tokens appended, 16/2 heads: 119 us, 83% of the copy bandwidth; 4 x 30720 tokens read,
// 2 heads: 42 us, 89%; into and out of 4 bits the packing and unpacking count as much).  A warp owns a few consecutive tokens: its lanes find their sequences, positions and page
// slots once (and, when rotating, the cosines and sines of all their angles, shared by every head),
// and then stream the tokens' rows.
#include <math.h>

#include "common.cuh"
#include "q4.cuh"

namespace cpattn {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Where a token's K and V rows live: the record index of kv head 0 (page (rank, id) of the pool
// times the kv heads) and the row within the page; head < 0: no row to touch.
struct Slot {
  long long head;
  int row;
};

struct Placement {
  int B, Hkv, cp, I, max_blocks;
  long long pool;
  const int32_t *cu, *start, *tables;
  int32_t* err;
};

// The sequence of token row `row`, B if it lies behind the last one (the whole warp, one row a lane).
// A few hundred sequences: the lanes compare all ends with the warp's first row at once, one load
// latency, and each walks on from there; more: a binary search each.
CP_DEV int seq_of(const Placement& p, int row0, int row) {
  if (p.B > 256) {
    const int s = seq_of_row(p.cu, p.B, row);
    return row < ld(p.cu + s + 1) ? s : p.B;
  }
  int s = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int b = b0 + (int)(threadIdx.x & 31);
    s += __popc(__ballot_sync(0xffffffffu, b < p.B && ld(p.cu + b + 1) <= row0));
  }
  while (s < p.B && ld(p.cu + s + 1) <= row) ++s;
  return s;
}

// Position and slot of token row `row`.  false: behind the last sequence.  A position without a page
// (negative, past the table, an id outside the pool) is reported and its slot left empty.
CP_DEV bool locate(const Placement& p, int row0, int row, long long& pos, Slot& slot) {
  slot.head = -1;
  slot.row = 0;
  pos = -1;
  const int s = seq_of(p, row0, row);
  if (s >= p.B || row < ld(p.cu + s)) return false;
  pos = (long long)ld(p.start + s) + (row - ld(p.cu + s));
  if (pos >= 0) {
    const unsigned turn = (unsigned)pos / (unsigned)p.I, l = turn / (unsigned)p.cp;  // positions fit 32 bits
    const int r = (int)(turn - l * (unsigned)p.cp);
    const long long local = (long long)l * p.I + ((unsigned)pos - turn * (unsigned)p.I), col = local / kQ4Page;
    const int id = col < p.max_blocks ? ld(p.tables + ((long long)r * p.B + s) * p.max_blocks + col) : -1;
    if (id >= 0 && id < p.pool) {
      slot.head = (r * p.pool + id) * p.Hkv;
      slot.row = (int)(local % kQ4Page);
    }
  }
  if (slot.head < 0) report(p.err, CP_ERR_DEVICE_BOUNDS);
  return true;
}

// ------------------------------------------------------------------------------ 8-value pieces
template <typename T>
CP_DEV void load8(const T* p, float (&x)[8]);
template <>
CP_DEV void load8(const float* p, float (&x)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
template <>
CP_DEV void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  x[0] = bf16_lo(a.x), x[1] = bf16_hi(a.x), x[2] = bf16_lo(a.y), x[3] = bf16_hi(a.y);
  x[4] = bf16_lo(a.z), x[5] = bf16_hi(a.z), x[6] = bf16_lo(a.w), x[7] = bf16_hi(a.w);
}
CP_DEV void store8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
CP_DEV uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
CP_DEV void store8(__nv_bfloat16* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}

// ------------------------------------------------------------------------------ write
struct WriteParams {
  Placement at;
  int N, T, Hq, heads, half, rot;  // T: tokens per warp; heads: heads (of q, k and v) per warp
  long long q_stride, k_stride, v_stride, qo_stride;
  const void *q, *k, *v;
  void *q_out, *k_out;
  uint8_t *k_cache, *v_cache;
  const double* inv_freq;
};
constexpr int kWriteTokens = 2;  // most tokens a warp owns

// Rotation.  The angle pos * inv_freq of a far position needs more bits than fp32 has, so it is
// kept in turns: inv_freq / 2 pi as a 64-bit fraction of a turn, times the integer position modulo
// 2^64, which drops whole turns exactly.  The top 32 bits are the angle in [-1/2, 1/2) turns, off by
// 2^-26 turns at most after the conversion to fp32.
//
// The fraction by integers, from inv_freq = mant 2^(e - 1075): mant times 2^66 / 2 pi (its first 64
// bits), shifted.  The handful of fp64 operations that it takes otherwise, on a chip with two fp64 lanes
// per SM and clock, cost more than the 64-bit products here (2 x 32768 tokens, 16/2 heads: 124 against
// 120 us).
CP_DEV unsigned long long turns_of(long long inv_freq) {
  const int e = (int)(inv_freq >> 52) & 0x7ff;
  const unsigned long long frac = (unsigned long long)inv_freq & 0xfffffffffffffull;
  const unsigned long long mant = e == 0 ? frac : frac | (1ull << 52);
  constexpr unsigned long long kPerTurn = 0xa2f9836e4e441529ull;  // floor(2^66 / 2 pi)
  const unsigned long long lo = mant * kPerTurn, hi = __umul64hi(mant, kPerTurn);
  const int right = 1077 - max(e, 1);  // turns 2^64 = mant kPerTurn 2^-right
  unsigned long long t;
  if (right >= 128) t = 0ull;
  else if (right >= 64) t = hi >> (right - 64);
  else if (right > 0) t = (lo >> right) | (hi << (64 - right));
  else t = right > -64 ? lo << -right : 0ull;
  return inv_freq < 0 ? 0ull - t : t;
}

// The pieces (of 8 dims) a head's thread j handles, and whether they are rotated.  Half style: a
// piece of the first half with its partner in the second; pairs style: two neighbours.
struct Pieces {
  int c0, c1;
  bool rot;
};
CP_DEV Pieces pieces_of(int j, int rot, int half) {
  const int rp = rot >> 4;  // threads of a head whose pieces are rotated
  Pieces s;
  s.rot = j < rp;
  if (half && s.rot) {
    s.c0 = j;
    s.c1 = j + rp;
  } else {
    s.c0 = 2 * j;  // half style: 2 rp + 2 (j - rp), the pieces behind the rotated ones
    s.c1 = 2 * j + 1;
  }
  return s;
}

// Scales below this go the long way: their reciprocal or remainders may leave fp32's normal range.
constexpr float kQ4Tiny = 9.860761315262648e-32f;  // 2^-103

// min / max that keep a NaN
CP_DEV float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
CP_DEV float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The integer nearest to t / d (ties to even), for 0 <= t / d well below 2^22 and inv = 1 / d to a few
// ulps, without a division: round the product, and see by the remainder (exact: one fma, and a difference
// of multiples of t's last place) whether the neighbour is nearer.
CP_DEV float nearest_quotient(float t, float d, float half, float inv) {
  constexpr float kRound = 12582912.f;  // 1.5 2^23: what is added to it is rounded to an integer
  const float z = fmaf(t, inv, kRound), n = z - kRound, r = fmaf(-n, d, t), a = fabsf(r);
  const bool off = a > half || (a == half && (__float_as_uint(z) & 1u) != 0u);
  return off ? n + copysignf(1.f, r) : n;
}

// Codes of one head's row by the D / 16 neighbouring threads that hold it (pieces c0, c1 each):
// per group of 64 dims the minimum rounded to bf16, the range above it / 15 rounded to bf16 (at least 0), and
// code = nearest integer to (x - minimum) / scale, ties to even, within 0..15.  A group with an
// infinity or a NaN (or a range beyond bf16) is stored as NaN.
template <int D>
CP_DEV void quantise(const float (&a)[8], const float (&b)[8], const Pieces& s, uint8_t* rec, int row,
                     int j, bool live) {
  constexpr int GR = D / kQ4Group, LPH = D / 16;
  float mna = a[0], mxa = a[0], mnb = b[0], mxb = b[0];
#pragma unroll
  for (int e = 1; e < 8; ++e) {
    mna = min_nan(mna, a[e]), mxa = max_nan(mxa, a[e]);
    mnb = min_nan(mnb, b[e]), mxb = max_nan(mxb, b[e]);
  }
  float sc[GR], mn[GR];
#pragma unroll
  for (int g = 0; g < GR; ++g) {
    const bool ia = GR == 1 || (s.c0 >> 3) == g, ib = GR == 1 || (s.c1 >> 3) == g;
    float lo = min_nan(ia ? mna : INFINITY, ib ? mnb : INFINITY);
    float hi = max_nan(ia ? mxa : -INFINITY, ib ? mxb : -INFINITY);
#pragma unroll
    for (int o = 1; o < LPH; o <<= 1) {
      lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    mn[g] = __bfloat162float(__float2bfloat16_rn(lo));
    // (never below 0: the minimum's rounding may pass the greatest value of a nearly constant group)
    sc[g] = __bfloat162float(__float2bfloat16_rn(max_nan((hi - mn[g]) / 15.f, 0.f)));
    if (!(isfinite(mn[g]) && isfinite(sc[g]))) {
      mn[g] = NAN;
      sc[g] = 0.f;
    }
  }
  if (!live) return;
  auto word = [&](const float (&x)[8], int c) {
    const int g = GR == 1 ? 0 : c >> 3;
    const float m = g == 0 ? mn[0] : mn[GR - 1], d = g == 0 ? sc[0] : sc[GR - 1];
    uint32_t w = 0;
    if (d >= kQ4Tiny) {
      const float inv = 1.f / d, half = 0.5f * d;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = fminf(fmaxf(nearest_quotient(x[e] - m, d, half, inv), 0.f), 15.f);
        w |= (__float_as_uint(n + 8388608.f) & 15u) << (4 * e);  // 2^23 + n: n in the low bits
      }
    } else if (d > 0.f) {
#pragma unroll
      for (int e = 0; e < 8; ++e) w |= (uint32_t)fminf(fmaxf(rintf((x[e] - m) / d), 0.f), 15.f) << (4 * e);
    }
    reinterpret_cast<uint32_t*>(rec + row * (D / 2))[q4_word<D>(c)] = w;
  };
  word(a, s.c0);
  word(b, s.c1);
  if (j < GR) {
    const float m = j == 0 ? mn[0] : mn[GR - 1], d = j == 0 ? sc[0] : sc[GR - 1];
    reinterpret_cast<uint32_t*>(rec + 8 * D)[row * GR + j] = pack2(d, m);
  }
}

// Two fp32 values per instruction (the f32x2 forms of the sm_100 family).
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
CP_DEV uint64_t fmul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Cosines and sines of the 8 pairs a lane rotates, as packed pairs of neighbours.
struct Turns {
  uint64_t c[4], s[4];
};
// x, y <- x cos - y sin, y cos + x sin
CP_DEV void turn2(uint64_t& x, uint64_t& y, uint64_t c, uint64_t s) {
  const uint64_t u = x, minus = s ^ 0x8000000080000000ull;
  x = ffma2(y, minus, fmul2(u, c));
  y = ffma2(u, s, fmul2(y, c));
}
CP_DEV void rotate(float (&a)[8], float (&b)[8], const Turns& w, int half) {
  if (half) {  // (a[e], b[e])
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint64_t x = f2(a[2 * e], a[2 * e + 1]), y = f2(b[2 * e], b[2 * e + 1]);
      turn2(x, y, w.c[e], w.s[e]);
      f2u(x, a[2 * e], a[2 * e + 1]);
      f2u(y, b[2 * e], b[2 * e + 1]);
    }
  } else {  // (a[2 e], a[2 e + 1]), then b's
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      uint64_t x = f2(a[4 * e], a[4 * e + 2]), y = f2(a[4 * e + 1], a[4 * e + 3]);
      turn2(x, y, w.c[e], w.s[e]);
      f2u(x, a[4 * e], a[4 * e + 2]);
      f2u(y, a[4 * e + 1], a[4 * e + 3]);
      x = f2(b[4 * e], b[4 * e + 2]), y = f2(b[4 * e + 1], b[4 * e + 3]);
      turn2(x, y, w.c[e + 2], w.s[e + 2]);
      f2u(x, b[4 * e], b[4 * e + 2]);
      f2u(y, b[4 * e + 1], b[4 * e + 3]);
    }
  }
}

// Cosine and sine of an angle in turns.  fp32 rows take the full-accuracy function; rows that are
// bf16 take the special-function unit's (off by 2^-21.4 at most on half a turn either way: 2^12 below the
// rounding of a row stored as bf16, and where such a row is quantised, enough to give a value that lies
// within 2^-21 of its pair's length of the middle between two codes the other one), a fifth of the instructions.
template <typename T>
CP_DEV void cos_sin(float turn, float& c, float& s) {
  if constexpr (sizeof(T) == 4) {
    sincospif(2.f * turn, &s, &c);
  } else {
    const float x = turn * 6.283185307179586f;
    c = __cosf(x);
    s = __sinf(x);
  }
}

// A warp owns T tokens (and `heads` of their q, k and v heads): its lanes find the tokens' slots, share
// the cosines and sines of their angles in shared memory, and then take D / 16 lanes per head, 16 dims
// (two 16-byte pieces of bf16) a lane.  A lane's dims are the same for every head, so its cosines and
// sines stay in registers for a token.  No barrier of the CTA: the chain of dependent loads before the
// first store (sequence ends, start, page table) is one warp's, hidden behind the others.  Many warps
// with one row each in flight beat fewer with two or three (2 x 32768 tokens, 16/2 heads: 32 warps per
// SM took 145 us where 24 took 172 and 16 took 181), and then the instructions per row: heads walked by
// adding to a pointer and the rotation on packed pairs, 145 -> 124 us.
template <typename T, int D, bool Q4>
__global__ void __launch_bounds__(kThreads, 4) rope_write_kernel(const WriteParams p) {
  constexpr int LPH = D / 16;    // lanes per head
  constexpr int HPW = 32 / LPH;  // heads the warp takes at a time
  __shared__ __align__(16) float cs_all[kWarps][2][D / 2];  // cosines, sines of a token's angles
  chained_start();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long first = ((long long)blockIdx.x * kWarps + warp) * p.T;
  if (first >= p.N) return;
  const int row0 = (int)first, nt = min(p.T, p.N - row0), h = p.rot >> 1, Hkv = p.at.Hkv;
  // q heads [q_lo, q_hi) and k, v heads [m_lo, m_hi) (v's after k's) are this warp's
  const int h_lo = blockIdx.y * p.heads, h_hi = min(p.Hq + 2 * Hkv, h_lo + p.heads);
  const int q_lo = min(h_lo, p.Hq), q_hi = min(h_hi, p.Hq), m_lo = max(h_lo - p.Hq, 0), m_hi = max(h_hi - p.Hq, 0);
  const int j = lane % LPH, hw = lane / LPH;
  const Pieces ps = pieces_of(j, p.rot, p.half);
  const int d0 = 8 * ps.c0, d1 = 8 * ps.c1;

  unsigned long long f[D / 64];  // frequencies lane, lane + 32 in turns per position
#pragma unroll
  for (int i = 0; i < D / 64; ++i) f[i] = lane + 32 * i < h ? turns_of(ld(reinterpret_cast<const long long*>(p.inv_freq) + lane + 32 * i)) : 0ull;
  Slot mine;
  long long my_pos = -1;
  const bool in = locate(p.at, row0, min(row0 + lane, row0 + nt - 1), my_pos, mine);
  if (!in) my_pos = -1;  // behind the last sequence; a negative position (reported) is skipped too

  for (int t = 0; t < nt; ++t) {
    const int row = row0 + t;
    const long long pos = __shfl_sync(0xffffffffu, my_pos, t);
    if (pos < 0) continue;
    Turns w;
    if (h > 0) {
      float(*const cs)[D / 2] = cs_all[warp];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < D / 64; ++i)
        if (lane + 32 * i < h) {
          const float turn = (float)(int)(uint32_t)((f[i] * (unsigned long long)pos) >> 32) * 2.3283064365386963e-10f;  // 2^-32
          cos_sin<T>(turn, cs[0][lane + 32 * i], cs[1][lane + 32 * i]);
        }
      __syncwarp();
      if (ps.rot) {  // half style: the 8 angles of piece c0; pairs style: 4 of each piece
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          w.c[e] = *reinterpret_cast<const uint64_t*>(&cs[0][8 * j + 2 * e]);
          w.s[e] = *reinterpret_cast<const uint64_t*>(&cs[1][8 * j + 2 * e]);
        }
      }
    }
    {
      const T* src = static_cast<const T*>(p.q) + row * p.q_stride + (q_lo + hw) * D;
      T* dst = static_cast<T*>(p.q_out) + row * p.qo_stride + (q_lo + hw) * D;
      for (int hd = q_lo + hw; hd < q_hi; hd += HPW, src += HPW * D, dst += HPW * D) {
        float a[8], b[8];
        load8(src + d0, a);
        load8(src + d1, b);
        if (ps.rot) rotate(a, b, w, p.half);
        store8(dst + d0, a);
        store8(dst + d1, b);
      }
    }
    Slot sl;
    sl.head = __shfl_sync(0xffffffffu, mine.head, t);
    sl.row = __shfl_sync(0xffffffffu, mine.row, t);
    for (int m0 = m_lo; m0 < m_hi; m0 += HPW) {  // whole warps: the 4-bit form reduces over a head's lanes
      const int m = m0 + hw;
      const bool live = m < m_hi, is_v = m >= Hkv;
      const int g = is_v ? m - Hkv : m;
      float a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, b[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (live) {
        const T* src = (is_v ? static_cast<const T*>(p.v) + row * p.v_stride : static_cast<const T*>(p.k) + row * p.k_stride) + g * D;
        load8(src + d0, a);
        load8(src + d1, b);
        if (ps.rot && !is_v) rotate(a, b, w, p.half);
        if (!is_v && p.k_out != nullptr) {
          T* dst = static_cast<T*>(p.k_out) + ((long long)row * Hkv + g) * D;
          store8(dst + d0, a);
          store8(dst + d1, b);
        }
      }
      uint8_t* cache = is_v ? p.v_cache : p.k_cache;
      if constexpr (Q4) {
        if (sl.head >= 0)
          quantise<D>(a, b, ps, cache + (sl.head + g) * q4_record_bytes(D), sl.row, j, live);
      } else if (live && sl.head >= 0) {
        T* dst = reinterpret_cast<T*>(cache) + ((sl.head + g) * kQ4Page + sl.row) * D;
        store8(dst + d0, a);
        store8(dst + d1, b);
      }
    }
  }
}

// ------------------------------------------------------------------------------ read
struct ReadParams {
  Placement at;
  int N, T;  // T: tokens per warp
  const uint8_t *k_cache, *v_cache;
  void *k_out, *v_out;
};

// A warp owns T <= 32 tokens: lane t finds token t's slot, then V lanes per row stream the tokens' rows
// (K's heads, then V's), 16 output bytes a lane, U of them in flight.  `load` brings what one needs.
template <int V, int U, typename Load, typename Store>
CP_DEV void stream_rows(const ReadParams& p, Slot* slots, Load load, Store store) {
  constexpr int RPW = 32 / V;  // rows the warp takes at a time
  chained_start();
  const int lane = threadIdx.x & 31;
  const long long first = ((long long)blockIdx.x * kWarps + (threadIdx.x >> 5)) * p.T;
  if (first >= p.N) return;
  const int row0 = (int)first, nt = min(p.T, p.N - row0), Hkv = p.at.Hkv;
  long long pos;
  Slot mine;
  locate(p.at, row0, min(row0 + lane, row0 + nt - 1), pos, mine);
  slots[lane] = mine;
  __syncwarp();
  const int v = lane % V, m_first = lane / V;
  int t = 0, m0 = 0;  // token, and first of the rows (of 2 Hkv) taken at this step: the same in all lanes
  while (t < nt) {
    decltype(load(true, 0ll, 0, 0)) x[U];
    long long dst[U];  // 16-byte piece of the output (K's or V's), -1: none
    bool is_v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int m = m0 + m_first;
      is_v[u] = m >= Hkv;
      const int g = is_v[u] ? m - Hkv : m;
      dst[u] = -1;
      if (t < nt && m < 2 * Hkv) {
        const Slot sl = slots[t];
        if (sl.head >= 0) {
          x[u] = load(is_v[u], sl.head + g, sl.row, v);
          dst[u] = ((long long)(row0 + t) * Hkv + g) * V + v;
        }
      }
      m0 += RPW;
      if (m0 >= 2 * Hkv) m0 = 0, ++t;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (dst[u] >= 0) store(is_v[u], dst[u], x[u]);
  }
}

// Rows of the cache's own type, V 16-byte pieces each, copied.
template <int V>
__global__ void __launch_bounds__(kThreads) read_rows_kernel(const ReadParams p) {
  __shared__ Slot slots[kWarps][32];
  stream_rows<V, 4>(
      p, slots[threadIdx.x >> 5],
      [&](bool is_v, long long head, int row, int v) {
        return ld(reinterpret_cast<const uint4*>(is_v ? p.v_cache : p.k_cache) + (head * kQ4Page + row) * V + v);
      },
      [&](bool is_v, long long at, const uint4& x) { static_cast<uint4*>(is_v ? p.v_out : p.k_out)[at] = x; });
}

// The 8 values of a word of codes.  A code in place (n 16^e, e its nibble within a half word) below 2^23
// in the mantissa of 2^23 is a float without a conversion (a quarter of the rate of an addition);
// scale / 16^e is exact, so each value is rounded once (the product is exact).
// (10112 tokens of 8 heads, d = 128: 19.6 -> 17.5 us with two words a lane.)
CP_DEV void q4_values(uint32_t w, uint32_t sm, float (&x)[8]) {
  const float sc = bf16_lo(sm), mn = bf16_hi(sm);
  float s = sc;
#pragma unroll
  for (int e = 0; e < 4; ++e, s *= 0.0625f) {
    const uint32_t mask = 15u << (4 * e);
    x[e] = fmaf(s, __uint_as_float((w & mask) | 0x4b000000u) - 8388608.f, mn);
    x[e + 4] = fmaf(s, __uint_as_float((w >> 16 & mask) | 0x4b000000u) - 8388608.f, mn);
  }
}

// 4-bit rows to the values they stand for: a lane turns two words (16 codes; of both groups, d = 128) into
// 16 values.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) read_q4_kernel(const ReadParams p) {
  constexpr int GR = D / kQ4Group, V = D / 16;
  __shared__ Slot slots[kWarps][32];
  stream_rows<V, 4>(
      p, slots[threadIdx.x >> 5],
      [&](bool is_v, long long head, int row, int c) {
        const uint8_t* rec = (is_v ? p.v_cache : p.k_cache) + head * q4_record_bytes(D);
        const uint2 w = ld(reinterpret_cast<const uint2*>(rec + row * (D / 2)) + c);
        const uint32_t* sm = reinterpret_cast<const uint32_t*>(rec + 8 * D) + row * GR;
        const uint32_t s0 = ld(sm);
        return make_uint4(w.x, w.y, s0, GR == 2 ? ld(sm + GR - 1) : s0);
      },
      [&](bool is_v, long long at, const uint4& w) {
        float x[8];
        T* out = static_cast<T*>(is_v ? p.v_out : p.k_out) + at / V * D;
        const int c = (int)(at % V);
        q4_values(w.x, w.z, x);
        store8(out + (GR == 2 ? 8 * c : 16 * c), x);
        q4_values(w.y, w.w, x);
        store8(out + (GR == 2 ? 64 + 8 * c : 16 * c + 8), x);
      });
}

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
    sms = 152;
  return sms;
}

}  // namespace
}  // namespace cpattn

cudaError_t cp_launch_rope_write(const cp_rope_write_args& a, cudaStream_t s) {
  using namespace cpattn;
  WriteParams p;
  p.at = Placement{a.num_seqs, a.num_kv_heads, a.cp, a.interleave, a.max_blocks, a.pool_pages,
                   a.cu_new, a.start_pos, a.block_tables, a.err};
  p.N = a.total_new;
  p.Hq = a.q != nullptr ? a.num_q_heads : 0;
  p.half = a.rope_style == CP_ROPE_HALF;
  p.rot = a.rot_dim;
  p.q_stride = a.q_stride;
  p.k_stride = a.k_stride;
  p.v_stride = a.v_stride;
  p.qo_stride = a.q_out_stride;
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  p.q_out = a.q_out;
  p.k_out = a.k_out;
  p.k_cache = static_cast<uint8_t*>(a.k_cache);
  p.v_cache = static_cast<uint8_t*>(a.v_cache);
  p.inv_freq = a.inv_freq;
  // tokens per warp: few enough that every SM gets its warps; with fewer tokens than that, a token's
  // heads are split over warps too (each then computes the token's angles again)
  const long long warps = 32ll * sm_count();
  const int nh = p.Hq + 2 * a.num_kv_heads, at_a_time = 32 / (a.head_dim / 16);
  long long t = p.N / warps;
  p.T = (int)(t < 1 ? 1 : (t > kWriteTokens ? kWriteTokens : t));
  long long pieces = p.T == 1 ? warps / p.N : 1;
  const long long most = (nh + at_a_time - 1) / at_a_time;
  pieces = pieces < 1 ? 1 : (pieces > most ? most : pieces);
  const long long each = ((nh + pieces - 1) / pieces + at_a_time - 1) / at_a_time * at_a_time;
  p.heads = (int)each;
  const long long per_cta = (long long)kWarps * p.T;
  const dim3 grid((unsigned)((p.N + per_cta - 1) / per_cta), (unsigned)((nh + each - 1) / each));
  auto go = [&](auto kern) -> cudaError_t {
    return launch_chained(kern, dim3(grid), kThreads, 0, s, p);
  };
  const bool q4 = a.cache_q4 != 0, bf = a.dtype == CP_BF16;
  if (a.head_dim == 128) {
    if (bf) return q4 ? go(rope_write_kernel<__nv_bfloat16, 128, true>)
                      : go(rope_write_kernel<__nv_bfloat16, 128, false>);
    return q4 ? go(rope_write_kernel<float, 128, true>) : go(rope_write_kernel<float, 128, false>);
  }
  if (bf) return q4 ? go(rope_write_kernel<__nv_bfloat16, 64, true>)
                    : go(rope_write_kernel<__nv_bfloat16, 64, false>);
  return q4 ? go(rope_write_kernel<float, 64, true>) : go(rope_write_kernel<float, 64, false>);
}

cudaError_t cp_launch_kv_read(const cp_kv_read_args& a, cudaStream_t s) {
  using namespace cpattn;
  ReadParams p;
  p.at = Placement{a.num_seqs, a.num_kv_heads, a.cp, a.interleave, a.max_blocks, a.pool_pages,
                   a.cu_out, a.start_pos, a.block_tables, a.err};
  p.N = a.total;
  p.k_cache = static_cast<const uint8_t*>(a.k_cache);
  p.v_cache = static_cast<const uint8_t*>(a.v_cache);
  p.k_out = a.k_out;
  p.v_out = a.v_out;
  const int d = a.head_dim;
  const int row_bytes = d * (a.out_dtype == CP_BF16 ? 2 : 4);
  // tokens per warp: a lane each, fewer where that would leave SMs without their warps
  const long long t = p.N / (32ll * sm_count());
  p.T = (int)(t < 1 ? 1 : (t > 8 ? 8 : t));
  const long long per_cta = (long long)kWarps * p.T;
  const unsigned grid = (unsigned)((p.N + per_cta - 1) / per_cta);
  auto go = [&](auto kern) -> cudaError_t {
    return launch_chained(kern, dim3(grid), kThreads, 0, s, p);
  };
  if (a.cache_q4) {
    if (d == 128) return a.out_dtype == CP_BF16 ? go(read_q4_kernel<__nv_bfloat16, 128>) : go(read_q4_kernel<float, 128>);
    return a.out_dtype == CP_BF16 ? go(read_q4_kernel<__nv_bfloat16, 64>) : go(read_q4_kernel<float, 64>);
  }
  if (row_bytes == 128) return go(read_rows_kernel<8>);
  if (row_bytes == 256) return go(read_rows_kernel<16>);
  return go(read_rows_kernel<32>);
}
