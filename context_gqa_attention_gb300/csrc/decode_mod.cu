// Decode over the round-robin paged cache with modified scores (cp_decode_attention_mod), one query
// token per sequence; bf16 and fp32 caches.
//
// "Add utility functions to enable pass-kv prefill and allgather decode" (vLLM PR 26059),
// Purpose: decode KV stays on the CP ranks round-robin, each rank attends the new query over its
// own tokens and the partials are combined.
//
//   s_j = scale q.k_j;  s_j = cap tanh(s_j / cap);  s_j -= slope |i - j|     (each optional)
//   over the keys j in [lo, L), lo = max(0, L - window, kv_start);  out = softmax(s) V
//
// Work unit (one CTA of 4 warps): split s of rank r's visible tokens of sequence b, kv head g, all
// query heads of the group; a warp takes every fourth page (16 tokens).  Both products run on the
// tensor cores with the *tokens* as the M dimension of S^T = K Q^T (16 tokens x 8 heads per MMA)
// and the head's dims as the M dimension of O^T = V^T P^T, so a page costs D / 16 + D / 16 MMAs
// for up to 8 query heads, and K and V go from global memory straight into the A fragments: the
// contraction order of K's dims and the row order of V's dims are free, so each thread's 16-byte
// piece of a row is a set of whole fragments, and no shared memory or ldmatrix is needed.
// P^T (tokens x heads -> heads x tokens) is transposed between the products by movmatrix.
// Bound by HBM: every K and V byte is read once (64 sequences of 1024..32768 tokens, 32/8 heads, cap 50:
// 671 us, as fast as a copy of the same bytes).
#include "decode_mod.cuh"

namespace cpattn {
namespace {

struct Piece {  // 16 bytes of a row in 32-bit words
  uint32_t w[4];
};
CP_DEV void load_piece(Piece& x, const uint8_t* p) {
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(x.w[0]), "=r"(x.w[1]), "=r"(x.w[2]), "=r"(x.w[3]) : "l"(p));
}

// What one thread (row id gid = lane / 4, column id tid = lane % 4) holds of a page of one head.
//   K of tokens gid and gid + 8;  V of tokens 2 tid, 2 tid + 1, 2 tid + 8, 2 tid + 9.
// K and V are loaded apart: K's registers are refilled with the next page's as soon as the scores are
// computed, V's after the second product, so loads are in flight during most of an iteration
// without a second set of registers.
template <int D>
struct PageK {
  Piece x[2][D / 32];  // 16-byte pieces tid, tid + 4, ..
  static CP_DEV int at(int gid, int tid) { return gid * (2 * D) + tid * 16; }
  CP_DEV void load(const uint8_t* r) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int c = 0; c < D / 32; ++c) load_piece(x[i][c], r + i * (16 * D) + c * 64);
  }
};
template <int D>
struct PageV {
  Piece x[4][D / 64];  // pieces gid, gid + 8
  static CP_DEV int at(int gid, int tid) { return tid * (4 * D) + gid * 16; }
  CP_DEV void load(const uint8_t* r) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < D / 64; ++c) load_piece(x[i][c], r + (i & 1) * (2 * D) + (i >> 1) * (16 * D) + c * 128);
  }
};

// NT: tiles of 8 query heads.
template <int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, NT == 1 ? 3 : 2) decode_mod_kernel(const ModParams p) {
  using T = __nv_bfloat16;
  constexpr int HR = 8 * NT;         // head rows (query heads of the group, padded)
  constexpr int KS = D / 16;         // MMAs of each product
  constexpr int kRec = 2 * kPage * D;  // bytes of a head's page
  __shared__ __align__(16) WarpParts<D, HR> parts;
  Unit u;
  if (!take_unit<T, D, HR>(p, parts, u)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tid = lane & 3;

  // table entries of this warp's pages pg0 + warp + j kWarps, 32 at a time (lane i holds the i-th), a
  // batch ahead
  const int32_t* trow = p.tables + ((long long)u.r * p.B + u.b) * p.max_blocks;
  const int pg0 = u.l0 / kPage, pg1 = (u.l1 + kPage - 1) / kPage;
  const int iters = (pg1 - pg0 - warp + kWarps - 1) / kWarps;
  auto fetch_ids = [&](int j0) -> int {
    const int pg = pg0 + (j0 + lane) * kWarps + warp;
    int id = -1;
    if (pg < pg1 && pg < p.max_blocks) id = ld(trow + pg);
    return id >= 0 && id < p.pool ? id : -1;
  };
  int ids = fetch_ids(0), ids_next = fetch_ids(32);
  auto page_of = [&](int k) -> int {  // -1: none (its tokens are masked)
    if ((k & 31) == 0 && k > 0) {
      ids = ids_next;
      ids_next = fetch_ids(k + 32);
    }
    return __shfl_sync(0xffffffffu, ids, k & 31);
  };
  const int page_stride = p.Hkv * kRec;  // Hkv <= 65535: below 2^31
  const long long unit_base = (long long)u.r * p.pool * page_stride + (long long)u.g * kRec;
  const uint8_t* const kbase = p.kc + unit_base + PageK<D>::at(gid, tid);
  const uint8_t* const vbase = p.vc + unit_base + PageV<D>::at(gid, tid);
  PageK<D> kx;
  PageV<D> vx;
  int id = page_of(0), id_nxt = -1;
  if (id >= 0) {
    kx.load(kbase + (long long)id * page_stride);
    vx.load(vbase + (long long)id * page_stride);
  }

  // Q^T as the B operand of S^T = K Q^T: the dims of MMA ks as K's pieces bring them, arranged in
  // shared memory by the whole CTA (16 bytes of q, 8 dims, are 4 operand words of one lane)
  uint32_t(*const q_ops)[32][2 * KS + 4] = reinterpret_cast<uint32_t(*)[32][2 * KS + 4]>(&parts.o[0][0][0]);
  static_assert(sizeof(parts.o) >= sizeof(uint32_t) * NT * 32 * (2 * KS + 4), "q operands");
  constexpr int TPH = D / 8;  // threads per head
  for (int i = threadIdx.x; i < HR * TPH; i += kWarps * 32) {
    const int head = i / TPH, c = i % TPH;
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (head < p.G)
      x = ld(reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) +
                                               ((long long)u.b * p.Hq + (long long)u.g * p.G + head) * D) + c);
    *reinterpret_cast<uint4*>(&q_ops[head / 8][(head % 8) * 4 + c % 4][(c / 4) * 4]) = x;
  }
  __syncthreads();
  uint32_t qb[NT][KS][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int w = 0; w < KS / 2; ++w) {
      const uint4 x = *reinterpret_cast<const uint4*>(&q_ops[nt][lane][4 * w]);
      qb[nt][2 * w][0] = x.x, qb[nt][2 * w][1] = x.y, qb[nt][2 * w + 1][0] = x.z, qb[nt][2 * w + 1][1] = x.w;
    }
  __syncthreads();  // the warps' parts take this memory at the end
  const Mods<NT> mods(p, u, tid);
  const float scale = p.scale * kLog2e;

  // per head of this thread's columns (2 tid, 2 tid + 1): reference m (log2; neg = -m, 0 before the
  // first score) and the sum of this thread's tokens
  float m[NT][2], neg[NT][2], l[NT][2], o[NT][KS][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int c = 0; c < 2; ++c) m[nt][c] = -INFINITY, neg[nt][c] = 0.f, l[nt][c] = 0.f;
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
  }

  bool bad = false;
  for (int k = 0; k < iters; ++k) {
    const int t0 = (pg0 + k * kWarps + warp) * kPage;  // the page's first local token
    const bool edge = id < 0 || t0 < u.a || t0 + kPage > u.l1;  // some token of it is not visible
    auto visible = [&](int token) { return id >= 0 && t0 + token >= u.a && t0 + token < u.l1; };

    // ---- S^T: rows = tokens gid, gid + 8; columns = heads 2 tid, 2 tid + 1
    float s[NT][4];  // [token half * 2 + head], log2 units
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const int w = (ks % 2) * 2;
      const Piece &k0 = kx.x[0][ks / 2], &k1 = kx.x[1][ks / 2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        mma16816(s[nt], k0.w[w], k1.w[w], k0.w[w + 1], k1.w[w + 1], qb[nt][ks][0], qb[nt][ks][1]);
    }
    // ---- the next page's K into the registers that are free now
    if (k + 1 < iters) {
      id_nxt = page_of(k + 1);
      if (id_nxt >= 0) kx.load(kbase + (long long)id_nxt * page_stride);
    }

#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] *= scale;
    mods.apply(s, p, u, t0 + gid);
    if (edge) {
      bad |= id < 0 && t0 < u.l1;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (!visible(gid + 8 * h)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) s[nt][2 * h] = s[nt][2 * h + 1] = -INFINITY;
        }
    }
    // The reference moves only when some score exceeds it by more than 2^8 (fp32 sums hold that
    // with room to spare), so the reduction over the 8 rows of lanes is rare.
    bool grow = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) grow |= fmaxf(s[nt][h], s[nt][2 + h]) > m[nt][h] + kMaxGrowth;
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float alpha = new_reference(fmaxf(s[nt][h], s[nt][2 + h]), m[nt][h], neg[nt][h]);
          l[nt][h] *= alpha;
#pragma unroll
          for (int i = 0; i < KS; ++i) {
            o[nt][i][h] *= alpha;
            o[nt][i][2 + h] *= alpha;
          }
        }
    }

    // ---- P^T as the B operand of O^T = V^T P^T, rounded to bf16 (V's type: an MMA takes one); the
    // sums keep 32 bits
    uint32_t pb[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = sm100::ex2(s[nt][e] + neg[nt][e & 1]);
      l[nt][0] += s[nt][0] + s[nt][2];
      l[nt][1] += s[nt][1] + s[nt][3];
#pragma unroll
      for (int h = 0; h < 2; ++h) pb[nt][h] = transpose8x8(pack2(s[nt][2 * h], s[nt][2 * h + 1]));
    }
    if (edge) {  // rows behind the sequence may hold anything, and 0 times NaN is NaN
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if (!visible(2 * tid + (x & 1) + 8 * (x >> 1))) {
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
#pragma unroll
            for (int w = 0; w < 4; ++w) vx.x[x][c].w[w] = 0u;
        }
      }
    }
    // ---- O^T: rows = dims, columns = heads
#pragma unroll
    for (int x = 0; x < KS; ++x) {
      const int c = x / 4, w = x % 4;
      const uint32_t a0 = low_halves(vx.x[0][c].w[w], vx.x[1][c].w[w]);
      const uint32_t a1 = high_halves(vx.x[0][c].w[w], vx.x[1][c].w[w]);
      const uint32_t a2 = low_halves(vx.x[2][c].w[w], vx.x[3][c].w[w]);
      const uint32_t a3 = high_halves(vx.x[2][c].w[w], vx.x[3][c].w[w]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][x], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
    }
    if (k + 1 < iters && id_nxt >= 0) vx.load(vbase + (long long)id_nxt * page_stride);
    id = id_nxt;
  }
  if (bad && lane == 0) report(p.err, CP_ERR_DEVICE_BOUNDS);

  // ---- this warp's part: sums over the lanes that share a column, output rows per head
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float sum = column_sum(l[nt][h]);
      const int head = 8 * nt + 2 * tid + h;
      if (gid == 0) {
        parts.m[warp][head] = m[nt][h];
        parts.l[warp][head] = sum;
      }
      const float(&x)[KS][4] = o[nt];
#pragma unroll
      for (int i = 0; i < KS; i += 4) {  // four MMAs (dims 2 j, 2 j + 1 of a piece): 8 dims
        float4* const at = reinterpret_cast<float4*>(&parts.o[warp][head][16 * i + 8 * gid]);
        at[0] = make_float4(x[i][h], x[i][2 + h], x[i + 1][h], x[i + 1][2 + h]);
        at[1] = make_float4(x[i + 2][h], x[i + 2][2 + h], x[i + 3][h], x[i + 3][2 + h]);
      }
    }
  finish<T, D, HR>(p, parts, u.b, u.g, u.part, u.live);
}

// ------------------------------------------------------------------------------ fp32 caches
// Two fp32 values per instruction: no more arithmetic a cycle, but half the instructions.
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

// fp32 K and V keep their 24 bits, so the products run on the CUDA cores: two lanes per token for
// q.k, alternating over its 16-byte vectors, D / 4 lanes per row for P V.  A page's K vectors are all in
// flight at once, and refilled with the next page's as soon as the scores are computed; V's likewise
// after the second product.
// Bound by latency and issue at 8 to 12 warps per SM (16 sequences of 300..4000 tokens, 16/2 heads,
// d = 128, cap 30: 39 us; 45 with a maximum per page and scalar arithmetic).
template <int D, int HR>
__global__ void __launch_bounds__(kWarps * 32, D == 64 && HR <= 4 ? 3 : 2) decode_mod_f32_kernel(const ModParams p) {
  constexpr int NCH = D / 4;      // lanes per V row
  constexpr int TG = 32 / NCH;    // V rows a warp reads at a time
  constexpr int NK = D / 8, NV = kPage / TG;
  __shared__ __align__(16) WarpParts<D, HR> parts;
  __shared__ __align__(16) float qs[HR][D];
  __shared__ float ps[kWarps][kPage][HR];
  Unit u;
  if (!take_unit<float, D, HR>(p, parts, u)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tk = lane >> 1, half = lane & 1, vc = lane % NCH, vt = lane / NCH;
  const int32_t* trow = p.tables + ((long long)u.r * p.B + u.b) * p.max_blocks;
  const int pg1 = (u.l1 + kPage - 1) / kPage;
  const long long page_stride = (long long)p.Hkv * (kPage * D);
  const long long unit_base = (long long)u.r * p.pool * page_stride + (long long)u.g * (kPage * D);
  const float* const kbase = reinterpret_cast<const float*>(p.kc) + unit_base + tk * D + half * 4;
  const float* const vbase = reinterpret_cast<const float*>(p.vc) + unit_base + vt * D + vc * 4;
  auto page_of = [&](int pg) -> int {  // -1: none (its tokens are masked)
    int id = -1;
    if (pg < pg1 && pg < p.max_blocks) id = ld(trow + pg);
    return id >= 0 && id < p.pool ? id : -1;
  };
  float4 k[NK], v[NV];
  auto load_k = [&](int id) {
#pragma unroll
    for (int c = 0; c < NK; ++c) k[c] = ld(reinterpret_cast<const float4*>(kbase + id * page_stride) + 2 * c);
  };
  auto load_v = [&](int id) {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = ld(reinterpret_cast<const float4*>(vbase + id * page_stride + i * TG * D));
  };
  int pg = u.l0 / kPage + warp, id = page_of(pg), id_nxt = page_of(pg + kWarps);
  if (id >= 0) {
    load_k(id);
    load_v(id);
  }
  const float* qg = static_cast<const float*>(p.q) + ((long long)u.b * p.Hq + (long long)u.g * p.G) * D;
  for (int i = threadIdx.x; i < HR * D; i += blockDim.x) (&qs[0][0])[i] = i < p.G * D ? qg[i] : 0.f;
  __syncthreads();
  float m[HR], l[HR];      // reference (log2), and the sum of this lane's token
  uint64_t acc[HR][2];     // pairs of dims
#pragma unroll
  for (int h = 0; h < HR; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
    acc[h][0] = acc[h][1] = f2(0.f, 0.f);
  }
  bool bad = false;
  for (; pg < pg1; pg += kWarps) {
    const int t0 = pg * kPage, t = t0 + tk;
    const bool on = id >= 0 && t >= u.a && t < u.l1;
    bad |= id < 0;
    uint64_t dot[HR];
#pragma unroll
    for (int h = 0; h < HR; ++h) dot[h] = f2(0.f, 0.f);
#pragma unroll
    for (int c = 0; c < NK; ++c) {
      const uint64_t k0 = f2(k[c].x, k[c].y), k1 = f2(k[c].z, k[c].w);
#pragma unroll
      for (int h = 0; h < HR; ++h) {
        const float4 q = *reinterpret_cast<const float4*>(&qs[h][8 * c + 4 * half]);
        dot[h] = ffma2(f2(q.x, q.y), k0, ffma2(f2(q.z, q.w), k1, dot[h]));
      }
    }
    if (id_nxt >= 0) load_k(id_nxt);
    const int id_after = page_of(pg + 2 * kWarps);
    const float dist = p.slopes != nullptr ? distance(p, u, t) : 0.f;
    float s[HR];
    bool grow = false;
#pragma unroll
    for (int h = 0; h < HR; ++h) {
      float lo, hi;
      f2u(dot[h], lo, hi);
      lo += hi;
      lo += __shfl_xor_sync(0xffffffffu, lo, 1);
      float x = lo * p.scale;
      if (p.softcap > 0.f) x = p.softcap * tanhf(x / p.softcap);
      if (p.slopes != nullptr && h < p.G) x -= ld(p.slopes + u.g * p.G + h) * dist;
      s[h] = on ? x * kLog2e : -INFINITY;
      grow |= s[h] > m[h] + kMaxGrowth;
    }
    if (__any_sync(0xffffffffu, grow)) {  // as in the bf16 kernel: rare
#pragma unroll
      for (int h = 0; h < HR; ++h) {
        const float m_new = fmaxf(m[h], warp_max(s[h]));
        const float alpha = m_new == m[h] ? 1.f : exp2f(m[h] - m_new);
        m[h] = m_new;
        l[h] *= alpha;
        acc[h][0] = fmul2(acc[h][0], f2(alpha, alpha));
        acc[h][1] = fmul2(acc[h][1], f2(alpha, alpha));
      }
    }
#pragma unroll
    for (int h = 0; h < HR; ++h) {
      const float e = exp2f(s[h] - (m[h] == -INFINITY ? 0.f : m[h]));
      if (half == 0) {
        l[h] += e;
        ps[warp][tk][h] = e;
      }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int r = vt + i * TG;
      // rows behind the sequence may hold anything, and 0 times NaN is NaN
      const bool seen = id >= 0 && t0 + r >= u.a && t0 + r < u.l1;
      const float4 x = seen ? v[i] : make_float4(0.f, 0.f, 0.f, 0.f);
      const uint64_t x0 = f2(x.x, x.y), x1 = f2(x.z, x.w);
#pragma unroll
      for (int h = 0; h < HR; ++h) {
        const float w = ps[warp][r][h];
        const uint64_t w2 = f2(w, w);
        acc[h][0] = ffma2(w2, x0, acc[h][0]);
        acc[h][1] = ffma2(w2, x1, acc[h][1]);
      }
    }
    if (id_nxt >= 0) load_v(id_nxt);
    __syncwarp();
    id = id_nxt;
    id_nxt = id_after;
  }
  if (bad && lane == 0) report(p.err, CP_ERR_DEVICE_BOUNDS);
#pragma unroll
  for (int h = 0; h < HR; ++h) {
    const float sum = warp_sum(l[h]);
    if (lane == 0) {
      parts.m[warp][h] = m[h];
      parts.l[warp][h] = sum;
    }
    float a[4];
    f2u(acc[h][0], a[0], a[1]);
    f2u(acc[h][1], a[2], a[3]);
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int o = NCH; o < 32; o <<= 1) a[e] += __shfl_xor_sync(0xffffffffu, a[e], o);
    if (vt == 0) *reinterpret_cast<float4*>(&parts.o[warp][h][4 * vc]) = make_float4(a[0], a[1], a[2], a[3]);
  }
  finish<float, D, HR>(p, parts, u.b, u.g, u.part, u.live);
}

template <int D>
cudaError_t launch_d(const ModParams& p, int dtype, cudaStream_t s) {
  if (dtype != CP_F32)
    return p.G <= 8 ? launch_decode(decode_mod_kernel<D, 1>, p, 0, 3, s) : launch_decode(decode_mod_kernel<D, 2>, p, 0, 2, s);
  const int per_sm = D == 64 && p.G <= 4 ? 3 : 2;
  return launch_decode(p.G <= 2 ? decode_mod_f32_kernel<D, 2> : p.G <= 4 ? decode_mod_f32_kernel<D, 4>
                                                                        : decode_mod_f32_kernel<D, 8>, p, 0, per_sm, s);
}

}  // namespace
}  // namespace cpattn

cudaError_t cp_launch_decode_mod(const cp_decode_args& a, const cp_score_mod& mod, float scale,
                                 const CpDecodeWorkspace* ws, void* out, float* out_lse, cudaStream_t s) {
  using namespace cpattn;
  const ModParams p = decode_mod_params(a, mod, scale, ws, out, out_lse);
  return a.head_dim == 64 ? launch_d<64>(p, a.dtype, s) : launch_d<128>(p, a.dtype, s);
}
