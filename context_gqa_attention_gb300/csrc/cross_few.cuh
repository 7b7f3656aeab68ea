// What the kernels for few query rows share (cross_few.cu: bf16, cross_f32.cu: f32; internal): the keys of a part, the
// joining of warps', CTAs' and parts' rows, and the launch.
#pragma once
#include <cuda.h>

#include "cross.cuh"

namespace cpattn {
namespace {

constexpr float kMaxGrowth = 8.f;            // log2 units the scores may exceed the running reference

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
// What W slices of the CTA's keys made of R rows, in shared memory: reference, sum, unnormalised row.
// PAD: what keeps the rows' banks apart, for the kernel's way of writing them.
template <int D, int W, int R, int PAD>
struct Slices {
  float o[W][R][D + PAD];
  float m[W][R], l[W][R];
};

// Slices -> the CTA's part; parts -> result, or to the workspace.  cluster: parts that meet in shared memory (1: none).
template <typename T, int D, int W, int R, int PAD>
CP_DEV void finish(const CrossParams& p, const CrossItem& w, Slices<D, W, R, PAD>& s, int cluster, int piece) {
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

// ------------------------------------------------------------------------------ warp-wide products
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

// The maps of k and v, a tile of whose keys is fetched at a time.
inline bool few_maps(const cp_cross_args& a, const CrossParams& p, int tile, CUtensorMap* k, CUtensorMap* v) {
  const unsigned long long cols = (unsigned long long)p.Hkv * a.head_dim;
  const bool any = p.Nkv > 0;  // (no key: never loaded from)
  const unsigned long long n = any ? p.Nkv : 1, ks = any ? a.k_stride : cols, vs = any ? a.v_stride : cols;
  const int elem = a.dtype == CP_F32 ? 4 : 2;
  const unsigned blocks = (unsigned)(a.head_dim * elem / 128);
  return cp_make_columns_map(k, any ? p.k : p.q, elem, cols * elem / 128, n, ks, tile, blocks) &&
         cp_make_columns_map(v, any ? p.v : p.q, elem, cols * elem / 128, n, vs, tile, blocks);
}

}  // namespace
}  // namespace cpattn

// The f32 kernel's side of the launch: CTAs of it on an SM for items of so many rows, and the launch of the items, each in
// `parts` parts of which `cluster` meet in shared memory.
int cp_cross_f32_ctas(int rows);
cudaError_t cp_launch_cross_f32(const cp_cross_args& a, const CrossPlan& plan, int parts, int cluster, float scale, void* ws,
                                size_t ws_bytes, void* out, float* lse, cudaStream_t s);
