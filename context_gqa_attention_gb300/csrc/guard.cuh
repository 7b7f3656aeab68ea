// Infinities and NaN in V that some row does not see (internal).
#pragma once

#include "common.cuh"
#include "sm100.cuh"

namespace cpattn {
namespace {

// ------------------------------------------------------------------------------ V guard
// 0 times an infinity or a NaN is NaN, so such a V element must not meet a row that does not see
// its key.  In a key tile that some row of the CTA sees only in part, the two guard warps clear
// the V rows behind the last key that any row sees (another sequence's tokens, or anything behind
// the last sequence), and in the others every element that is not finite; they say whether there
// was one, and the rows that do see it add it back at the end (see restore).
// Nearly always there is none, so the tile is only read, several vectors at a time (the MMAs wait for this: cleaning
// each vector as it came took 5k cycles a tile, longer than the tile's softmax).
template <int D, int BN>
CP_DEV bool guard_v(uint8_t* sv, int last, int part) {
  // 16-byte vectors of the tile's two (one) 64-column blocks, 128 rows of 128 bytes each; the
  // swizzle only permutes the vectors within a row
  constexpr int kVec = BN * D * 2 / 16, kAtOnce = 8;
  uint4* v = reinterpret_cast<uint4*>(sv);
  // exponent of all ones: adding one to it carries into the sign's place
  auto odd = [](uint32_t w) -> uint32_t { return (w & 0x7f807f80u) + 0x00800080u; };
  if (last < BN)
    for (int i = part; i < kVec; i += 64)
      if (((i >> 3) & (BN - 1)) >= last) v[i] = make_uint4(0u, 0u, 0u, 0u);
  uint32_t any = 0;
#pragma unroll 1
  for (int i = part; i < kVec; i += 64 * kAtOnce) {
    uint4 x[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) x[k] = v[i + 64 * k];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) any |= (odd(x[k].x) | odd(x[k].y)) | (odd(x[k].z) | odd(x[k].w));
  }
  if ((any & 0x80008000u) == 0u) return false;
#pragma unroll 1
  for (int i = part; i < kVec; i += 64) {
    uint32_t* w = reinterpret_cast<uint32_t*>(v + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] &= ~(((odd(w[e]) & 0x80008000u) >> 15) * 0xffffu);  // 0xffff in each half that is not finite
  }
  return true;
}

// What the guard took out of V for a row that sees it: p > 0 times an infinity or a NaN is that
// infinity or NaN, whatever p is.  Rare and slow: the row's keys within the unclean tiles.
template <int D>
CP_DEV void restore(float (&o)[32], const __nv_bfloat16* v, long long stride, int col, int k0, int k1) {
  for (int j = k0; j < k1; ++j)
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const float x = __bfloat162float(v[(long long)j * stride + col + k]);
      if (!isfinite(x)) o[k] += x;
    }
}

}  // namespace
}  // namespace cpattn
