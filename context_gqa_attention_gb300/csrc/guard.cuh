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
template <int D, int BN>
CP_DEV bool guard_v(uint8_t* sv, int last, int part) {
  bool unclean = false;
  // 16-byte vectors of the tile's two (one) 64-column blocks, 128 rows of 128 bytes each; the
  // swizzle only permutes the vectors within a row
  constexpr int kVec = BN * D * 2 / 16;
#pragma unroll 4
  for (int i = part; i < kVec; i += 64) {
    const int row = (i >> 3) & (BN - 1);
    uint4* p = reinterpret_cast<uint4*>(sv) + i;
    if (row >= last) {
      *p = make_uint4(0u, 0u, 0u, 0u);
      continue;
    }
    uint4 x = *p;
    uint32_t* w = reinterpret_cast<uint32_t*>(&x);
    uint32_t any = 0;
    // exponent of all ones: adding one to it carries into the sign's place
#pragma unroll
    for (int e = 0; e < 4; ++e) any |= ((w[e] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
    if (any != 0u) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t bad = ((w[e] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
        w[e] &= ~((bad >> 15) * 0xffffu);  // 0xffff in each half that is not finite
      }
      *p = x;
      unclean = true;
    }
  }
  return unclean;
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
