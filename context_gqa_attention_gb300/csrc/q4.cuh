// The 4-bit K/V page record shared by the kernels that write, read and attend it (layout in
// include/cpattn.h): one kv head's 16 tokens in 9 d bytes, 16 rows of d / 2 bytes and then, per
// token and group of 64 dims, the bf16 pair (scale, minimum).  value = minimum + scale * code.
#pragma once

#include "common.cuh"

namespace cpattn {

constexpr int kQ4Page = 16;   // tokens per record
constexpr int kQ4Group = 64;  // dims that share a scale and a minimum

CP_DEV long long q4_record_bytes(int d) { return 9ll * d; }

// Word (8 codes, 32 bits) of a row that holds dims 8 c .. 8 c + 7.  With two groups their words
// alternate, so that a thread's 8- or 16-byte piece of a row holds as much of one group as of the
// other: the attention kernel applies a group's scale once per accumulator, after its MMAs.
template <int D>
CP_DEV int q4_word(int c) {
  if constexpr (D == 64) return c;
  else return 2 * (c & 7) + (c >> 3);
}

CP_DEV float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
CP_DEV float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

}  // namespace cpattn
