// The 8-bit checkpoint's encoding of 32-column blocks, shared by its row pass
// and the gate/up GEMM's epilogue.
#pragma once

#include "common.h"
#include "tile.h"

namespace moe {
namespace save8 {

using tile::u32x2_t;

// Largest of the four lanes of a quad (quad permutations: lane xor 1, xor 2).
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xf, 0xf, true);
  v = o > v ? o : v;
  o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xf, 0xf, true);
  return o > v ? o : v;
}

// Codes of a lane's 8 values of a block whose four lanes call together (past
// the row's end: zeros), and the block's scale byte.  Magnitudes compare as
// integers, where infinities and NaN come out largest: such a block gets the
// scale byte 255 (NaN) and decodes to NaN throughout.
__device__ __forceinline__ u32x2_t encode8(const float (&f)[8], uint32_t* byte) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __float_as_uint(f[i]) & 0x7fffffffu;
    m = b > m ? b : m;
  }
  m = quad_max(m);
  // amax = c 2^e with c in [1, 2): X = e - 8, plus one when c > 1.75 (448 =
  // 1.75 2^8); a subnormal amax lies far below the clamp at -127
  int X = (int)(m >> 23) - 135 + ((m & 0x7fffffu) > 0x600000u ? 1 : 0);
  X = m == 0 ? 0 : (X < -127 ? -127 : X);
  const bool bad = m >= 0x7f800000u;
  *byte = bad ? 255u : (uint32_t)(X + 127);
  const float inv = __uint_as_float((uint32_t)(127 - X) << 23);  // 2^-X: exact products, at most 448
  u32x2_t q;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * h] * inv, f[4 * h + 1] * inv, 0, false);
    v = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * h + 2] * inv, f[4 * h + 3] * inv, v, true);
    q[h] = bad ? 0x7f7f7f7fu : (uint32_t)v;
  }
  return q;
}

}  // namespace save8
}  // namespace moe
