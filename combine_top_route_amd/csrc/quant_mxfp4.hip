// MXFP4 encoding of weights (OCP microscaling): e2m1 codes, two to a byte, the
// even column in the low half, and one E8M0 scale byte per 32 columns of a row.
// For a block with largest magnitude amax the scale is 2^X with X the smallest
// integer such that amax <= 6 2^X (so nothing saturates; X >= -127, and 0 for a
// block of zeros); each value becomes the code nearest to x / 2^X, ties to even.
// A block with an infinity or NaN gets the scale byte 255 (NaN).
//
// Bound by memory: 2 bytes read and 17/32 written a value.  A lane takes 8
// values (16 bytes), four lanes a block, whose largest magnitude they exchange
// by DPP (403 M values, the gate/up weights of 128 experts at d = 2048, I = 768:
// 162 us, 6.3 TB/s).
#include "common.h"
#include "save8.h"
#include "tile.h"

namespace moe {
namespace {

using tile::u32x4_t;

__global__ __launch_bounds__(256) void quant_mxfp4_kernel(const u32x4_t* __restrict__ src, int64_t n,
                                                          uint32_t* __restrict__ q, uint8_t* __restrict__ s) {
  const int64_t i = folded_block() * 256 + threadIdx.x;
  if (i >= n) return;  // n is a multiple of 4: whole blocks leave together
  const u32x4_t v = __builtin_nontemporal_load(src + i);
  float f[8];
  uint32_t m = 0;  // magnitudes compare as integers; infinities and NaN come out largest
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t b = j & 1 ? v[j >> 1] & 0xffff0000u : v[j >> 1] << 16;
    f[j] = __uint_as_float(b);
    m = max(m, b & 0x7fffffffu);
  }
  m = save8::quad_max(m);
  // amax = c 2^e with c in [1, 2): X = e - 2, plus one when c > 1.5 (6 = 1.5
  // 2^2); a subnormal amax lies far below the clamp at -127
  int X = (int)(m >> 23) - 129 + ((m & 0x7fffffu) > 0x400000u ? 1 : 0);
  X = m == 0 ? 0 : (X < -127 ? -127 : X);
  const bool bad = m >= 0x7f800000u;
  const float inv = __uint_as_float((uint32_t)(127 - X) << 23);  // 2^-X: exact products, at most 6
  uint32_t code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, f[0] * inv, f[1] * inv, 1.0f, 0);
  code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, f[2] * inv, f[3] * inv, 1.0f, 1);
  code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, f[4] * inv, f[5] * inv, 1.0f, 2);
  code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, f[6] * inv, f[7] * inv, 1.0f, 3);
  q[i] = bad ? 0x77777777u : code;
  if ((threadIdx.x & 3) == 0) s[i >> 2] = bad ? 255 : (uint8_t)(X + 127);
}

}  // namespace

hipError_t launch_quant_mxfp4(const LaunchCtx& c, const void* src, int64_t values, uint8_t* q, uint8_t* s) {
  const int64_t n = values / 8;
  MOE_LAUNCH(c, "quant_mxfp4", quant_mxfp4_kernel, folded_grid(cdiv(n, 256)), dim3(256), 0, (const u32x4_t*)src, n,
             (uint32_t*)q, s);
  return hipSuccess;
}

}  // namespace moe
