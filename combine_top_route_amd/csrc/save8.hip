// 8-bit activation checkpoint: the gate/up pre-activations H = [g | u] of the
// expert-sorted rows, kept between forward and backward as e4m3 codes with one
// E8M0 scale per 32 columns of either half (the MXFP8 row encoding: X the
// smallest exponent with amax <= 448 2^X, the code of h 2^-X to nearest even):
// 2 I + 2 ceil(I/32) bytes a row instead of the 6 I of a bf16 H and Aw.  Aw is
// not kept: the backward's row pass rebuilds it from the decoded H.
//
//   forward:  codes, scales = encode(H);  aw = w silu(min(g, L)) clamp(u, -L, L)
//   backward: g, u = decode;  s = sigmoid(min(g, L));  a = silu u;  dw = <G, a>;
//             aw = w a;  dA = w G;  dg = dA u s (1 + g (1 - s));  du = dA g s
//             (zero where a clamp is active)
//
// Both are one pass over the rows, bound by memory: at I = 768 in bf16 the
// forward moves 6.2 KB a row and the backward 7.7 KB.  A wave takes a row, or
// several short ones; a lane takes 8 columns of both halves, so a block of 32 is
// four neighbouring lanes, whose largest magnitude two DPP steps find.
#include "common.h"
#include "save8.h"
#include "tile.h"

namespace moe {
namespace {

using save8::encode8;
using tile::u32x2_t;
using tile::u32x4_t;

template <typename T>
__device__ __forceinline__ void load8(float (&f)[8], const T* p) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u32x4_t v = *(const u32x4_t*)(p + 4 * h);
#pragma unroll
      for (int i = 0; i < 4; ++i) f[4 * h + i] = __uint_as_float(v[i]);
    }
  } else {
    const u32x4_t v = *(const u32x4_t*)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(v[i] << 16);
      f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    }
  }
}

// NT: non-temporal stores, where a launch writes more than the last-level cache
// holds (131072 rows of I = 768 in bf16: forward 142 us without, 134 with;
// backward 176 and 168); a smaller result is left there for its reader.
template <bool NT, typename V>
__device__ __forceinline__ void put(V v, V* p) {
  if constexpr (NT) __builtin_nontemporal_store(v, p);
  else *p = v;
}
constexpr int64_t kLastLevelCache = int64_t(256) << 20;

template <bool NT, typename T>
__device__ __forceinline__ void store8(T* p, const float (&f)[8]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      u32x4_t v;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __float_as_uint(f[4 * h + i]);
      put<NT>(v, (u32x4_t*)(p + 4 * h));
    }
  } else {
    u32x4_t v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
    put<NT>(v, (u32x4_t*)p);
  }
}

__device__ __forceinline__ void decode8(float (&f)[8], u32x2_t q, uint32_t byte) {
  // 2^X; byte 0 is 2^-127, a subnormal, byte 255 NaN
  const float s = __uint_as_float(byte == 0 ? 0x00400000u : (byte == 255u ? 0x7fc00000u : byte << 23));
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[h], false);
    const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[h], true);
    f[4 * h] = lo[0] * s;
    f[4 * h + 1] = lo[1] * s;
    f[4 * h + 2] = hi[0] * s;
    f[4 * h + 3] = hi[1] * s;
  }
}

template <typename T, bool NT>
__global__ __launch_bounds__(256) void save8_kernel(const T* __restrict__ H, const float* __restrict__ topk_w,
                                                    const int32_t* __restrict__ src_of, int R, int I, int lsh,
                                                    float lim, T* __restrict__ aw, uint8_t* __restrict__ codes,
                                                    uint8_t* __restrict__ scales) {
  const int L = 1 << lsh, r = ((int)(blockIdx.y * gridDim.x + blockIdx.x) << (8 - lsh)) + (int)(threadIdx.x >> lsh);
  if (r >= R) return;
  const int lane = (int)threadIdx.x & (L - 1);
  const int nb = (I + 31) / 32;
  const float wr = aw ? topk_w[src_of[r]] : 0.0f;
  const T* Hr = H + (int64_t)r * 2 * I;
  uint8_t* cr = codes + (int64_t)r * 2 * I;
  uint8_t* sr = scales + (int64_t)r * 2 * nb;
  for (int c = lane; c < nb * 4; c += L) {
    const bool in = c * 8 < I;  // I is a multiple of 8: a lane's columns are in or out together
    float g[8] = {}, u[8] = {};
    if (in) {
      load8(g, Hr + c * 8);
      load8(u, Hr + I + c * 8);
    }
    uint32_t bg, bu;
    const u32x2_t qg = encode8(g, &bg), qu = encode8(u, &bu);
    if (in) {
      put<NT>(qg, (u32x2_t*)(cr + c * 8));
      put<NT>(qu, (u32x2_t*)(cr + I + c * 8));
      if (aw) {
        float a[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float gc = clip_gate(g[i], lim);
          a[i] = wr * (gc * sigmoidf_(gc) * clip_up(u[i], lim));
        }
        store8<NT>(aw + (int64_t)r * I + c * 8, a);
      }
    }
    if ((c & 3) == 0) {
      sr[c >> 2] = (uint8_t)bg;
      sr[nb + (c >> 2)] = (uint8_t)bu;
    }
  }
}

template <typename T, bool NT>
__global__ __launch_bounds__(256) void swiglu_bwd8_kernel(const T* __restrict__ G, const uint8_t* __restrict__ codes,
                                                          const uint8_t* __restrict__ scales,
                                                          const float* __restrict__ topk_w,
                                                          const int32_t* __restrict__ src_of, int R, int I, int lsh,
                                                          float lim, T* __restrict__ dH, T* __restrict__ aw,
                                                          float* __restrict__ dw) {
  const int L = 1 << lsh, r = ((int)(blockIdx.y * gridDim.x + blockIdx.x) << (8 - lsh)) + (int)(threadIdx.x >> lsh);
  if (r >= R) return;
  const int lane = (int)threadIdx.x & (L - 1);
  const int nb = (I + 31) / 32;
  const float wr = topk_w[src_of[r]];
  const uint8_t* cr = codes + (int64_t)r * 2 * I;
  const uint8_t* sr = scales + (int64_t)r * 2 * nb;
  const T* Gr = G + (int64_t)r * I;
  T* dr = dH + (int64_t)r * 2 * I;
  float part = 0.0f;
  for (int c = lane; c * 8 < I; c += L) {
    float gv[8], g[8], u[8], a[8], dg[8], du[8];
    load8(gv, Gr + c * 8);
    decode8(g, *(const u32x2_t*)(cr + c * 8), sr[c >> 2]);
    decode8(u, *(const u32x2_t*)(cr + I + c * 8), sr[nb + (c >> 2)]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float gc = clip_gate(g[i], lim), uc = clip_up(u[i], lim);
      const float s = sigmoidf_(gc);
      const float act = gc * s * uc;
      part += gv[i] * act;
      const float dA = wr * gv[i];
      a[i] = wr * act;
      dg[i] = g[i] > lim ? 0.0f : dA * uc * s * (1.0f + gc * (1.0f - s));
      du[i] = fabsf(u[i]) > lim ? 0.0f : dA * gc * s;
    }
    store8<NT>(dr + c * 8, dg);
    store8<NT>(dr + I + c * 8, du);
    if (aw) store8<NT>(aw + (int64_t)r * I + c * 8, a);
  }
  for (int off = L / 2; off >= 1; off >>= 1) part += __shfl_xor(part, off, kWave);
  if (lane == 0) dw[r] = part;
}

// log2 of the lanes that a row takes: 64, or fewer where its columns fill no more
// (38304 rows of I = 112 in bf16, backward: 24 us with 64, 10 with 16).
int row_lanes(int I) { return I > 256 ? 6 : I > 128 ? 5 : I > 64 ? 4 : 3; }

// The work-groups of R rows, in two dimensions: a launch takes less than 2^32
// threads in one, and rows at a wave each reach 2^33.
dim3 row_groups(int R, int I) {
  const int64_t n = cdiv(R, 256 >> row_lanes(I)), x = n < (1 << 23) ? n : 1 << 23;
  return dim3((unsigned)x, (unsigned)cdiv(n, x));
}

template <typename T, bool NT>
hipError_t save(const LaunchCtx& c, const void* H, const float* topk_w, const int32_t* src_of, int R, int I, float lim,
                void* aw, uint8_t* codes, uint8_t* scales) {
  MOE_LAUNCH(c, "swiglu_save8", (save8_kernel<T, NT>), row_groups(R, I), dim3(256), 0,
             (const T*)H, topk_w, src_of, R, I, row_lanes(I), lim, (T*)aw, codes, scales);
  return hipSuccess;
}
template <typename T, bool NT>
hipError_t backward(const LaunchCtx& c, const void* G, const uint8_t* codes, const uint8_t* scales,
                    const float* topk_w, const int32_t* src_of, int R, int I, float lim, void* dH, void* aw,
                    float* dw) {
  MOE_LAUNCH(c, "swiglu_bwd8", (swiglu_bwd8_kernel<T, NT>), row_groups(R, I), dim3(256), 0,
             (const T*)G, codes, scales, topk_w, src_of, R, I, row_lanes(I), lim, (T*)dH, (T*)aw, dw);
  return hipSuccess;
}
}  // namespace

hipError_t launch_save8(const LaunchCtx& c, int dtype, const void* H, const float* topk_w, const int32_t* src_of,
                        int R, int I, float lim, void* aw, uint8_t* codes, uint8_t* scales) {
  const int es = dtype == F32 ? 4 : 2;
  const bool nt = (int64_t)R * I * (2 + (aw ? es : 0)) > kLastLevelCache;
  const auto run = dtype == F32 ? (nt ? save<float, true> : save<float, false>)
                                : (nt ? save<bf16_t, true> : save<bf16_t, false>);
  return run(c, H, topk_w, src_of, R, I, lim, aw, codes, scales);
}

hipError_t launch_swiglu_bwd8(const LaunchCtx& c, int dtype, const void* G, const uint8_t* codes,
                              const uint8_t* scales, const float* topk_w, const int32_t* src_of, int R, int I,
                              float lim, void* dH, void* aw, float* dw) {
  const int es = dtype == F32 ? 4 : 2;
  const bool nt = (int64_t)R * I * (aw ? 3 : 2) * es > kLastLevelCache;
  const auto run = dtype == F32 ? (nt ? backward<float, true> : backward<float, false>)
                                : (nt ? backward<bf16_t, true> : backward<bf16_t, false>);
  return run(c, G, codes, scales, topk_w, src_of, R, I, lim, dH, aw, dw);
}

}  // namespace moe
