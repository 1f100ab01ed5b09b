// The router's projection and its gradients:
//   logits[t, e] = sum_c x[t, c] w[e, c]
//   dx[t, c] = dx_in[t, c] + sum_e dlogits[t, e] w[e, c]
//   dw[e, c] = sum_t dlogits[t, e] x[t, c]
// with float32 sums and one rounding each.  E is small beside d and T, so all
// three are bound by reading x (and dx_in) and writing dx once: at T = 16384,
// d = 2048, E = 128 in bf16 75 MB forward and 210 MB backward.
//
// A bf16 MFMA multiplies bf16 operands, and x and w are; a float32 dlogits is
// split into the bf16 nearest to it and the bf16 nearest to the rest, which
// leaves 2^-18 of it, and both parts are multiplied: the products stay bound by
// memory, and rounding dlogits to bf16 alone would cost 2^-9.  Float32 tensors
// go through the float32 MFMA.
//
// No product uses atomics: K or T is split over waves or work-groups and the
// parts are added in a fixed order.
#include "common.h"
#include "tile.h"

namespace moe {
namespace {

using tile::s16x4_t;
using tile::s16x8_t;
using tile::u32x4_t;

constexpr uint32_t kPast = 0xffffff00u;  // an offset past every buffer here: loads give 0
typedef __amdgpu_buffer_rsrc_t rsrc_t;
__device__ __forceinline__ rsrc_t buffer_of(const void* p, uint64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, (int)(uint32_t)bytes, 0x00020000);
}
__device__ __forceinline__ u32x4_t load16(rsrc_t r, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0);
}

// One value of a tensor in either type.
__device__ __forceinline__ float value_at(const float* p) { return *p; }
__device__ __forceinline__ float value_at(const bf16_t* p) { return bf2f(*p); }

// s + a b over the 16 (float) or 32 (bf16) values of K in two 16-byte operands.
template <typename T>
__device__ __forceinline__ f32x4_t mma16(u32x4_t a, u32x4_t b, f32x4_t s) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      s = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[i]), __uint_as_float(b[i]), s, 0, 0, 0);
    return s;
  } else {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b),
                                                   s, 0, 0, 0);
  }
}

// ------------------------------------------------------------------ forward
// Work-group: 16 MB tokens by 16 NB experts.  Each of the 8 waves computes the
// whole tile over every eighth 128-byte unit of K straight from memory (no
// operand is read twice by a work-group), and the eight parts meet in LDS.
constexpr int kFwdWaves = 8;

template <typename T, int MB, int NB>
__global__ __launch_bounds__(kFwdWaves * 64, 2) void router_fwd_kernel(const T* __restrict__ x,
                                                                       const T* __restrict__ w, int Tn, int E, int d,
                                                                       void* __restrict__ logits, int logits_f32) {
  constexpr int MR = MB * NB > 16 ? 16 / NB : MB;  // token blocks per LDS round: at most 128 KB
  extern __shared__ __align__(16) float red[];     // [wave][MR][NB][16 tokens][16 experts]
  const int lane = threadIdx.x & 63, wave = tile::wave_id(), q = lane >> 4, col = lane & 15;
  const int64_t t0 = (int64_t)blockIdx.x * (16 * MB);
  const int e0 = blockIdx.y * (16 * NB);
  const int bytes = d * (int)sizeof(T);
  const int tn = (int)(Tn - t0 < 16 * MB ? Tn - t0 : 16 * MB), en = min(E - e0, 16 * NB);
  // rows past the end of either buffer read as zeros
  const rsrc_t xb = buffer_of(x + t0 * d, (uint64_t)tn * bytes);
  const rsrc_t wb = buffer_of(w + (int64_t)e0 * d, (uint64_t)en * bytes);
  f32x4_t acc[MB][NB];
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int n = 0; n < NB; ++n) acc[m][n] = f32x4_t{0, 0, 0, 0};
  for (int off = wave * 128; off < bytes; off += kFwdWaves * 128) {
    u32x4_t xv[MB][2], wv[NB][2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int o = off + c * 64 + q * 16;
      const bool ok = o < bytes;
#pragma unroll
      for (int m = 0; m < MB; ++m) xv[m][c] = load16(xb, ok ? (uint32_t)((m * 16 + col) * bytes + o) : kPast);
#pragma unroll
      for (int n = 0; n < NB; ++n) wv[n][c] = load16(wb, ok ? (uint32_t)((n * 16 + col) * bytes + o) : kPast);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int n = 0; n < NB; ++n) acc[m][n] = mma16<T>(wv[n][c], xv[m][c], acc[m][n]);
  }
  // a lane holds 4 experts (rows 4 q ..) of token `col`
#pragma unroll
  for (int m0 = 0; m0 < MB; m0 += MR) {
    if (m0) __syncthreads();
#pragma unroll
    for (int m = 0; m < MR; ++m)
#pragma unroll
      for (int n = 0; n < NB; ++n)
        *(f32x4_t*)(red + (((wave * MR + m) * NB + n) * 16 + col) * 16 + q * 4) = acc[m0 + m][n];
    __syncthreads();
    for (int o = threadIdx.x; o < MR * NB * 64; o += kFwdWaves * 64) {  // four experts each
      const int e4 = o % (NB * 4), tt = o / (NB * 4);                  // consecutive threads: consecutive experts
      const int m = tt >> 4, c = tt & 15, n = e4 >> 2;
      f32x4_t s = {0, 0, 0, 0};
#pragma unroll
      for (int v = 0; v < kFwdWaves; ++v) {
        const f32x4_t p = *(const f32x4_t*)(red + (((v * MR + m) * NB + n) * 16 + c) * 16 + (e4 & 3) * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] += p[i];
      }
      const int t = (m0 + m) * 16 + c;
      if (t < tn) {
        const int64_t at = (t0 + t) * E + e0 + e4 * 4;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (e4 * 4 + i < en) {
            if (logits_f32) ((float*)logits)[at + i] = s[i];
            else ((bf16_t*)logits)[at + i] = f2bf(s[i]);
          }
      }
    }
  }
}

template <typename T, int MB, int NB>
hipError_t fwd(const LaunchCtx& c, const RouterArgs& a, void* logits) {
  constexpr int MR = MB * NB > 16 ? 16 / NB : MB;
  constexpr size_t smem = (size_t)kFwdWaves * MR * NB * 1024;
  HIP_RET(tile::allow_smem_once<router_fwd_kernel<T, MB, NB>>(smem));
  MOE_LAUNCH(c, "router_fwd", (router_fwd_kernel<T, MB, NB>),
             dim3((unsigned)cdiv(a.T, 16 * MB), (unsigned)cdiv(a.E, 16 * NB)), dim3(kFwdWaves * 64), smem,
             (const T*)a.x, (const T*)a.w, a.T, a.E, a.d, logits, a.logits_dtype == F32);
  return hipSuccess;
}

// The largest tile that still gives about a work-group per CU: a larger one
// reads w less often, a smaller one spreads a few tokens over more of the chip.
template <typename T, int NB>
hipError_t fwd_tokens(const LaunchCtx& c, const RouterArgs& a, void* logits) {
  const int64_t cols = cdiv(a.E, 16 * NB);
  if (cdiv(a.T, 64) * cols >= 192) return fwd<T, 4, NB>(c, a, logits);
  if (cdiv(a.T, 32) * cols >= 192) return fwd<T, 2, NB>(c, a, logits);
  if (NB == 1 || cdiv(a.T, 16) * cols >= 128) return fwd<T, 1, NB>(c, a, logits);
  if constexpr (NB > 1) return fwd_tokens<T, NB / 2>(c, a, logits);
  return hipSuccess;
}
template <typename T>
hipError_t fwd_any(const LaunchCtx& c, const RouterArgs& a, void* logits) {
  if (a.E <= 16) return fwd_tokens<T, 1>(c, a, logits);
  if (a.E <= 32) return fwd_tokens<T, 2>(c, a, logits);
  if (a.E <= 64) return fwd_tokens<T, 4>(c, a, logits);
  return fwd_tokens<T, 8>(c, a, logits);
}

// ------------------------------------------------- backward, first launch
// dw parts: work-group (E block of 128, d block of 128, run of tokens); steps
// of TS tokens pass through LDS as they lie in memory, [token][column], and a
// transposing LDS read (16-bit) or plain 4-byte reads (K = 4 float32 MFMA)
// hand the MFMA its token-contiguous operands.  Parts are float32 [run][E][d].
// The remaining work-groups write w's transpose [d][Ep] for the second launch
// (bf16: K = expert has to be contiguous there).
constexpr int kDwE = 128, kDwD = 128;

template <typename T> struct DwTile;
template <> struct DwTile<bf16_t> {
  static constexpr int TS = 64, STRIDE = 288;  // bytes a row: 256 + 32 (row r starts at bank 8 r)
};
template <> struct DwTile<float> {
  static constexpr int TS = 32, STRIDE = 576;  // 512 + 64 (16 r)
};

__device__ __forceinline__ void split_bf16(float v, bf16_t& hi, bf16_t& lo) {
  hi = f2bf(v);
  const float h = bf2f(hi);
  // beside an infinity the rest would be infinite or NaN; hi carries it alone
  lo = fabsf(h) < __builtin_huge_valf() ? f2bf(v - h) : (bf16_t)0;
}

template <typename T, typename LT>
__device__ __forceinline__ void dw_part(const RouterArgs& a, char* smem, int eb, int db, int run) {
  constexpr int TS = DwTile<T>::TS, ST = DwTile<T>::STRIDE;
  constexpr bool LO = sizeof(T) == 2 && sizeof(LT) == 4;  // dlogits has a second part
  constexpr int XV = TS * kDwD * (int)sizeof(T) / (512 * 16);  // 16-byte loads of x per thread
  constexpr int LV = TS * kDwE / 512;                          // dlogits values per thread, consecutive experts
  char* xs = smem;
  char* hs = smem + TS * ST;
  char* ls = smem + 2 * TS * ST;
  const int lane = threadIdx.x & 63, wave = tile::wave_id(), q = lane >> 4, col = lane & 15;
  const int e0 = eb * kDwE, d0 = db * kDwD;
  const int64_t tb = (int64_t)run * a.run_tokens;
  const int tn = (int)(a.T - tb < a.run_tokens ? a.T - tb : a.run_tokens);
  const int xrow = a.d * (int)sizeof(T);
  const T* xp = (const T*)a.x + tb * a.d;
  const LT* lp = (const LT*)a.dlogits + tb * a.E;
  // this thread's dlogits values: row lr, experts le .. le + LV of the block
  const int lr = (int)threadIdx.x / (kDwE / LV), le = ((int)threadIdx.x % (kDwE / LV)) * LV;
  const bool lvec = (a.E * sizeof(LT)) % 16 == 0 && ((uintptr_t)a.dlogits & 15) == 0 && e0 + le + LV <= a.E;
  u32x4_t xv[XV];
  float lv[LV];
  auto fetch = [&](int s) {  // tokens s .. s + TS of the run; zeros past its end and past E and d
#pragma unroll
    for (int i = 0; i < XV; ++i) {
      const int u = (int)threadIdx.x + i * 512;
      const int r = u / (kDwD * (int)sizeof(T) / 16), cb = (u % (kDwD * (int)sizeof(T) / 16)) * 16;
      xv[i] = u32x4_t{0, 0, 0, 0};
      if (s + r < tn && d0 * (int)sizeof(T) + cb < xrow)
        xv[i] = *(const u32x4_t*)((const char*)(xp + (int64_t)(s + r) * a.d + d0) + cb);
    }
    const LT* p = lp + (int64_t)(s + lr) * a.E + e0 + le;
#pragma unroll
    for (int i = 0; i < LV; ++i) lv[i] = 0.0f;
    if (s + lr < tn) {
      if (lvec) {
#pragma unroll
        for (int i = 0; i < LV * (int)sizeof(LT) / 16; ++i) {
          const u32x4_t v = ((const u32x4_t*)p)[i];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if constexpr (sizeof(LT) == 4) {
              lv[4 * i + j] = __uint_as_float(v[j]);
            } else {
              lv[8 * i + 2 * j] = __uint_as_float(v[j] << 16);
              lv[8 * i + 2 * j + 1] = __uint_as_float(v[j] & 0xffff0000u);
            }
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < LV; ++i)
          if (e0 + le + i < a.E) lv[i] = value_at(p + i);
      }
    }
  };
  const int we = (wave >> 2) * 64, wd = (wave & 3) * 32;  // this wave's 64 experts by 32 columns
  f32x4_t acc[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x4_t{0, 0, 0, 0};
  fetch(0);
  for (int s = 0; s < tn; s += TS) {
    __syncthreads();  // the previous step's reads are done
#pragma unroll
    for (int i = 0; i < XV; ++i) {
      const int u = (int)threadIdx.x + i * 512;
      const int r = u / (kDwD * (int)sizeof(T) / 16), cb = (u % (kDwD * (int)sizeof(T) / 16)) * 16;
      *(u32x4_t*)(xs + r * ST + cb) = xv[i];
    }
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < LV; i += 4)
        *(f32x4_t*)(hs + lr * ST + (le + i) * 4) = f32x4_t{lv[i], lv[i + 1], lv[i + 2], lv[i + 3]};
    } else {
#pragma unroll
      for (int i = 0; i < LV; i += 8) {
        u32x4_t h, l;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          bf16_t h0, l0, h1, l1;
          split_bf16(lv[i + 2 * j], h0, l0);
          split_bf16(lv[i + 2 * j + 1], h1, l1);
          h[j] = (uint32_t)h0 | ((uint32_t)h1 << 16);
          l[j] = (uint32_t)l0 | ((uint32_t)l1 << 16);
        }
        *(u32x4_t*)(hs + lr * ST + (le + i) * 2) = h;
        if constexpr (LO) *(u32x4_t*)(ls + lr * ST + (le + i) * 2) = l;
      }
    }
    __syncthreads();
    if (s + TS < tn) fetch(s + TS);  // lands while this step computes
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int k = 0; k < TS; k += 4) {
        float av[4], bv[2];
#pragma unroll
        for (int i = 0; i < 4; ++i) av[i] = *(const float*)(hs + (k + q) * ST + (we + i * 16 + col) * 4);
#pragma unroll
        for (int j = 0; j < 2; ++j) bv[j] = *(const float*)(xs + (k + q) * ST + (wd + j * 16 + col) * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(av[i], bv[j], acc[i][j], 0, 0, 0);
      }
    } else {
      // eight tokens 8 q .. of column `col`: the 16 lanes of a group read 4
      // tokens by 16 columns and get them transposed
      auto frag = [&](const char* base, int k, int c0) {
        const char* p = base + (k + q * 8 + (col >> 2)) * ST + (c0 + 4 * (col & 3)) * 2;
        const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)p);
        const s16x4_t hi =
            __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)(p + 4 * ST));
        return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
      };
#pragma unroll
      for (int k = 0; k < TS; k += 32) {
        bf16x8_t bv[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) bv[j] = frag(xs, k, wd + j * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bf16x8_t h = frag(hs, k, we + i * 16);
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(h, bv[j], acc[i][j], 0, 0, 0);
          if constexpr (LO) {
            const bf16x8_t l = frag(ls, k, we + i * 16);
#pragma unroll
            for (int j = 0; j < 2; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(l, bv[j], acc[i][j], 0, 0, 0);
          }
        }
      }
    }
  }
  float* part = a.parts + (int64_t)run * a.E * a.d;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int e = e0 + we + i * 16 + q * 4 + m, c = d0 + wd + j * 16 + col;
        if (e < a.E && c < a.d) part[(int64_t)e * a.d + c] = acc[i][j][m];
      }
}

// wt[c][e] = w[e][c] for 64 columns, experts up to the next multiple of 32
// (zeros past E).
__device__ __forceinline__ void transpose_w(const RouterArgs& a, char* smem, int cb) {
  bf16_t* s = (bf16_t*)smem;  // [32 experts][64 + 2 columns]
  const int c0 = cb * 64;
  for (int e0 = 0; e0 < a.Ep; e0 += 32) {
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * 64; i += 512) {
      const int e = i >> 6, c = i & 63;
      s[e * 66 + c] = e0 + e < a.E && c0 + c < a.d ? ((const bf16_t*)a.w)[(int64_t)(e0 + e) * a.d + c0 + c] : 0;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * 64; i += 512) {
      const int c = i >> 5, e = i & 31;
      if (c0 + c < a.d) a.wt[(int64_t)(c0 + c) * a.Ep + e0 + e] = s[e * 66 + c];
    }
  }
}

template <typename T, typename LT>
__global__ __launch_bounds__(512, 4) void router_dw_kernel(RouterArgs a) {
  constexpr int parts = sizeof(T) == 2 && sizeof(LT) == 4 ? 3 : 2;
  __shared__ __align__(16) char smem[parts * DwTile<T>::TS * DwTile<T>::STRIDE];
  int b = blockIdx.x;
  if (b < a.dw_groups) {
    const int db = b % a.d_blocks;
    b /= a.d_blocks;
    dw_part<T, LT>(a, smem, b % a.e_blocks, db, b / a.e_blocks);
  } else if constexpr (sizeof(T) == 2) {
    transpose_w(a, smem, b - a.dw_groups);
  }
}

// ------------------------------------------------ backward, second launch
// dx: one wave keeps the operands of 16 DT columns of d and up to 128 experts
// in registers and runs over blocks of 16 tokens, whose dlogits it reads from
// the caches.  The MFMA's rows are columns of d, taken so that a lane holds
// 4 DT consecutive ones of its token.
constexpr int kDxWaves = 4, kDxE = 128;

// Values e .. e + n of dlogits row t; zeros past E or T.
template <typename LT, int N>
__device__ __forceinline__ void dl_row(float (&v)[N], const RouterArgs& a, int64_t t, int e, bool vec) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.0f;
  if (t >= a.T) return;
  const LT* p = (const LT*)a.dlogits + t * a.E + e;
  if (vec && e + N <= a.E) {
    constexpr int PER = 16 / (int)sizeof(LT);
    if constexpr (N >= PER) {
#pragma unroll
      for (int i = 0; i < N / PER; ++i) {
        const u32x4_t u = ((const u32x4_t*)p)[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (sizeof(LT) == 4) {
            v[4 * i + j] = __uint_as_float(u[j]);
          } else {
            v[8 * i + 2 * j] = __uint_as_float(u[j] << 16);
            v[8 * i + 2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
          }
        }
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (e + i < a.E) v[i] = value_at(p + i);
}

template <typename T, typename LT>
__device__ __forceinline__ void dx_part(const RouterArgs& a, int cb, int run) {
  constexpr bool BF = sizeof(T) == 2;
  constexpr bool LO = BF && sizeof(LT) == 4;
  constexpr int DT = BF ? 4 : 2;            // tiles of 16 columns per wave
  constexpr int KS = BF ? 32 : 16;          // experts per 16-byte operand step
  constexpr int NK = kDxE / KS;
  const int lane = threadIdx.x & 63, wave = tile::wave_id(), q = lane >> 4, col = lane & 15;
  const int c0 = (cb * kDxWaves + wave) * 16 * DT;
  if (c0 >= a.d) return;
  const bool vec = (a.E * sizeof(LT)) % 16 == 0 && ((uintptr_t)a.dlogits & 15) == 0;
  // operand row `col` of tile j is column c0 + (col / 4) 4 DT + 4 j + col % 4,
  // so that result rows 4 q .. of the tiles are 4 DT consecutive columns
  u32x4_t wv[DT][NK];
  auto load_w = [&](int e0) {
#pragma unroll
    for (int j = 0; j < DT; ++j) {
      const int c = c0 + (col >> 2) * 4 * DT + 4 * j + (col & 3);
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        wv[j][k] = u32x4_t{0, 0, 0, 0};
        if constexpr (BF) {
          const int e = e0 + k * KS + q * 8;
          if (c < a.d && e < a.Ep) wv[j][k] = *(const u32x4_t*)(a.wt + (int64_t)c * a.Ep + e);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int e = e0 + k * KS + q * 4 + i;
            if (c < a.d && e < a.E) wv[j][k][i] = __float_as_uint(((const float*)a.w)[(int64_t)e * a.d + c]);
          }
        }
      }
    }
  };
  const int ebs = (a.E + kDxE - 1) / kDxE;
  if (ebs == 1) load_w(0);
  const int64_t tb = (int64_t)run * a.dx_tokens, te = tb + a.dx_tokens < a.T ? tb + a.dx_tokens : a.T;
  const int cl = c0 + q * 4 * DT;  // this lane's columns
  for (int64_t t0 = tb; t0 < te; t0 += 16) {
    const int64_t t = t0 + col;
    const bool live = t < te;
    // d is a multiple of 8, so 8-column groups are in or out together
    u32x4_t in[DT * 4 * sizeof(T) / 16];
    if (a.dx_in) {
#pragma unroll
      for (int i = 0; i < (int)(DT * 4 * sizeof(T) / 16); ++i) {
        const int c = cl + i * (16 / (int)sizeof(T));
        in[i] = u32x4_t{0, 0, 0, 0};
        if (live && c < a.d) in[i] = *(const u32x4_t*)((const T*)a.dx_in + t * a.d + c);
      }
    }
    f32x4_t acc[DT];
#pragma unroll
    for (int j = 0; j < DT; ++j) acc[j] = f32x4_t{0, 0, 0, 0};
    for (int eb = 0; eb < ebs; ++eb) {
      const int e0 = eb * kDxE;
      if (ebs > 1) load_w(e0);
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        if (e0 + k * KS < a.E) {
          if constexpr (BF) {
            float v[8];
            dl_row<LT, 8>(v, a, live ? t : a.T, e0 + k * KS + q * 8, vec);
            u32x4_t h, l;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              bf16_t h0, l0, h1, l1;
              split_bf16(v[2 * i], h0, l0);
              split_bf16(v[2 * i + 1], h1, l1);
              h[i] = (uint32_t)h0 | ((uint32_t)h1 << 16);
              l[i] = (uint32_t)l0 | ((uint32_t)l1 << 16);
            }
#pragma unroll
            for (int j = 0; j < DT; ++j) acc[j] = mma16<T>(wv[j][k], h, acc[j]);
            if constexpr (LO) {
#pragma unroll
              for (int j = 0; j < DT; ++j) acc[j] = mma16<T>(wv[j][k], l, acc[j]);
            }
          } else {
            float v[4];
            dl_row<LT, 4>(v, a, live ? t : a.T, e0 + k * KS + q * 4, vec);
            const u32x4_t b = {__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                               __float_as_uint(v[3])};
#pragma unroll
            for (int j = 0; j < DT; ++j) acc[j] = mma16<T>(wv[j][k], b, acc[j]);
          }
        }
      }
    }
    if (live) {
#pragma unroll
      for (int i = 0; i < (int)(DT * 4 * sizeof(T) / 16); ++i) {
        constexpr int PER = 16 / (int)sizeof(T);
        const int c = cl + i * PER;
        if (c < a.d) {
          u32x4_t o;
          if constexpr (BF) {
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              float lo = acc[(i * PER + 2 * m) / 4][(2 * m) & 3], hi = acc[(i * PER + 2 * m) / 4][(2 * m + 1) & 3];
              if (a.dx_in) {
                lo += __uint_as_float(in[i][m] << 16);
                hi += __uint_as_float(in[i][m] & 0xffff0000u);
              }
              o[m] = pack_bf16x2(lo, hi);
            }
          } else {
#pragma unroll
            for (int m = 0; m < 4; ++m)
              o[m] = __float_as_uint(a.dx_in ? acc[i][m] + __uint_as_float(in[i][m]) : acc[i][m]);
          }
          *(u32x4_t*)((T*)a.dx + t * a.d + c) = o;
        }
      }
    }
  }
}

// dw = the sum of the parts, in run order; 4 values a thread.
template <typename T>
__device__ __forceinline__ void join_dw(const RouterArgs& a, int b) {
  const int64_t n = (int64_t)a.E * a.d, i = ((int64_t)b * kDxWaves * 64 + threadIdx.x) * 4;
  if (i >= n) return;  // d is a multiple of 8: whole groups of 4
  f32x4_t s = {0, 0, 0, 0};
  for (int r = 0; r < a.runs; ++r) {
    const f32x4_t v = *(const f32x4_t*)(a.parts + r * n + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] += v[j];
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) ((T*)a.dw)[i + j] = from_f32<T>(s[j]);
}

template <typename T, typename LT>
__global__ __launch_bounds__(kDxWaves * 64) void router_dx_kernel(RouterArgs a) {
  const int b = blockIdx.x;
  if (b < a.dx_groups) dx_part<T, LT>(a, b % a.dx_blocks, b / a.dx_blocks);
  else join_dw<T>(a, b - a.dx_groups);
}

template <typename T, typename LT>
hipError_t bwd(const LaunchCtx& c, const RouterArgs& a) {
  const unsigned tr = sizeof(T) == 2 ? (unsigned)cdiv(a.d, 64) : 0;
  MOE_LAUNCH(c, "router_dw", (router_dw_kernel<T, LT>), dim3((unsigned)a.dw_groups + tr), dim3(512), 0, a);
  MOE_LAUNCH(c, "router_dx", (router_dx_kernel<T, LT>),
             dim3((unsigned)(a.dx_groups + cdiv((int64_t)a.E * a.d, kDxWaves * 256))), dim3(kDxWaves * 64), 0, a);
  return hipSuccess;
}

}  // namespace

RouterPlan router_plan(int64_t T, int64_t d, int64_t E, int dtype) {
  RouterPlan p;
  const int step = dtype == F32 ? DwTile<float>::TS : DwTile<bf16_t>::TS;
  // two work-groups per CU, in whole steps, at least four of them a run (the
  // parts cost E d floats of traffic each way)
  const int64_t tiles = cdiv(d, kDwD) * cdiv(E, kDwE);
  const int64_t want = cdiv(512, tiles) < 1 ? 1 : cdiv(512, tiles);
  int64_t steps = cdiv(cdiv(T, step), want);
  if (steps < 4) steps = 4;
  p.run_tokens = steps * step;
  p.runs = cdiv(T, p.run_tokens);
  return p;
}

hipError_t launch_router_fwd(const LaunchCtx& c, const RouterArgs& a, void* logits) {
  return a.dtype == F32 ? fwd_any<float>(c, a, logits) : fwd_any<bf16_t>(c, a, logits);
}

hipError_t launch_router_bwd(const LaunchCtx& c, RouterArgs a) {
  a.d_blocks = (int)cdiv(a.d, kDwD);
  a.e_blocks = (int)cdiv(a.E, kDwE);
  a.dw_groups = a.d_blocks * a.e_blocks * a.runs;
  a.dx_blocks = (int)cdiv(a.d, 16 * (a.dtype == F32 ? 2 : 4) * kDxWaves);
  // four work-groups per CU, at least two token blocks each
  int64_t tok = cdiv(cdiv((int64_t)a.T * a.dx_blocks, 1024), 16) * 16;
  if (tok < 32) tok = 32;
  a.dx_tokens = (int)tok;
  a.dx_groups = a.dx_blocks * (int)cdiv(a.T, tok);
  if (a.dtype == F32) return a.logits_dtype == F32 ? bwd<float, float>(c, a) : bwd<float, bf16_t>(c, a);
  return a.logits_dtype == F32 ? bwd<bf16_t, float>(c, a) : bwd<bf16_t, bf16_t>(c, a);
}

}  // namespace moe
