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
// leaves 2^-17 of it, and both parts are multiplied: the products stay bound by
// memory, and rounding dlogits to bf16 alone would cost 2^-8.  Float32 tensors
// go through the float32 MFMA.
//
// No product uses atomics: K or T is split over waves or work-groups and the
// parts are added in a fixed order.
#include <type_traits>

#include "common.h"
#include "rowload.h"
#include "tile.h"

namespace moe {
namespace {

using namespace rowload;
using tile::s16x4_t;
using tile::s16x8_t;
using tile::u32x4_t;

// Place b of n work-groups: the eight XCDs, which take work-groups in turn, get
// consecutive places, here the column blocks of a few runs of tokens, whose
// dlogits they share in their L2 (dx 40 us at the size above in plain order,
// 35 in this one).
__device__ __forceinline__ int xcd_share(int b, int n) {
  const int x = b & 7;
  return x * (n >> 3) + min(x, n & 7) + (b >> 3);
}

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
// whole tile over every eighth 128-byte unit of K from its own loads (no
// operand is read twice by a work-group), and the eight parts meet in LDS.
constexpr int kFwdWaves = 8;

template <int MB, int NB>
constexpr size_t fwd_smem() {  // the waves' turning space, then MR token blocks of parts
  constexpr int MR = MB * NB > 16 ? 16 / NB : MB;
  const size_t turn = (size_t)kFwdWaves * 4096, parts = (size_t)kFwdWaves * MR * NB * 1024;
  return turn > parts ? turn : parts;
}

template <typename T, int MB, int NB>
__global__ __launch_bounds__(kFwdWaves * 64, 2) void router_fwd_kernel(const T* __restrict__ x,
                                                                       const T* __restrict__ w, int Tn, int E, int d,
                                                                       void* __restrict__ logits, int logits_f32) {
  constexpr int MR = MB * NB > 16 ? 16 / NB : MB;  // token blocks per LDS round: at most 128 KB
  extern __shared__ __align__(16) char smem[];
  const int lane = threadIdx.x & 63, wave = tile::wave_id(), q = lane >> 4, col = lane & 15;
  const int64_t t0 = (int64_t)blockIdx.x * (16 * MB);
  const int e0 = blockIdx.y * (16 * NB);
  const int bytes = d * (int)sizeof(T);
  const int tn = (int)(Tn - t0 < 16 * MB ? Tn - t0 : 16 * MB), en = min(E - e0, 16 * NB);
  // rows past the end of either buffer read as zeros
  const rsrc_t xb = buffer_of(x + t0 * d, (uint64_t)tn * bytes);
  const rsrc_t wb = buffer_of(w + (int64_t)e0 * d, (uint64_t)en * bytes);
  lds_t* turn = (lds_t*)smem + wave * 4096;
  const uint32_t row[2] = {(uint32_t)load_row(0) * bytes, (uint32_t)load_row(1) * bytes};
  f32x4_t acc[MB][NB];
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int n = 0; n < NB; ++n) acc[m][n] = f32x4_t{0, 0, 0, 0};
  for (int off = wave * 128; off < bytes; off += kFwdWaves * 128) {
    u32x4_t xv[MB][2], wv[MB * NB > 16 ? NB / 2 : NB][2];
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      const uint32_t r[2] = {row[0] + m * 16 * bytes, row[1] + m * 16 * bytes};
      load_rows(xv[m], xb, r, off, bytes);
    }
    // at the largest tile half of w's rows wait for x's registers
    constexpr int NH = MB * NB > 16 ? NB / 2 : NB;
    auto load_w = [&](int n) {
      const uint32_t r[2] = {row[0] + n * 16 * bytes, row[1] + n * 16 * bytes};
      load_rows(wv[n % NH], wb, r, off, bytes);
    };
#pragma unroll
    for (int n = 0; n < NH; ++n) load_w(n);
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      put_rows(turn + (m & 1) * 2048, xv[m]);
#pragma unroll
      for (int c = 0; c < 2; ++c) xv[m][c] = get_chunk(turn + (m & 1) * 2048, col, 4 * c + q);
    }
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      put_rows(turn + (n & 1) * 2048, wv[n % NH]);
      if (n + NH < NB) load_w(n + NH);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const u32x4_t wf = get_chunk(turn + (n & 1) * 2048, col, 4 * c + q);
#pragma unroll
        for (int m = 0; m < MB; ++m) acc[m][n] = mma16<T>(wf, xv[m][c], acc[m][n]);
      }
    }
  }
  // parts [wave][MR][NB][16 tokens][16 experts]: a lane holds 4 experts (rows
  // 4 q ..) of token `col`; threads then add them 16 bytes by 16 bytes as they lie
  float* red = (float*)smem;
  const bool vec = E % 4 == 0;
#pragma unroll
  for (int m0 = 0; m0 < MB; m0 += MR) {
    __syncthreads();
#pragma unroll
    for (int m = 0; m < MR; ++m)
#pragma unroll
      for (int n = 0; n < NB; ++n)
        *(f32x4_t*)(red + ((wave * MR + m) * NB + n) * 256 + part_at(col, q)) = acc[m0 + m][n];
    __syncthreads();
    for (int o = threadIdx.x; o < MR * NB * 64; o += kFwdWaves * 64) {
      f32x4_t s = {0, 0, 0, 0};
#pragma unroll
      for (int v = 0; v < kFwdWaves; ++v) {
        const f32x4_t p =
            *(const f32x4_t*)(red + (v * MR * NB + (o >> 6)) * 256 + part_at((o >> 2) & 15, o & 3));
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] += p[i];
      }
      const int e = (o >> 6) % NB * 16 + (o & 3) * 4, t = (m0 + (o >> 6) / NB) * 16 + ((o >> 2) & 15);
      if (t < tn && e < en) {
        const int64_t at = (t0 + t) * E + e0 + e;
        if (vec && logits_f32) {
          *(f32x4_t*)((float*)logits + at) = s;
        } else if (vec) {
          *(uint2*)((bf16_t*)logits + at) = uint2{pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3])};
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (e + i < en) {
              if (logits_f32) ((float*)logits)[at + i] = s[i];
              else ((bf16_t*)logits)[at + i] = f2bf(s[i]);
            }
        }
      }
    }
  }
}

template <typename T, int MB, int NB>
hipError_t fwd(const LaunchCtx& c, const RouterArgs& a, void* logits) {
  constexpr size_t smem = fwd_smem<MB, NB>();
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
  // Float32 is bound by its MFMA, which a second read of x for another 64 experts
  // does not slow down and more, smaller work-groups share out better (T = 8192,
  // d = 2000, E = 128: 46 us with 128 experts a work-group, 42 with 64).
  if (a.E <= 64 || sizeof(T) == 4) return fwd_tokens<T, 4>(c, a, logits);
  if constexpr (sizeof(T) != 4) return fwd_tokens<T, 8>(c, a, logits);
}

// ---------------------------------------------------------------- backward
// dw parts: work-group (E block of 128, d block of 128, run of tokens).  Steps
// of TS tokens pass through two LDS buffers as they lie in memory,
// [token][column], two more steps' loads in flight in registers; a transposing
// LDS read (16-bit) or plain 4-byte reads (the K = 4 float32 MFMA) hand the
// MFMA its token-contiguous operands.  Parts are float32 [run][E][d].  (In a
// launch of its own with two work-groups per CU 30 us at the size above, of
// which loads and staging alone took 19; one work-group with 64-token steps 35,
// blocks of 64 experts with 64-token steps and half the parts 31.)
constexpr int kDwE = 128, kDwD = 128;

template <typename T> struct DwTile;
// `at` is the place of byte b of row r.  16-bit: a transposing read's first 32
// lanes take 32 bytes each of rows r .. r + 3 and r + 8 .. r + 11, so the row's
// 32-byte chunks are XORed with a number that differs between those eight and
// the lanes meet all 64 banks once.  Float32: row r starts at bank 16 r, for
// reads of 16 columns of four rows.
template <> struct DwTile<bf16_t> {
  static constexpr int TS = 32, STRIDE = 256;
  static __device__ __forceinline__ int at(int r, int b) {
    return r * STRIDE + (b ^ (((r & 3) | ((r >> 1) & 4)) << 5));
  }
};
template <> struct DwTile<float> {
  static constexpr int TS = 32, STRIDE = 576;
  static __device__ __forceinline__ int at(int r, int b) { return r * STRIDE + b; }
};

__device__ __forceinline__ void split_bf16(float v, bf16_t& hi, bf16_t& lo) {
  hi = f2bf(v);
  const float h = bf2f(hi);
  // beside an infinity the rest would be infinite or NaN; hi carries it alone
  lo = fabsf(h) < __builtin_huge_valf() ? f2bf(v - h) : (bf16_t)0;
}

// The rest lo must not meet an infinity of x or w: 0 inf, or a rest of the other
// sign, would make a NaN of the formula's infinity, which hi gives alone.  (At the
// size above 60.3 us without what follows from this, 61.2 with.)
__device__ __forceinline__ bool is_finite(float v) { return fabsf(v) < __builtin_huge_valf(); }
// Of bf16 operands: whether one is not finite, and the same with those as zeros.
struct NotFinite {
  typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
  u16x2_t most = {0, 0};  // largest magnitudes of the low and the high halves
  __device__ __forceinline__ void see(u32x4_t v) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2_t, v[i] & 0x7fff7fffu));
  }
  __device__ __forceinline__ bool any() const { return __any(most[0] >= 0x7f80u || most[1] >= 0x7f80u); }
};
__device__ __forceinline__ u32x4_t finite_only(u32x4_t v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((v[i] & 0x7f80u) == 0x7f80u) v[i] &= 0xffff0000u;
    if ((v[i] & 0x7f800000u) == 0x7f800000u) v[i] &= 0xffffu;
  }
  return v;
}

// Sixteen bytes of dlogits as floats.
template <typename LT>
__device__ __forceinline__ void unpack16(float* f, u32x4_t v) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (sizeof(LT) == 4) {
      f[j] = __uint_as_float(v[j]);
    } else {
      f[2 * j] = __uint_as_float(v[j] << 16);
      f[2 * j + 1] = __uint_as_float(v[j] & 0xffff0000u);
    }
  }
}

// A tile of dlogits, rows t0 .. t0 + ROWS (of which `rows` exist) by experts
// e0 .. e0 + 128, loaded by NT threads 16 bytes each (neighbours contiguous)
// and stored for the MFMAs at Place::at(row, byte): float32, or the two bf16
// parts in hs and ls.  Rows and experts that do not exist become zeros.
template <typename T, typename LT, int ROWS, int NT, class Place>
struct DlTile {
  static constexpr int PER = 16 / (int)sizeof(LT);       // values per load
  static constexpr int UPR = 128 / PER;                  // loads per row
  static constexpr int N = ROWS * UPR / NT;              // loads per thread
  static constexpr bool LO = sizeof(T) == 2 && sizeof(LT) == 4;
  u32x4_t v[N];
  __device__ __forceinline__ void load(const LT* p, int E, int e0, int rows, bool vec) {
    if (vec) {  // E is a multiple of PER and the rows are aligned
      const rsrc_t b = buffer_of(p, (uint64_t)min(rows, ROWS) * E * sizeof(LT));
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int u = (int)threadIdx.x + i * NT, e = e0 + (u % UPR) * PER;
        v[i] = load16(b, (uint32_t)((u / UPR * E + e) * (int)sizeof(LT)), e < E);
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int u = (int)threadIdx.x + i * NT, r = u / UPR, e = e0 + (u % UPR) * PER;
      v[i] = u32x4_t{0, 0, 0, 0};
      const LT* a = p + (int64_t)r * E + e;
#pragma unroll
      for (int j = 0; j < PER; ++j)
        if (r < rows && e + j < E) {
          if constexpr (sizeof(LT) == 4) v[i][j] = __float_as_uint(a[j]);
          else v[i][j >> 1] |= (uint32_t)a[j] << (16 * (j & 1));
        }
    }
  }
  __device__ __forceinline__ void store(char* hs, char* ls) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int u = (int)threadIdx.x + i * NT, r = u / UPR, c = (u % UPR) * PER;
      if constexpr (sizeof(T) == 4) {
        float f[PER];
        unpack16<LT>(f, v[i]);
#pragma unroll
        for (int j = 0; j < PER; j += 4)
          *(f32x4_t*)(hs + Place::at(r, (c + j) * 4)) = f32x4_t{f[j], f[j + 1], f[j + 2], f[j + 3]};
      } else if constexpr (!LO) {
        *(u32x4_t*)(hs + Place::at(r, c * 2)) = v[i];
      } else {
        uint2 h, l;
        bf16_t a[4], b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) split_bf16(__uint_as_float(v[i][j]), a[j], b[j]);
        h.x = (uint32_t)a[0] | ((uint32_t)a[1] << 16);
        h.y = (uint32_t)a[2] | ((uint32_t)a[3] << 16);
        l.x = (uint32_t)b[0] | ((uint32_t)b[1] << 16);
        l.y = (uint32_t)b[2] | ((uint32_t)b[3] << 16);
        *(uint2*)(hs + Place::at(r, c * 2)) = h;
        *(uint2*)(ls + Place::at(r, c * 2)) = l;
      }
    }
  }
};

template <typename T, typename LT>
__device__ __forceinline__ bool dl_vec(const RouterArgs& a) { return (a.E * sizeof(LT)) % 16 == 0; }

template <typename T, typename LT>
constexpr int dw_stage() { return (sizeof(T) == 2 && sizeof(LT) == 4 ? 3 : 2) * DwTile<T>::TS * DwTile<T>::STRIDE; }

// A wave's sums over one run, with the products of dlogits' second part if REST.
// A sum that comes out not finite is taken from the first part's products alone,
// in a second pass over the run that only such sums cause.
template <typename T, typename LT, bool REST>
__device__ __forceinline__ void dw_sums(f32x4_t (&acc)[4][2], const RouterArgs& a, char* smem, int e0, int d0,
                                        int run) {
  constexpr int TS = DwTile<T>::TS, ST = DwTile<T>::STRIDE;
  constexpr int XU = kDwD * (int)sizeof(T) / 16;          // 16-byte loads per row of x
  constexpr int XV = TS * XU / 512;
  const int lane = threadIdx.x & 63, wave = tile::wave_id(), q = lane >> 4, col = lane & 15;
  const int64_t tb = (int64_t)run * a.run_tokens;
  const int tn = (int)(a.T - tb < a.run_tokens ? a.T - tb : a.run_tokens);
  const int xrow = a.d * (int)sizeof(T);
  const T* xp = (const T*)a.x + tb * a.d;
  const LT* lp = (const LT*)a.dlogits + tb * a.E;
  const bool vec = dl_vec<T, LT>(a);
  u32x4_t xr[2][XV];
  DlTile<T, LT, TS, 512, DwTile<T>> dlr[2];
  auto fetch = [&](auto set, int s) {  // tokens s .. s + TS of the run; zeros past its end and past E and d
    auto& xv = xr[set.value];
    auto& dl = dlr[set.value];
    const rsrc_t xb = buffer_of(xp + (int64_t)s * a.d, (uint64_t)min(tn - s, TS) * xrow);
#pragma unroll
    for (int i = 0; i < XV; ++i) {
      const int u = (int)threadIdx.x + i * 512, at = d0 * (int)sizeof(T) + (u % XU) * 16;
      xv[i] = load16(xb, (uint32_t)(u / XU * xrow + at), at < xrow);
    }
    dl.load(lp + (int64_t)s * a.E, a.E, e0, tn - s, vec);
  };
  auto stage = [&](auto set, char* b) {
    const auto& xv = xr[set.value];
    const auto& dl = dlr[set.value];
#pragma unroll
    for (int i = 0; i < XV; ++i) {
      const int u = (int)threadIdx.x + i * 512, r = u / XU, cb = (u % XU) * 16;
      *(u32x4_t*)(b + DwTile<T>::at(r, cb)) = xv[i];
    }
    dl.store(b + TS * ST, b + 2 * TS * ST);
  };
  const int we = (wave >> 2) * 64, wd = (wave & 3) * 32;
  const bool busy = e0 + we < a.E && d0 + wd < a.d;  // uniform: this quarter exists
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x4_t{0, 0, 0, 0};
  std::integral_constant<int, 0> set0;
  std::integral_constant<int, 1> set1;
  fetch(set0, 0);
  if (TS < tn) fetch(set1, TS);
  stage(set0, smem);
  if (2 * TS < tn) fetch(set0, 2 * TS);
  auto step = [&](auto set, auto next, int s) {  // the step at token s, in buffer and registers `set`
    __syncthreads();  // this step's buffer is written, the other one's reads are done
    const char* xs = smem + set.value * dw_stage<T, LT>();
    const char* hs = xs + TS * ST;
    const char* ls = hs + TS * ST;
    if (s + TS < tn) {
      stage(next, smem + next.value * dw_stage<T, LT>());
      if (s + 3 * TS < tn) fetch(next, s + 3 * TS);
    }
    if (busy) {
      if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < TS; k += 4) {
          float av[4], bv[2];
#pragma unroll
          for (int i = 0; i < 4; ++i) av[i] = *(const float*)(hs + DwTile<T>::at(k + q, (we + i * 16 + col) * 4));
#pragma unroll
          for (int j = 0; j < 2; ++j) bv[j] = *(const float*)(xs + DwTile<T>::at(k + q, (wd + j * 16 + col) * 4));
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(av[i], bv[j], acc[i][j], 0, 0, 0);
        }
      } else {
        // eight tokens 8 q .. of column `col`: the 16 lanes of a group read 4
        // tokens by 16 columns and get them transposed
        auto frag = [&](const char* base, int c0) {
          typedef __attribute__((address_space(3))) s16x4_t* lds_p;
          const int r = q * 8 + (col >> 2), b = (c0 + 4 * (col & 3)) * 2;
          const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_p)(base + DwTile<T>::at(r, b)));
          const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_p)(base + DwTile<T>::at(r + 4, b)));
          return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        };
        static_assert(TS == 32, "a step is one MFMA's K");
        bf16x8_t bv[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) bv[j] = frag(xs, wd + j * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bf16x8_t h = frag(hs, we + i * 16);
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(h, bv[j], acc[i][j], 0, 0, 0);
          if constexpr (REST) {
            const bf16x8_t l = frag(ls, we + i * 16);
#pragma unroll
            for (int j = 0; j < 2; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(l, bv[j], acc[i][j], 0, 0, 0);
          }
        }
      }
    }
  };
  for (int s = 0; s < tn; s += 2 * TS) {
    step(set0, set1, s);
    if (s + TS < tn) step(set1, set0, s + TS);
  }
}

template <typename T, typename LT>
__device__ __forceinline__ void dw_part(const RouterArgs& a, char* smem, int eb, int db, int run) {
  constexpr bool LO = sizeof(T) == 2 && sizeof(LT) == 4;  // dlogits has a second part
  const int lane = threadIdx.x & 63, wave = tile::wave_id(), q = lane >> 4, col = lane & 15;
  const int e0 = eb * kDwE, d0 = db * kDwD, we = (wave >> 2) * 64, wd = (wave & 3) * 32;
  float* part = a.parts + (int64_t)run * a.E * a.d;
  f32x4_t acc[4][2];
  // the sums (those of `which`, a bit each, if given); returns the ones that are not finite
  auto write = [&](uint32_t which) {
    uint32_t bad = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const int e = e0 + we + i * 16 + q * 4 + m, c = d0 + wd + j * 16 + col;
          const uint32_t bit = 1u << ((i * 2 + j) * 4 + m);
          if (e < a.E && c < a.d && (which & bit)) {
            if (LO && !is_finite(acc[i][j][m])) bad |= bit;
            if (a.runs > 1) part[(int64_t)e * a.d + c] = acc[i][j][m];
            else ((T*)a.dw)[(int64_t)e * a.d + c] = from_f32<T>(acc[i][j][m]);
          }
        }
    return bad;
  };
  dw_sums<T, LT, LO>(acc, a, smem, e0, d0, run);
  const uint32_t bad = write(~0u);
  if constexpr (LO) {
    if (__syncthreads_or(bad != 0)) {
      dw_sums<T, LT, false>(acc, a, smem, e0, d0, run);
      write(bad);
    }
  }
}

// dx: 8 waves, each with the operands of 16 DT columns of w and up to 128
// experts in registers, over blocks of 32 tokens whose dlogits pass through LDS
// once for all of them.  Tile j of a wave holds columns base + DT col + j, so a
// lane's results are DT neighbouring columns.
constexpr int kDxWaves = 8, kDxTok = 32, kDxE = 128;
template <typename T> constexpr int dx_tiles = 8 / (int)sizeof(T);
template <typename T> constexpr int dx_steps = kDxE * (int)sizeof(T) / 64;

// The DT operands of K step k: experts e0 .. of column c + j, 16 bytes a lane,
// from 8 bytes (DT columns) of each expert's row; zeros past E and d.
template <typename T>
__device__ __forceinline__ void w_operands(u32x4_t (&o)[dx_tiles<T>], rsrc_t w, int e0, int E, int d, int c) {
  constexpr int PER = 16 / (int)sizeof(T);
  tile::u32x2_t v[PER];
#pragma unroll
  for (int m = 0; m < PER; ++m) {
    const uint32_t at = (uint32_t)((e0 + m) * d + c) * (uint32_t)sizeof(T);
    v[m] = __builtin_bit_cast(tile::u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(
                                                 w, (int)(e0 + m < E && c < d ? at : kPast), 0, 0));
  }
#pragma unroll
  for (int j = 0; j < dx_tiles<T>; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4)
        o[j][i] = v[i][j];
      else
        o[j][i] = __builtin_amdgcn_perm(v[2 * i + 1][j >> 1], v[2 * i][j >> 1], j & 1 ? 0x07060302u : 0x05040100u);
    }
}

template <typename T> constexpr int dx_stride = 128 * (int)sizeof(T) + 16;  // bytes per token row in LDS
template <typename T> struct DxPlace {
  static __device__ __forceinline__ int at(int r, int b) { return r * dx_stride<T> + b; }
};

// MULTI: more than 128 experts; w's operands then pass through the registers a
// step at a time, for all 32 tokens, instead of staying in them.
template <typename T, typename LT, bool MULTI>
__device__ __forceinline__ void dx_part(const RouterArgs& a, char* smem, int cb, int run) {
  constexpr bool LO = sizeof(T) == 2 && sizeof(LT) == 4;
  constexpr int DT = dx_tiles<T>, NK = dx_steps<T>, ST = dx_stride<T>, PER = 16 / (int)sizeof(T);
  constexpr int HG = MULTI ? 2 : 1;  // groups of 16 tokens whose sums are held together
  const int lane = threadIdx.x & 63, wave = tile::wave_id(), q = lane >> 4, col = lane & 15;
  const int wcb = cb * kDxWaves + wave;             // this wave's block of 16 DT columns
  const bool busy = wcb * 16 * DT < a.d;            // uniform
  const int c = wcb * 16 * DT + col * DT;           // this lane's DT columns; d is a multiple of 8
  const bool in = c < a.d;
  const bool vec = dl_vec<T, LT>(a);
  const int ebs = a.dx_eblocks;
  const rsrc_t wb = buffer_of(a.w, (uint64_t)a.E * a.d * sizeof(T));
  u32x4_t wv[MULTI ? 1 : NK][DT];
  if (!MULTI && busy) {
#pragma unroll
    for (int k = 0; k < NK; ++k) {
      w_operands<T>(wv[MULTI ? 0 : k], wb, (k * 4 + q) * PER, a.E, a.d, c);
      __builtin_amdgcn_sched_barrier(0);  // one step's loads at a time hold registers
    }
  }
  // Weights that are not finite enter the MFMAs as zeros where dlogits has a second
  // part, and `infinite` adds their products with the first part.
  bool w_bad = false;  // uniform: the wave holds such a weight
  auto clean = [&](u32x4_t (*o)[DT], int n) {
    NotFinite bad;
#pragma unroll
    for (int k = 0; k < n; ++k)
#pragma unroll
      for (int j = 0; j < DT; ++j) bad.see(o[k][j]);
    const bool any = bad.any();
    if (any) {
#pragma unroll
      for (int k = 0; k < n; ++k)
#pragma unroll
        for (int j = 0; j < DT; ++j) o[k][j] = finite_only(o[k][j]);
    }
    return any;
  };
  if (LO && !MULTI && busy) w_bad = clean(wv, MULTI ? 1 : NK);
  const int64_t tb = (int64_t)run * a.dx_tokens, te = tb + a.dx_tokens < a.T ? tb + a.dx_tokens : a.T;
  DlTile<T, LT, kDxTok, kDxWaves * 64, DxPlace<T>> dl;
  auto fetch = [&](int64_t t, int eb) {
    dl.load((const LT*)a.dlogits + t * a.E, a.E, eb * kDxE, (int)(te - t < kDxTok ? te - t : kDxTok), vec);
  };
  tile::u32x2_t old[2][4];
  f32x4_t acc[HG][DT];
  auto clear = [&]() {
#pragma unroll
    for (int h = 0; h < HG; ++h)
#pragma unroll
      for (int j = 0; j < DT; ++j) acc[h][j] = f32x4_t{0, 0, 0, 0};
  };
  // acc[g] += step k of expert block eb for tokens 16 h ..
  auto step = [&](const char* hs, const char* ls, int g, int h, int k) {
    const int at = (h * 16 + col) * ST + (k * 4 + q) * 16;
    const u32x4_t hv = *(const u32x4_t*)(hs + at);
#pragma unroll
    for (int j = 0; j < DT; ++j) acc[g][j] = mma16<T>(hv, wv[MULTI ? 0 : k][j], acc[g][j]);
    if constexpr (LO) {
      const u32x4_t lv = *(const u32x4_t*)(ls + at);
#pragma unroll
      for (int j = 0; j < DT; ++j) acc[g][j] = mma16<T>(lv, wv[MULTI ? 0 : k][j], acc[g][j]);
    }
  };
  // acc[g] += the products of tokens 16 h .. with this lane's weights of block eb
  // that are not finite
  auto infinite = [&](const char* hs, int g, int h, int eb) {
    const int n = min(a.E - eb * kDxE, kDxE);
#pragma unroll 1
    for (int e = 0; e < n; ++e) {
      const tile::u32x2_t w2 = __builtin_bit_cast(tile::u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(
          wb, (int)(in ? (uint32_t)((eb * kDxE + e) * a.d + c) * (uint32_t)sizeof(T) : kPast), 0, 0));
#pragma unroll
      for (int j = 0; j < DT; ++j) {
        const float w = __uint_as_float(j & 1 ? w2[j >> 1] & 0xffff0000u : w2[j >> 1] << 16);
        if (is_finite(w)) continue;
#pragma unroll
        for (int m = 0; m < 4; ++m)
          acc[g][j][m] += bf2f(*(const bf16_t*)(hs + (h * 16 + q * 4 + m) * ST + e * 2)) * w;
      }
    }
  };
  // result row 4 q + m is a token, and tile j column c + j of it; rows past the
  // run's end lie past the buffers' and are neither read nor written
  const uint32_t rowb = (uint32_t)a.d * sizeof(T);
  auto rows_at = [&](const void* p, int64_t t0) {
    return buffer_of((const T*)p + t0 * a.d, (uint64_t)(te - t0 < kDxTok ? te - t0 : kDxTok) * rowb);
  };
  auto place = [&](int h, int m) {
    return (int)(in ? (uint32_t)(h * 16 + q * 4 + m) * rowb + (uint32_t)c * (uint32_t)sizeof(T) : kPast);
  };
  auto write = [&](int64_t t0, int g, int h) {
    const rsrc_t out = rows_at(a.dx, t0);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      float v[DT];
#pragma unroll
      for (int j = 0; j < DT; ++j) v[j] = acc[g][j][m];
      tile::u32x2_t o;
      if constexpr (sizeof(T) == 2) {
        if (a.dx_in) {
          v[0] += __uint_as_float(old[h][m][0] << 16);
          v[1] += __uint_as_float(old[h][m][0] & 0xffff0000u);
          v[2] += __uint_as_float(old[h][m][1] << 16);
          v[3] += __uint_as_float(old[h][m][1] & 0xffff0000u);
        }
        o = tile::u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
      } else {
        if (a.dx_in) {
          v[0] += __uint_as_float(old[h][m][0]);
          v[1] += __uint_as_float(old[h][m][1]);
        }
        o = tile::u32x2_t{__float_as_uint(v[0]), __float_as_uint(v[1])};
      }
      __builtin_amdgcn_raw_buffer_store_b64(o, out, place(h, m), 0, 0);
    }
  };
  fetch(tb, 0);
  int buf = 0;
  for (int64_t t0 = tb; t0 < te; t0 += kDxTok) {
    if (a.dx_in && busy) {
      const rsrc_t src = rows_at(a.dx_in, t0);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int m = 0; m < 4; ++m)
          old[h][m] = __builtin_bit_cast(tile::u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(src, place(h, m), 0, 0));
    }
    if (MULTI) clear();
    for (int eb = 0; eb < (MULTI ? ebs : 1); ++eb, buf ^= 1) {
      char* hs = smem + buf * 2 * kDxTok * ST;
      char* ls = hs + kDxTok * ST;
      dl.store(hs, ls);
      __syncthreads();  // written; the other buffer's reads are done once every wave is here again
      if (eb + 1 < (MULTI ? ebs : 1)) fetch(t0, eb + 1);
      else if (t0 + kDxTok < te) fetch(t0 + kDxTok, 0);
      if (!busy) continue;
      if constexpr (MULTI) {
        w_bad = false;
#pragma unroll 1
        for (int k = 0; k < NK; ++k) {
          if (eb * kDxE + k * 4 * PER >= a.E) break;
          w_operands<T>(wv[0], wb, eb * kDxE + (k * 4 + q) * PER, a.E, a.d, c);
          if (LO) w_bad |= clean(wv, 1);
          step(hs, ls, 0, 0, k);
          step(hs, ls, 1, 1, k);
        }
        if constexpr (LO) {
          if (w_bad) {
            infinite(hs, 0, 0, eb);
            infinite(hs, HG - 1, 1, eb);
          }
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          clear();
#pragma unroll
          for (int k = 0; k < NK; ++k)
            if (k * 4 * PER < a.E) step(hs, ls, 0, h, k);
          if constexpr (LO) {
            if (w_bad) infinite(hs, 0, h, 0);
          }
          write(t0, 0, h);
        }
      }
    }
    if (MULTI && busy) {
      write(t0, 0, 0);
      write(t0, HG - 1, 1);
    }
  }
}

// dw = the sum of the parts: 4 values a lane, every fourth run a wave, then the
// four waves' sums in order (6726 tokens, d = 136, E = 6: 17 us with all runs in
// one wave, 6 so).
constexpr int kJoinWaves = 4;
template <typename T>
__global__ __launch_bounds__(kJoinWaves * 64) void router_join_kernel(RouterArgs a) {
  __shared__ f32x4_t sums[kJoinWaves * 64];
  const int lane = threadIdx.x & 63, wave = tile::wave_id();
  const int64_t n = (int64_t)a.E * a.d, i = ((int64_t)blockIdx.x * 64 + lane) * 4;
  f32x4_t s = {0, 0, 0, 0};
  if (i < n) {  // d is a multiple of 8: whole groups of 4
#pragma unroll 8
    for (int r = wave; r < a.runs; r += kJoinWaves) {
      const f32x4_t v = *(const f32x4_t*)(a.parts + r * n + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] += v[j];
    }
  }
  sums[threadIdx.x] = s;
  __syncthreads();
  if (wave != 0 || i >= n) return;
#pragma unroll
  for (int w = 1; w < kJoinWaves; ++w) {
    const f32x4_t v = sums[w * 64 + lane];
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] += v[j];
  }
  if constexpr (sizeof(T) == 4) *(f32x4_t*)((float*)a.dw + i) = s;
  else *(uint2*)((bf16_t*)a.dw + i) = uint2{pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3])};
}

template <typename T, typename LT>
constexpr size_t bwd_smem() {
  const size_t w = 2 * dw_stage<T, LT>(), x = 4 * kDxTok * dx_stride<T>;
  return w > x ? w : x;
}

// The dw work-groups and the dx ones, one of each on a CU at a time: dw waits for
// its barriers and LDS while dx moves rows, and the other way round (in a launch
// each, two work-groups of one kind on a CU: 30 and 35 us at the size above;
// together 54).  The longer ones start first: dx where the rows are many (16384
// tokens, d = 2048: 56 us with dw first, 53 with dx; 2048 tokens: 11.8 and 13.3).
template <typename T, typename LT, bool MULTI>
__global__ __launch_bounds__(512, 4) void router_bwd_kernel(RouterArgs a) {
  extern __shared__ __align__(16) char smem[];
  int b = (int)blockIdx.x - (a.dx_first ? a.dx_groups : 0);
  if (a.dx_first ? b >= 0 : b < a.dw_groups) {
    b = xcd_share(b, a.dw_groups);
    const int db = b % a.d_blocks;
    b /= a.d_blocks;
    dw_part<T, LT>(a, smem, b % a.e_blocks, db, b / a.e_blocks);
  } else {
    b = xcd_share(a.dx_first ? b + a.dx_groups : b - a.dw_groups, a.dx_groups);
    dx_part<T, LT, MULTI>(a, smem, b % a.dx_blocks, b / a.dx_blocks);
  }
}

template <typename T, typename LT, bool MULTI>
hipError_t bwd(const LaunchCtx& c, const RouterArgs& a) {
  constexpr size_t smem = bwd_smem<T, LT>();
  HIP_RET(tile::allow_smem_once<router_bwd_kernel<T, LT, MULTI>>(smem));
  MOE_LAUNCH(c, "router_bwd", (router_bwd_kernel<T, LT, MULTI>), dim3((unsigned)(a.dw_groups + a.dx_groups)), dim3(512),
             smem, a);
  if (a.runs > 1)
    MOE_LAUNCH(c, "router_join", router_join_kernel<T>, dim3((unsigned)cdiv((int64_t)a.E * a.d, 256)),
               dim3(kJoinWaves * 64), 0, a);
  return hipSuccess;
}
template <typename T, typename LT>
hipError_t bwd(const LaunchCtx& c, const RouterArgs& a) {
  return a.dx_eblocks > 1 ? bwd<T, LT, true>(c, a) : bwd<T, LT, false>(c, a);
}

}  // namespace

RouterPlan router_plan(int64_t T, int64_t d, int64_t E, int dtype) {
  RouterPlan p;
  const int step = dtype == F32 ? DwTile<float>::TS : DwTile<bf16_t>::TS;
  // A work-group per CU, beside a dx one, in whole steps: more cost more parts
  // (E d floats of traffic each way) than they hide (two: 66 us instead of 55 at
  // the size above).  Up to four steps are one run, whose sums are dw itself
  // without a second launch (51 tokens: 15.0 us with two runs, 12.0).
  const int64_t tiles = cdiv(d, kDwD) * cdiv(E, kDwE);
  const int64_t want = 256 / tiles < 1 ? 1 : 256 / tiles;
  p.run_tokens = T <= 4 * step ? 4 * step : cdiv(cdiv(T, step), want) * step;
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
  a.dx_eblocks = (int)cdiv(a.E, kDxE);
  a.dx_blocks = (int)cdiv(a.d, 16 * (a.dtype == F32 ? dx_tiles<float> : dx_tiles<bf16_t>) * kDxWaves);
  // a work-group per CU (each first loads its part of w), in whole blocks
  const int64_t tok = cdiv(cdiv((int64_t)a.T * a.dx_blocks, 256), kDxTok) * kDxTok;
  a.dx_tokens = (int)tok;
  a.dx_groups = a.dx_blocks * (int)cdiv(a.T, tok);
  a.dx_first = (int64_t)a.T * a.d * (a.dtype == F32 ? 4 : 2) > int64_t(32) << 20;
  if (a.dtype == F32) return a.logits_dtype == F32 ? bwd<float, float>(c, a) : bwd<float, bf16_t>(c, a);
  return a.logits_dtype == F32 ? bwd<bf16_t, float>(c, a) : bwd<bf16_t, bf16_t>(c, a);
}

}  // namespace moe
