// The norms before and after a block with its gate and residual scale, in one
// pass over the rows, and their gradients:
//   N(v; w) = v rsqrt(mean(v^2) + eps) w
//   z = a x + gate N(y; w_post)      (N(y) = y without w_post)
//   h = N(z; w_next)
// backward, from dz and dh:
//   zh = z rz,  t = dh w_next,  g = dz + rz (t - zh mean(t zh)),  dx = a g
//   u = y ry,  s = g gate w_post,  dy = ry (s - u mean(s u))
//   dw_next = sum_t dh zh,  dw_post = sum_t g gate u,  dgate = sum g u w_post
// (over t for a gate per channel, over the row for one per token).
//
// What bounds them: memory, 4 values a column forward (x, y, z, h) and 6
// backward (dz, dh, z, y, dx, dy).  A row stays in its lanes' registers between
// its sums and its results, so each is read once; no statistics are kept for
// the backward, which reads z and y anyway and sums their squares with the
// sums that it needs of the row.  Sums are float32 in a fixed order (lanes by
// DPP, waves through LDS, work-groups in order), without atomics.
#include <algorithm>

#include "common.h"
#include "tile.h"

namespace moe {
namespace {

using tile::u32x4_t;

template <typename T> struct Row;  // a 16-byte piece of a row
template <> struct Row<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ float get(const u32x4_t& v, int i) { return __uint_as_float(v[i]); }
  static __device__ __forceinline__ u32x4_t put(const float (&f)[N]) {
    return u32x4_t{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
  }
};
template <> struct Row<bf16_t> {
  static constexpr int N = 8;
  static __device__ __forceinline__ float get(const u32x4_t& v, int i) {
    return __uint_as_float(i & 1 ? v[i >> 1] & 0xffff0000u : v[i >> 1] << 16);
  }
  static __device__ __forceinline__ u32x4_t put(const float (&f)[N]) {
    return u32x4_t{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                   pack_bf16x2(f[6], f[7])};
  }
};

// ------------------------------------------------------------ sums over lanes
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xf, 0xf, true));
}
// Sum over aligned groups of L <= 64 lanes, in every lane.
template <int L>
__device__ __forceinline__ float lane_sum(float v) {
  static_assert(L >= 8 && L <= 64, "");
  v += dpp<0xB1>(v);   // quad: lane xor 1
  v += dpp<0x4E>(v);   // quad: lane xor 2
  v += dpp<0x141>(v);  // the other quad of eight (half-row mirror)
  if constexpr (L >= 16) v += dpp<0x140>(v);  // the other eight of a row (row mirror)
  if constexpr (L >= 32) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  }
  if constexpr (L >= 64) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  }
  return v;
}

// Sums of NS values over a row's L lanes, in every one of them; `part` (LDS, a
// float a wave and value, not in use by an earlier sum that a wave may still
// read) where a row has several waves.  Called by the whole work-group then.
template <int L, int NS>
__device__ __forceinline__ void row_sums(float (&v)[NS], float* part) {
#pragma unroll
  for (int i = 0; i < NS; ++i) v[i] = lane_sum<(L < 64 ? L : 64)>(v[i]);
  if constexpr (L > 64) {
    constexpr int W = L / 64;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < NS; ++i) part[wave * NS + i] = v[i];
    }
    __syncthreads();
    const float* p = part + wave / W * W * NS;
#pragma unroll
    for (int i = 0; i < NS; ++i) v[i] = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w)
#pragma unroll
      for (int i = 0; i < NS; ++i) v[i] += p[w * NS + i];
  }
}

// A work-group: 256 threads, or a row's lanes where those do not divide them.
constexpr int threads_of(int L) { return 256 % L ? L : 256; }
template <int L> constexpr int kThreads = threads_of(L);

// NV pieces of a row of `vecs`, this lane's; zeros past the end.
template <int L, int NV, bool NT = false>
__device__ __forceinline__ void load_row(u32x4_t (&v)[NV], const u32x4_t* p, int lane, int vecs) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    v[i] = u32x4_t{0, 0, 0, 0};
    if (lane + i * L < vecs) v[i] = NT ? __builtin_nontemporal_load(p + lane + i * L) : p[lane + i * L];
  }
}

__device__ __forceinline__ float rstd_of(float squares, const NormArgs& a) {
  return 1.0f / sqrtf(squares * a.inv_d + a.eps);
}

// -------------------------------------------------------------------- forward
template <typename T, int L, int NV>
__global__ __launch_bounds__(kThreads<L>) void norm_fwd_kernel(NormArgs a) {
  constexpr int N = Row<T>::N, ROWS = kThreads<L> / L;
  __shared__ float part[2][16];
  const int lane = threadIdx.x % L, vecs = a.d / N;
  const int64_t row = folded_block() * ROWS + threadIdx.x / L;
  const bool in = row < a.T;
  const int mine = in ? vecs : 0;  // a row past the last loads and stores nothing
  const int64_t at = row * vecs;
  u32x4_t xv[NV], yv[NV], wp[NV], wn[NV], gv[NV];
  load_row<L>(xv, (const u32x4_t*)a.x + at, lane, mine);
  if (a.y) load_row<L>(yv, (const u32x4_t*)a.y + at, lane, mine);
  if (a.w_post) load_row<L>(wp, (const u32x4_t*)a.w_post, lane, vecs);
  if (a.gate_kind == 1) load_row<L>(gv, (const u32x4_t*)a.gate, lane, vecs);
  if (a.w_next) load_row<L>(wn, (const u32x4_t*)a.w_next, lane, vecs);
  const float gt = a.gate_kind == 2 && in ? to_f32<T>(((const T*)a.gate)[row]) : 1.0f;
  float z[NV][N];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) z[i][j] = Row<T>::get(xv[i], j);
  if (a.y) {
    float r = 1.0f;
    if (a.w_post) {
      float s[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const float v = Row<T>::get(yv[i], j);
          s[0] = fmaf(v, v, s[0]);
        }
      row_sums<L>(s, part[0]);
      r = rstd_of(s[0], a);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        float b = Row<T>::get(yv[i], j);
        if (a.w_post) b = b * r * Row<T>::get(wp[i], j);
        if (a.gate_kind) b *= a.gate_kind == 1 ? Row<T>::get(gv[i], j) : gt;
        z[i][j] = fmaf(a.scale, z[i][j], b);
      }
      if (lane + i * L < mine) ((u32x4_t*)a.z + at)[lane + i * L] = Row<T>::put(z[i]);
    }
  }
  if (!a.w_next) return;
  // of z as it is before its rounding to T
  float s[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) s[0] = fmaf(z[i][j], z[i][j], s[0]);
  row_sums<L>(s, part[1]);
  const float r = rstd_of(s[0], a);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int j = 0; j < N; ++j) z[i][j] = z[i][j] * r * Row<T>::get(wn[i], j);
    if (lane + i * L < mine) ((u32x4_t*)a.h + at)[lane + i * L] = Row<T>::put(z[i]);
  }
}

// ------------------------------------------------------------------- backward
// A work-group takes rows group, group + groups, ... and sums its columns of
//   A = dh zh  and  B = g gate_t u  (gate_t: the gate per token, else 1)
// in registers; dw_next = A, dw_post = B gate_c, dgate_c = B w_post.
// column_finish turns the sums of one column into them.
template <typename T>
__device__ __forceinline__ void column_finish(const NormArgs& a, int c, float A, float B) {
  if (a.dw_next) ((T*)a.dw_next)[c] = from_f32<T>(A);
  if (a.dw_post) ((T*)a.dw_post)[c] = from_f32<T>(a.gate_kind == 1 ? B * to_f32<T>(((const T*)a.gate)[c]) : B);
  if (a.gate_kind == 1) ((T*)a.dgate)[c] = from_f32<T>(a.w_post ? B * to_f32<T>(((const T*)a.w_post)[c]) : B);
}

// NT: the rows are loaded past the caches.
template <typename T, int L, int NV, bool NT>
__global__ __launch_bounds__(kThreads<L>) void norm_bwd_kernel(NormArgs a) {
  constexpr int N = Row<T>::N, ROWS = kThreads<L> / L;
  __shared__ float part[2][48];
  __shared__ __align__(16) float col[ROWS > 1 ? ROWS * L * N : 1];
  const int lane = threadIdx.x % L, sub = threadIdx.x / L, vecs = a.d / N;
  // 32 columns a lane leave no registers for the weights and the next row, which
  // are then read where they are used (2048 rows of 16384 in bf16: 302 us with
  // them spilled, 116 so; in float32, with 32 more sums a lane, 382)
  constexpr bool LEAN = NV * N >= 32;
  constexpr int KEPT = LEAN ? 1 : NV;
  u32x4_t wp_[KEPT], wn_[KEPT], gv_[KEPT];
  if constexpr (!LEAN) {
    if (a.w_post) load_row<L>(wp_, (const u32x4_t*)a.w_post, lane, vecs);
    if (a.gate_kind == 1) load_row<L>(gv_, (const u32x4_t*)a.gate, lane, vecs);
    if (a.w_next) load_row<L>(wn_, (const u32x4_t*)a.w_next, lane, vecs);
  }
  const auto weight = [&](const u32x4_t (&kept)[KEPT], const void* p, int i) {
    if constexpr (LEAN) return lane + i * L < vecs ? ((const u32x4_t*)p)[lane + i * L] : u32x4_t{0, 0, 0, 0};
    else return kept[i];
  };
  float A[NV][N], B[NV][N];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) A[i][j] = B[i][j] = 0.0f;
  // the next row is on its way while one is worked on (16384 rows of 2048: 83 us, 92
  // without)
  struct In {
    u32x4_t dz[NV], dh[NV], z[NV], y[NV];
    float gt;
  };
  const auto load = [&](In& in, int64_t row) {
    const int mine = row < a.T ? vecs : 0;
    const int64_t at = row * vecs;
    if (a.dz) load_row<L, NV, NT>(in.dz, (const u32x4_t*)a.dz + at, lane, mine);
    if (a.w_next) {
      load_row<L, NV, NT>(in.dh, (const u32x4_t*)a.dh + at, lane, mine);
      load_row<L, NV, NT>(in.z, (const u32x4_t*)a.z_in + at, lane, mine);
    }
    if (a.y) load_row<L, NV, NT>(in.y, (const u32x4_t*)a.y + at, lane, mine);
    in.gt = a.gate_kind == 2 && row < a.T ? to_f32<T>(((const T*)a.gate)[row]) : 1.0f;
  };
  const int64_t step = (int64_t)gridDim.x * ROWS;
  In next;
  if constexpr (!LEAN) load(next, (int64_t)blockIdx.x * ROWS + sub);
  for (int64_t row0 = (int64_t)blockIdx.x * ROWS; row0 < a.T; row0 += step) {
    const int64_t row = row0 + sub, at = row * vecs;
    const bool in = row < a.T;
    const int mine = in ? vecs : 0;
    if constexpr (LEAN) load(next, row);
    const In now = next;
    if constexpr (!LEAN) load(next, row + step);
    const auto &dzv = now.dz, &dhv = now.dh, &zv = now.z, &yv = now.y;
    const float gt = now.gt;
    float s[3] = {0.0f, 0.0f, 0.0f};  // z^2, t z, y^2
    if (a.w_next) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const u32x4_t wn = weight(wn_, a.w_next, i);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const float z = Row<T>::get(zv[i], j);
          s[0] = fmaf(z, z, s[0]);
          s[1] = fmaf(Row<T>::get(dhv[i], j) * Row<T>::get(wn, j), z, s[1]);
        }
      }
    }
    if (a.w_post) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const float y = Row<T>::get(yv[i], j);
          s[2] = fmaf(y, y, s[2]);
        }
    }
    row_sums<L>(s, part[0]);
    const float rz = a.w_next ? rstd_of(s[0], a) : 0.0f;
    const float mz = s[1] * rz * a.inv_d;  // mean(t zh)
    const float ry = a.w_post ? rstd_of(s[2], a) : 1.0f;
    float g[NV][N];
    float q[1] = {0.0f};  // g w_post gate_c y
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      u32x4_t wn, wp, gv;
      if (a.w_next) wn = weight(wn_, a.w_next, i);
      if (a.w_post) wp = weight(wp_, a.w_post, i);
      if (a.gate_kind == 1) gv = weight(gv_, a.gate, i);
      float o[N];
#pragma unroll
      for (int j = 0; j < N; ++j) {
        float v = a.dz ? Row<T>::get(dzv[i], j) : 0.0f;
        if (a.w_next) {
          const float dh = Row<T>::get(dhv[i], j), zh = Row<T>::get(zv[i], j) * rz;
          v += rz * (dh * Row<T>::get(wn, j) - zh * mz);
          A[i][j] = fmaf(dh, zh, A[i][j]);
        }
        o[j] = a.scale * v;
        if (a.dy) {
          if (a.y) {
            const float y = Row<T>::get(yv[i], j);
            B[i][j] = fmaf(v * gt, y * ry, B[i][j]);
            if (a.w_post) v *= Row<T>::get(wp, j);
            if (a.gate_kind == 1) v *= Row<T>::get(gv, j);
            q[0] = fmaf(v, y, q[0]);
          }
        }
        g[i][j] = v;
      }
      if (lane + i * L < mine) ((u32x4_t*)a.dx + at)[lane + i * L] = Row<T>::put(o);
    }
    if (!a.dy) {
      if constexpr (L > 64) __syncthreads();  // part[0] is free again
      continue;
    }
    row_sums<L>(q, part[1]);
    if (a.gate_kind == 2 && in && lane == 0) ((T*)a.dgate)[row] = from_f32<T>(q[0] * ry);
    const float my = a.w_post ? gt * q[0] * ry * a.inv_d : 0.0f;  // mean(s u)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float o[N];
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float sv = gt * g[i][j];
        o[j] = a.w_post ? ry * (sv - Row<T>::get(yv[i], j) * ry * my) : sv;
      }
      if (lane + i * L < mine) ((u32x4_t*)a.dy + at)[lane + i * L] = Row<T>::put(o);
    }
  }
  if (!a.w_next && !(a.dw_post || a.gate_kind == 1)) return;
  // the work-group's rows of lanes, joined in order; then memory, or, where it
  // is the only work-group, the results
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float (&v)[N] = k ? B[i] : A[i];
      if constexpr (ROWS > 1) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < N; j += 4)
          *(f32x4_t*)&col[(sub * L + lane) * N + j] = f32x4_t{v[j], v[j + 1], v[j + 2], v[j + 3]};
        __syncthreads();
        if (sub == 0) {
          for (int r = 1; r < ROWS; ++r)
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] += col[(r * L + lane) * N + j];
        }
      }
    }
    const int c = (lane + i * L) * N;
    if (sub == 0 && c < a.d) {
      if (gridDim.x == 1) {
#pragma unroll
        for (int j = 0; j < N; ++j) column_finish<T>(a, c + j, A[i][j], B[i][j]);
      } else {
        float* p = a.parts + (int64_t)blockIdx.x * 2 * a.d + c;
#pragma unroll
        for (int j = 0; j < N; j += 4) {
          *(f32x4_t*)(p + j) = f32x4_t{A[i][j], A[i][j + 1], A[i][j + 2], A[i][j + 3]};
          *(f32x4_t*)(p + a.d + j) = f32x4_t{B[i][j], B[i][j + 1], B[i][j + 2], B[i][j + 3]};
        }
      }
    }
  }
}

// The work-groups' column sums, joined in order: 16 columns a work-group, the
// work-groups' parts in 32 slices.
template <typename T>
__global__ __launch_bounds__(256) void norm_join_kernel(NormArgs a, int groups) {
  // thread: (slice of the groups, four columns of A or B)
  constexpr int SL = 32;
  __shared__ __align__(16) float sh[SL][8][4];
  const int q = threadIdx.x & 7, slice = threadIdx.x >> 3;  // q: 4 pieces of A, then of B
  const int c = blockIdx.x * 16 + (q & 3) * 4;
  f32x4_t s = {0, 0, 0, 0};
  if (c < a.d) {
    const int per = (groups + SL - 1) / SL;
    const int g1 = min(groups, (slice + 1) * per);
    const float* p = a.parts + (q >> 2) * a.d + c;
#pragma unroll 8
    for (int g = slice * per; g < g1; ++g) {
      const f32x4_t v = *(const f32x4_t*)(p + (int64_t)g * 2 * a.d);
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] += v[j];
    }
  }
  *(f32x4_t*)sh[slice][q] = s;
  __syncthreads();
  if (threadIdx.x < 16) {
    const int col = blockIdx.x * 16 + threadIdx.x;
    float A = 0.0f, B = 0.0f;
    for (int i = 0; i < SL; ++i) {
      A += sh[i][threadIdx.x >> 2][threadIdx.x & 3];
      B += sh[i][4 + (threadIdx.x >> 2)][threadIdx.x & 3];
    }
    if (col < a.d) column_finish<T>(a, col, A, B);
  }
}

// How a row is spread: NV 16-byte pieces in each of L lanes.
struct Spread {
  int L, NV;
};

// Forward: one piece a lane for few rows (256 of 4096: 4.6 us, with four pieces
// 5.9; 2047 of 2048 8.5 and 9.5); for many, a wave a row while four pieces hold it (16384 rows of 2048 in
// bf16: 46 us with four waves a row, 43 with one).
Spread fwd_spread(int64_t T, int vecs) {
  Spread p = {8, 1};
  const int most = T >= 2048 ? 4 : 1;
  while (p.L * p.NV < vecs) {
    if (p.L >= 64 && p.NV < most) p.NV *= 2;
    else if (p.L < 1024) p.L *= 2;
    else p.NV *= 2;
  }
  return p;
}

// Backward: a row's four operands, the next row's and the two column sums take the
// registers, so one piece a lane up to eight waves a row (8192 rows of 4096: 81 us,
// with two pieces 89, with four 101; 2048 of 8192, eight waves and two pieces 47,
// sixteen and one 63).  Five or six waves where they hold it, of which two
// work-groups share a CU (8192 rows of 2560: 74 us with eight, 51 with five; of 2800
// 74 and 58; seven instead of eight, one a CU, gain nothing).
Spread bwd_spread(int vecs) {
  Spread p = {8, 1};
  while (p.L * p.NV < vecs) {
    if (p.L < 512) p.L *= 2;
    else p.NV *= 2;
  }
  if (p.L == 512 && vecs <= 384) p.L = vecs <= 320 ? 320 : 384;
  return p;
}

// Work-groups of the backward, of which each leaves a part of the column sums: on a
// CU two of up to six waves, one of eight (16384 rows of 2048: 83 us, with one 120,
// with four 96 and twice the parts to join).  Four where a third or more of a row's
// lanes have no column (16384 rows of 1032: 67 us with two, 57 with four; of 520 39
// and 34; in float32, 8192 of 600, 34 and 29).  Half as many where each would take
// one step (512 rows of 2048: 15.2 us in 512, 13.1 in 256; 2000 rows 19.9, in half
// 23.5), and no more than take the same number of steps (333 rows of 4096: 16.3 us
// in 256, of which 77 take a second row, 15.1 in 167; 257 rows 15.9 and 13.8).  A
// single one, which needs no parts and no join, for two steps of rows of one piece a
// lane: a call then launches once and takes 2.2 to 3.1 us less from Python, and in
// a replayed graph 0.1 to 2.8 more (us with the join and without, eager and
// captured: 2 rows of 2048 21.4 and 18.5, 6.5 and 8.5; of 4096 21.5 and 18.8, 7.1 and
// 9.9; 64 of 64 21.7 and 18.6, 8.4 and 9.2; more steps lose more than they save, 4
// rows of 2048 21.4 and 18.8, 6.6 and 11.8; so do longer rows, 2 of 16384 21.3 and
// 31.2, 13.5 and 31.1, in float32 43 and 84 both ways).
int64_t bwd_groups(int64_t T, Spread p, int vecs) {
  const int threads = threads_of(p.L);
  int64_t most = 256 * (p.L <= 256 && 3 * vecs < 2 * p.L ? 4 : p.L <= 384 ? 2 : 1);
  const int64_t blocks = cdiv(T, threads / p.L);
  if (blocks <= 2 && p.NV == 1) return 1;
  if (blocks <= most) most = std::max<int64_t>(256, most / 2);
  const int64_t steps = cdiv(blocks, most);
  return cdiv(blocks, steps);
}

template <typename T, int L, int NV>
hipError_t run_fwd(const LaunchCtx& c, const NormArgs& a) {
  MOE_LAUNCH(c, "norm_forward", (norm_fwd_kernel<T, L, NV>), folded_grid(cdiv(a.T, kThreads<L> / L)),
             dim3(kThreads<L>), 0, a);
  return hipSuccess;
}
template <typename T, int L, int NV>
hipError_t run_bwd(const LaunchCtx& c, const NormArgs& a) {
  const int groups = (int)bwd_groups(a.T, {L, NV}, a.d / Row<T>::N);
  // rows beyond the last-level cache leave it alone (16384 rows of 2048, 402 MB: 82
  // us without, 77 with, 81 with the stores too); below its size they may be there
  // from the step before (4096 rows: 27.7 and 29.1)
  const int64_t rows = 2 + 2 * (a.w_next != nullptr) + 2 * (a.dy != nullptr);
  if (rows * a.T * a.d * (int64_t)sizeof(T) > (int64_t(256) << 20))
    MOE_LAUNCH(c, "norm_backward", (norm_bwd_kernel<T, L, NV, true>), dim3((unsigned)groups), dim3(kThreads<L>), 0, a);
  else
    MOE_LAUNCH(c, "norm_backward", (norm_bwd_kernel<T, L, NV, false>), dim3((unsigned)groups), dim3(kThreads<L>), 0, a);
  if (groups > 1 && (a.dw_next || a.dw_post || a.gate_kind == 1))
    MOE_LAUNCH(c, "norm_join", norm_join_kernel<T>, dim3((unsigned)cdiv(a.d, 16)), dim3(256), 0, a, groups);
  return hipSuccess;
}

#define CASE(RUN, l, nv) \
  if (p.L == l && p.NV == nv) return RUN<T, l, nv>(c, a)
#define UP_TO_512(RUN) \
  CASE(RUN, 8, 1);     \
  CASE(RUN, 16, 1);    \
  CASE(RUN, 32, 1);    \
  CASE(RUN, 64, 1);    \
  CASE(RUN, 128, 1);   \
  CASE(RUN, 256, 1);   \
  CASE(RUN, 512, 1)
template <typename T>
hipError_t fwd(const LaunchCtx& c, const NormArgs& a) {
  const Spread p = fwd_spread(a.T, a.d / Row<T>::N);
  UP_TO_512(run_fwd);
  CASE(run_fwd, 1024, 1);
  CASE(run_fwd, 64, 2);
  CASE(run_fwd, 1024, 2);
  CASE(run_fwd, 64, 4);
  CASE(run_fwd, 128, 4);
  CASE(run_fwd, 256, 4);
  CASE(run_fwd, 512, 4);
  CASE(run_fwd, 1024, 4);
  return hipErrorInvalidValue;
}
template <typename T>
hipError_t bwd(const LaunchCtx& c, const NormArgs& a) {
  const Spread p = bwd_spread(a.d / Row<T>::N);
  UP_TO_512(run_bwd);
  CASE(run_bwd, 320, 1);
  CASE(run_bwd, 384, 1);
  CASE(run_bwd, 512, 2);
  CASE(run_bwd, 512, 4);
  if constexpr (sizeof(T) == 4) CASE(run_bwd, 512, 8);
  return hipErrorInvalidValue;
}
#undef UP_TO_512
#undef CASE

}  // namespace

int64_t norm_bwd_groups(int64_t T, int64_t d, int dtype) {
  const int vecs = (int)(d / (dtype == F32 ? 4 : 8));
  return bwd_groups(T, bwd_spread(vecs), vecs);
}
hipError_t launch_norm_fwd(const LaunchCtx& c, const NormArgs& a) {
  return a.dtype == F32 ? fwd<float>(c, a) : fwd<bf16_t>(c, a);
}
hipError_t launch_norm_bwd(const LaunchCtx& c, const NormArgs& a) {
  return a.dtype == F32 ? bwd<float>(c, a) : bwd<bf16_t>(c, a);
}

}  // namespace moe
