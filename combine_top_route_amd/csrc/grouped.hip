// Products of expert-sorted rows with their experts' MXFP4 matrices, ragged:
//   y[r] = W_e a_r,  offsets[e] <= r < offsets[e + 1],
//   a_r = x[src_of[r] / k] or x[r],
// or, with W_e = [gate; up], y[r] = silu(min(g, L)) clamp(u, -L, L).
//
// A work-group makes a tile of 256 rows of one expert by 256 columns (128 gate
// and the same up columns), eight waves of 128 x 64 in 32x32x16 MFMAs on bf16:
// a code times its power-of-two scale is a bfloat16 number, so the products are
// those of the decoded weights, summed in float32.  Codes stay codes until they
// are in registers: a K step of 64 moves 32 KB of rows and 8 KB of codes into
// LDS where bf16 weights would take 64 KB, and a lane turns a 16-byte piece (32
// codes, one scale) into four MFMA operands with 16 conversions beside 32
// MFMAs.  The K order inside a step is chosen for that: the lanes' halves take
// columns 0 .. 31 and 32 .. 63, operand kk columns 8 kk .. 8 kk + 7 of them, on
// either side.
#include <algorithm>

#include "common.h"
#include "tile.h"

namespace moe {
namespace {

using namespace tile;

constexpr int NW = 8, NT = NW * 64;
constexpr int TN = 256;            // columns of W a tile
constexpr int SLOT_A = 32 * 1024;  // [256 rows][64 values]
constexpr int SLOT_B = 18 * 1024;  // [256 rows][64 bytes: 128 codes], then scale words
constexpr int B_SCALES = 16 * 1024;
constexpr int LDS_BYTES = 3 * SLOT_A + 2 * SLOT_B;

// An expert's row tile: rows m0 .. of [.., seg1), column tile nt.
struct Tile {
  int e, m0, seg1, nt;
};

// Rows of expert e; whatever the offsets hold, inside the R rows there are.
__device__ __forceinline__ int first_row(const GroupedArgs& a, int e) { return min(max(a.offsets[e], 0), a.R); }

// The tile of this work-group, every wave for itself: lane l counts the row
// tiles of experts l P .. l P + P - 1.  False: none.
__device__ __forceinline__ bool find_tile(const GroupedArgs& a, int rows, int ntiles, Tile* t) {
  const int lane = threadIdx.x & 63;
  const int P = (a.E + 63) >> 6;
  int sum = 0;
  for (int i = 0; i < P; ++i) {
    const int e = lane * P + i;
    const int n = e < a.E ? first_row(a, e + 1) - first_row(a, e) : 0;
    sum += (max(n, 0) + rows - 1) / rows;
  }
  int incl = sum;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(incl, d, 64);
    if (lane >= d) incl += o;
  }
  const int total = __builtin_amdgcn_readlane(incl, 63);
  const int L = xcd_tile(blockIdx.y * gridDim.x + blockIdx.x, total * ntiles);
  if (L < 0) return false;
  const int own = __builtin_ctzll(__ballot(incl * ntiles > L));
  const int before = own ? __builtin_amdgcn_readlane(incl, own - 1) : 0;
  // the lane's experts in turn, the same in every lane
  int base = before;
  for (int i = 0; i < P; ++i) {
    const int e = own * P + i;
    if (e >= a.E) break;
    const int o0 = first_row(a, e), o1 = first_row(a, e + 1);
    const int n = (max(o1 - o0, 0) + rows - 1) / rows;
    if (L < (base + n) * ntiles) {
      const int at = L - base * ntiles;
      const int rt = a.row_major ? at / ntiles : at % n;
      t->nt = __builtin_amdgcn_readfirstlane(a.row_major ? at % ntiles : at / n);
      t->e = __builtin_amdgcn_readfirstlane(e);
      t->m0 = __builtin_amdgcn_readfirstlane(o0 + rt * rows);
      t->seg1 = __builtin_amdgcn_readfirstlane(o1);
      return true;
    }
    base += n;
  }
  return false;
}

// Row of W that column n of column tile nt stands for (past the last: the
// last, whose results are dropped).  SWIGLU: 32 gate rows, then the same up
// rows, in turn.
template <bool SWIGLU>
__device__ __forceinline__ int w_row(const GroupedArgs& a, int nt, int n) {
  if constexpr (SWIGLU) {
    const int c = min(nt * (TN / 2) + (n >> 6) * 32 + (n & 31), a.N / 2 - 1);
    return (n & 32) ? a.N / 2 + c : c;
  } else {
    return min(nt * TN + n, a.N - 1);
  }
}

// Direct loads of a K step's rows and of two steps' codes and scales.
template <int ROWS>
struct Loads {
  static constexpr int NA = ROWS / 64;
  const char* pa[NA];
  const char* pb[2];
  const char* ps;
  template <bool SWIGLU>
  __device__ __forceinline__ void init(const GroupedArgs& a, const Tile& t) {
    const int lane = threadIdx.x & 63, w = wave_id();
    int src[NA];
#pragma unroll
    for (int i = 0; i < NA; ++i) {  // rows past the segment repeat its last
      const int r = min(t.m0 + 8 * (w + NW * i) + (lane >> 3), t.seg1 - 1);
      src[i] = a.src_of ? min(max(a.src_of[r], 0), a.R - 1) : r;
    }
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const int row = 8 * (w + NW * i) + (lane >> 3);
      const int64_t s = a.src_of ? src[i] / a.k : src[i];
      pa[i] = (const char*)a.x + s * a.K * 2 + (((lane & 7) ^ mk_swz(row)) << 4);
    }
    const int64_t mat = (int64_t)t.e * a.N;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = 16 * (w + NW * i) + (lane >> 2);
      pb[i] = (const char*)a.codes + (mat + w_row<SWIGLU>(a, t.nt, row)) * (a.K / 2) + (((lane ^ (row >> 2)) & 3) << 4);
    }
    ps = (const char*)a.scales + (mat + w_row<SWIGLU>(a, t.nt, 32 * w + (lane & 31))) * (a.K / 32);
  }
  __device__ __forceinline__ void rows(lds_t* slot) {
    const int w = wave_id();
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      dma16(pa[i], slot + (w + NW * i) * 1024);
      pa[i] += 128;
    }
  }
  // 16 KB of codes and a scale word a row: 32 rows' words (and again the same) a wave
  __device__ __forceinline__ void codes(lds_t* slot) {
    const int w = wave_id();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      dma16(pb[i], slot + (w + NW * i) * 1024);
      pb[i] += 64;
    }
    dma4(ps, slot + B_SCALES + w * 256);
    ps += 4;
  }
};

__device__ __forceinline__ void wait_lgkm0() { __builtin_amdgcn_s_waitcnt(0xC07F); }  // lgkmcnt(0) alone

__device__ __forceinline__ u32x4_t lds16(const lds_t* p) {
  return *(const __attribute__((address_space(3))) u32x4_t*)p;
}

// Eight codes under a scale.
__device__ __forceinline__ bf16x8_t decode8(uint32_t c, float s) {
  u32x4_t o;
  o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0));
  o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1));
  o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2));
  o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3));
  return __builtin_bit_cast(bf16x8_t, o);
}

// One K step (P: the first or second half of the codes' 128 columns).
template <int TMX, int P>
__device__ __forceinline__ void step(const lds_t* __restrict__ As, const lds_t* __restrict__ Bs, int wm, int wn,
                                     f32x16_t (&acc)[TMX][2]) {
  const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
  u32x4_t code[2];
  float s[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int row = wn * 64 + j * 32 + r;
    code[j] = lds16(Bs + row * 64 + (((2 * P + h) ^ (row >> 2)) & 3) * 16);
    const uint32_t word =
        *(const __attribute__((address_space(3))) uint32_t*)(Bs + B_SCALES + (row >> 5) * 256 + (row & 31) * 4);
    s[j] = __uint_as_float(((word >> (16 * P + 8 * h)) & 0xffu) << 23);
  }
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) {
    bf16x8_t b[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) b[j] = decode8(code[j][kk], s[j]);
#pragma unroll
    for (int i = 0; i < TMX; ++i) {
      const bf16x8_t av =
          __builtin_bit_cast(bf16x8_t, lds16(As + mk_off(wm * (TMX * 32) + i * 32 + r, 4 * h + kk)));
#pragma unroll
      for (int j = 0; j < 2; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b[j], av, acc[i][j], 0, 0, 0);
    }
  }
}

// Rows of a step are in slot k mod 3, two steps ahead; codes of steps 2 s and
// 2 s + 1 in slot s mod 2, filled one such pair ahead.  Loads land in the order
// they left, so before the even step all but the next step's rows have, before
// the odd one all but what the even step issued.
template <int ROWS>
__device__ __forceinline__ void mainloop(Loads<ROWS>& ld, int pairs, lds_t* lds, f32x16_t (&acc)[ROWS / 64][2]) {
  constexpr int TMX = ROWS / 64, NA = Loads<ROWS>::NA;
  const int w = wave_id(), wm = w >> 2, wn = w & 3;
#pragma unroll
  for (int i = 0; i < TMX; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
  lds_t* const lb = lds + 3 * SLOT_A;
  ld.codes(lb);
  ld.rows(lds);
  ld.rows(lds + SLOT_A);
  int sa = 0;  // slot of the even step's rows
  auto next = [](int s, int n) { return s + n >= 3 ? s + n - 3 : s + n; };
  for (int p = 0; p < pairs; ++p) {
    const bool more = p + 1 < pairs;
    const lds_t* Bs = lb + (p & 1) * SLOT_B;
    wait_vmcnt<NA>();
    barrier_lds();
    if (more) {
      ld.codes(lb + ((p & 1) ^ 1) * SLOT_B);
      ld.rows(lds + next(sa, 2) * SLOT_A);
    }
    step<TMX, 0>(lds + sa * SLOT_A, Bs, wm, wn, acc);
    wait_lgkm0();  // the slots are read before the barrier that lets them go
    if (more) wait_vmcnt<NA + 3>();
    else wait_vmcnt<0>();
    barrier_lds();
    if (more) ld.rows(lds + sa * SLOT_A);
    step<TMX, 1>(lds + next(sa, 1) * SLOT_A, Bs, wm, wn, acc);
    wait_lgkm0();
    sa = next(sa, 2);
  }
}

// Accumulators: lane l has row i * 32 + l % 32 of the wave's tile; register v its
// column j * 32 + 8 (v / 4) + 4 (l / 32) + v % 4.  They leave through LDS.
template <int ROWS, bool SWIGLU>
__device__ __forceinline__ void tile_rows(const GroupedArgs& a, const Tile& t, lds_t* lds) {
  constexpr int TMX = ROWS / 64;
  constexpr int COLS = SWIGLU ? TN / 2 : TN, S = COLS * 2 + 16;
  f32x16_t acc[TMX][2];
  Loads<ROWS> ld;
  ld.template init<SWIGLU>(a, t);
  mainloop<ROWS>(ld, a.K / 128, lds, acc);
  barrier_lds();  // every wave is done with the slots
  const int lane = threadIdx.x & 63, w = wave_id(), wm = w >> 2, wn = w & 3;
#pragma unroll
  for (int i = 0; i < TMX; ++i) {
    lds_t* row = lds + (wm * (ROWS / 2) + i * 32 + (lane & 31)) * S;
#pragma unroll
    for (int j = 0; j < (SWIGLU ? 1 : 2); ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if constexpr (SWIGLU) {
            const float gc = clip_gate(acc[i][0][4 * g + q], a.lim);
            v[q] = gc * sigmoidf_(gc) * clip_up(acc[i][1][4 * g + q], a.lim);
          } else {
            v[q] = acc[i][j][4 * g + q];
          }
        }
        const int col = wn * (COLS / 4) + j * 32 + 8 * g + 4 * (lane >> 5);
        *(__attribute__((address_space(3))) u32x2_t*)(row + col * 2) =
            u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
      }
  }
  wait_lgkm0();
  barrier_lds();
  constexpr int CPR = COLS / 8;
  const int width = SWIGLU ? a.N / 2 : a.N, c0 = t.nt * COLS;
#pragma unroll
  for (int q = threadIdx.x; q < ROWS * CPR; q += NT) {
    const int row = q / CPR, c = c0 + (q % CPR) * 8;
    if (t.m0 + row < t.seg1 && c < width)
      *(u32x4_t*)((bf16_t*)a.y + (int64_t)(t.m0 + row) * width + c) = lds16(lds + row * S + (q % CPR) * 16);
  }
}

template <bool SWIGLU>
__global__ __launch_bounds__(NT) void grouped_tile_kernel(GroupedArgs a, int ntiles) {
  extern __shared__ __align__(16) char smem[];
  lds_t* lds = (lds_t*)smem;
  Tile t;
  if (!find_tile(a, 256, ntiles, &t)) return;
  const int rows = t.seg1 - t.m0;
  if (rows <= 64) tile_rows<64, SWIGLU>(a, t, lds);
  else if (rows <= 128) tile_rows<128, SWIGLU>(a, t, lds);
  else tile_rows<256, SWIGLU>(a, t, lds);
}

template <bool SWIGLU>
hipError_t run(const LaunchCtx& c, const GroupedArgs& a) {
  const int ntiles = (int)cdiv(a.N, TN);
  const int64_t row_tiles = a.R / 256 + std::min<int64_t>(a.E, a.R);  // at most
  // in two dimensions: a grid holds fewer than 2^32 threads along one
  const int64_t groups = cdiv(row_tiles * ntiles, 8) * 8, gx = std::min<int64_t>(groups, 1 << 22);
  const dim3 grid((unsigned)gx, (unsigned)cdiv(groups, gx));
  HIP_RET((allow_smem_once<grouped_tile_kernel<SWIGLU>>(LDS_BYTES)));
  MOE_LAUNCH(c, "grouped_product", grouped_tile_kernel<SWIGLU>, grid, dim3(NT), LDS_BYTES, a, ntiles);
  return hipSuccess;
}

}  // namespace

hipError_t launch_grouped(const LaunchCtx& c, const GroupedArgs& a) {
  return a.swiglu ? run<true>(c, a) : run<false>(c, a);
}

}  // namespace moe
