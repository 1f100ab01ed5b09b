// Products of expert-sorted rows with their experts' MXFP4 matrices, ragged:
//   y[r] = W_e a_r,  offsets[e] <= r < offsets[e + 1],
//   a_r = x[src_of[r] / k] or x[r],
// or, with W_e = [gate; up], y[r] = silu(min(g, L)) clamp(u, -L, L).
//
// Many rows: a work-group makes a tile of 128 rows of one expert by 256 columns
// (128 gate and the same up columns), four waves of 128 x 64 in 32x32x16 MFMAs on
// bf16: a code times its power-of-two scale is a bfloat16 number, so the products
// are those of the decoded weights, summed in float32.  What bounds it is the
// MFMA and what feeds it.  Codes stay codes until they are in registers: a K step
// of 64 moves 16 KB of rows and 8 KB of codes into LDS where bf16 weights would
// take 32 KB, and a lane turns a 16-byte piece (32 codes, one scale) into four
// MFMA operands with 16 conversions beside 16 MFMAs.  The K order inside a step is
// chosen for that: the lanes' halves take columns 0 .. 31 and 32 .. 63, operand kk
// columns 8 kk .. 8 kk + 7 of them, on either side.  The tile is as large as lets
// two work-groups share a CU's LDS and registers, one's barriers under the other's
// products: 131072 rows, K = 2048, N = 1536 with SwiGLU in 686 us, 1.20 PFLOP/s
// (779 with 256 x 256 tiles of eight waves, one work-group a CU; a library's bf16
// product of 8192^3 reaches 1.39), MFMA busy 65%.
//
// Fewer rows: the streaming tiles of mx4tile.h, bounded by the codes' way from
// memory; fewer still: the same with K over the waves.
#include <algorithm>

#include "common.h"
#include "mx4tile.h"
#include "tile.h"

namespace moe {
namespace {

using namespace tile;
using mx4::decode8;
using mx4::lds16;
using mx4::scale_of;
using mx4::Stream;
using mx4::wait_lgkm0;

constexpr int NW = 4, NT = NW * 64;
constexpr int TM = 128, TN = 256;          // rows and columns of W a tile
constexpr int SLOT_A = TM * 128;           // [rows][64 values]
constexpr int CODES_B = TN * 64;           // [columns][128 codes], then their scale words
constexpr int SLOT_B = CODES_B + TN * 4;
constexpr int LDS_BYTES = TM * (TN * 2 + 16);  // the ring, 2 SLOT_A + 2 SLOT_B, is smaller than the tile on its way out
static_assert(2 * SLOT_A + 2 * SLOT_B <= LDS_BYTES && 2 * LDS_BYTES <= 160 * 1024, "");

// An expert's row tile: rows m0 .. of [.., seg1), column tile nt.
struct Tile {
  int e, m0, seg1, nt;
};

// Sums over the lanes up to each: DPP shifts inside rows of 16 lanes, then the
// rows' last lanes to the rows behind.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // row_shr:1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row_bcast:15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // row_bcast:31 into rows 2 and 3
  return v;
}

// The tile of this work-group, every wave for itself: lane l counts the row
// tiles of experts l, l + 64, .., whose offsets it loads all at once.  EPL:
// experts a lane.  False: none.  (A kernel that leaves a table of the tiles
// behind costs a launch, 4 us; this about 1 us of each work-group, beside the
// others' work.)
template <int EPL>
__device__ __forceinline__ bool find_tile(const GroupedArgs& a, int rows, int ntiles, Tile* t) {
  const int lane = threadIdx.x & 63;
  int o0[EPL], o1[EPL], incl[EPL], total = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 64 * i;
    o0[i] = a.offsets[min(e, a.E)];
    o1[i] = a.offsets[min(e + 1, a.E)];
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {  // whatever the offsets hold, rows that there are
    o0[i] = min(max(o0[i], 0), a.R);
    o1[i] = min(max(o1[i], 0), a.R);
    const int n = (max(o1[i] - o0[i], 0) + rows - 1) / rows;
    incl[i] = total + wave_scan(n);
    total = __builtin_amdgcn_readlane(incl[i], 63);
  }
  // Counts of row tiles fit 32 bits whatever the offsets hold (E of them, each at
  // most R / rows + 1: below 2^31 by the largest E and R, and by the launcher's
  // rules, which give long inputs 128 rows a tile), their products with ntiles
  // do not: offsets that go back and forth count rows E / 2 times.  Tiles beyond
  // the grid's are not made (offsets in order never count so many).
  const int64_t groups = (int64_t)gridDim.x * gridDim.y, tiles = (int64_t)total * ntiles;
  const int L = xcd_tile(blockIdx.y * gridDim.x + blockIdx.x, (int)(tiles < groups ? tiles : groups));
  if (L < 0) return false;
  const int row = L / ntiles;  // among all row tiles, were they taken one by one
  int before = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const uint64_t past = __ballot(incl[i] > row);
    if (past) {
      const int l = __builtin_ctzll(past);
      if (l) before = __builtin_amdgcn_readlane(incl[i], l - 1);
      const int n = __builtin_amdgcn_readlane(incl[i], l) - before, at = L - before * ntiles;
      const int rt = a.row_major ? row - before : at % n;
      t->nt = a.row_major ? L - row * ntiles : at / n;
      t->e = l + 64 * i;
      t->m0 = __builtin_amdgcn_readlane(o0[i], l) + rt * rows;
      t->seg1 = __builtin_amdgcn_readlane(o1[i], l);
      return true;
    }
    before = __builtin_amdgcn_readlane(incl[i], 63);
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
template <int TMX>
struct Loads {
  static constexpr int NB = 5;  // loads of codes() a wave
  const char* pa[TMX];
  const char* pb[4];
  const char* ps;
  // Sends the first codes while the rows' indices are on their way (131072 rows of
  // 128 by 1536: 104 us with the codes behind the indices, 97 so).
  template <bool SWIGLU>
  __device__ __forceinline__ void begin(const GroupedArgs& a, const Tile& t, lds_t* first_codes) {
    const int lane = threadIdx.x & 63, w = wave_id();
    int src[TMX];
#pragma unroll
    for (int i = 0; i < TMX; ++i) {  // rows past the segment repeat its last
      const int r = min(t.m0 + 8 * (w + NW * i) + (lane >> 3), t.seg1 - 1);
      src[i] = a.src_of ? a.src_of[r] : r;
    }
    __builtin_amdgcn_sched_barrier(0);
    const int64_t mat = (int64_t)t.e * a.N;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 16 * (w + NW * i) + (lane >> 2);
      pb[i] = (const char*)a.codes + (mat + w_row<SWIGLU>(a, t.nt, row)) * (a.K / 2) + (((lane ^ (row >> 2)) & 3) << 4);
    }
    ps = (const char*)a.scales + (mat + w_row<SWIGLU>(a, t.nt, 64 * w + lane)) * (a.K / 32);
    codes(first_codes);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < TMX; ++i) {
      const int row = 8 * (w + NW * i) + (lane >> 3);
      const int64_t s = a.src_of ? min(max(src[i], 0), a.R - 1) / a.k : src[i];
      pa[i] = (const char*)a.x + s * a.K * 2 + (((lane & 7) ^ mk_swz(row)) << 4);
    }
  }
  __device__ __forceinline__ void rows(lds_t* slot) {
    const int w = wave_id();
#pragma unroll
    for (int i = 0; i < TMX; ++i) {
      dma16(pa[i], slot + (w + NW * i) * 1024);
      pa[i] += 128;
    }
  }
  __device__ __forceinline__ void codes(lds_t* slot) {
    const int w = wave_id();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      dma16(pb[i], slot + (w + NW * i) * 1024);
      pb[i] += 64;
    }
    dma4(ps, slot + CODES_B + w * 256);
    ps += 4;
  }
};

// One K step (P: the first or second half of the codes' 128 columns).  The
// operands of the next quarter are read and decoded while a quarter's products
// run.
template <int TMX, int P>
__device__ __forceinline__ void step(const lds_t* __restrict__ As, const lds_t* __restrict__ Bs,
                                     f32x16_t (&acc)[TMX][2]) {
  const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5, w = wave_id();
  u32x4_t code[2];
  uint32_t word[2];
  bf16x8_t av[2][TMX], bv[2][2];
  const auto rows = [&](int kk, bf16x8_t (&v)[TMX]) {
#pragma unroll
    for (int i = 0; i < TMX; ++i) v[i] = __builtin_bit_cast(bf16x8_t, lds16(As + mk_off(i * 32 + r, 4 * h + kk)));
  };
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int n = w * 64 + j * 32 + r;
    word[j] = *(const __attribute__((address_space(3))) uint32_t*)(Bs + CODES_B + n * 4);
    code[j] = lds16(Bs + n * 64 + (((2 * P + h) ^ (n >> 2)) & 3) * 16);
  }
  rows(0, av[0]);
  __builtin_amdgcn_sched_barrier(0);
  float s[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    s[j] = scale_of(word[j], 16 * P + 8 * h);
    bv[0][j] = decode8(code[j][0], s[j]);
  }
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) {
    const int c = kk & 1;
    if (kk < 3) rows(kk + 1, av[c ^ 1]);
#pragma unroll
    for (int i = 0; i < TMX; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bv[c][j], av[c][i], acc[i][j], 0, 0, 0);
    if (kk < 3) {
#pragma unroll
      for (int j = 0; j < 2; ++j) bv[c ^ 1][j] = decode8(code[j][kk + 1], s[j]);
      // a read and some of the conversions after each product
#pragma unroll
      for (int q = 0; q < 2 * TMX; ++q) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                   // MFMA
        if (q < TMX) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);      // DS read
        __builtin_amdgcn_sched_group_barrier(0x002, TMX > 2 ? 2 : 4, 0);     // VALU
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

// Rows of step k are in slot k mod 2, filled during step k - 1; codes of steps
// 2 p and 2 p + 1 in slot p mod 2, filled during the pair before.  Two
// work-groups share a CU, so that one's barriers and waits pass under the
// other's products.  Loads land in the order they left.
template <int TMX>
__device__ __forceinline__ void mainloop(Loads<TMX>& ld, int pairs, lds_t* lds, f32x16_t (&acc)[TMX][2]) {
#pragma unroll
  for (int i = 0; i < TMX; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
  lds_t* const lb = lds + 2 * SLOT_A;
  ld.rows(lds);
  for (int p = 0; p < pairs; ++p) {
    const bool more = p + 1 < pairs;
    const lds_t* Bs = lb + (p & 1) * SLOT_B;
    wait_vmcnt<0>();
    wait_lgkm0();  // the slots are read before the barrier that lets them go
    barrier_lds();
    ld.rows(lds + SLOT_A);
    if (more) ld.codes(lb + ((p & 1) ^ 1) * SLOT_B);
    step<TMX, 0>(lds, Bs, acc);
    if (more) wait_vmcnt<Loads<TMX>::NB>();
    else wait_vmcnt<0>();
    wait_lgkm0();
    barrier_lds();
    if (more) ld.rows(lds);
    step<TMX, 1>(lds + SLOT_A, Bs, acc);
  }
  wait_lgkm0();
  barrier_lds();  // every wave is done with the slots
}

// Accumulators: lane l has row i * 32 + l % 32 of the tile; register v the wave's
// column j * 32 + 8 (v / 4) + 4 (l / 32) + v % 4.  They leave through LDS, by
// non-temporal stores (131072 rows of 256 by 1024: 111 us without, 92 with).
template <int TMX, bool SWIGLU>
__device__ __forceinline__ void tile_rows(const GroupedArgs& a, const Tile& t, lds_t* lds) {
  constexpr int COLS = SWIGLU ? TN / 2 : TN, S = COLS * 2 + 16;
  f32x16_t acc[TMX][2];
  Loads<TMX> ld;
  ld.template begin<SWIGLU>(a, t, lds + 2 * SLOT_A);
  mainloop<TMX>(ld, a.K / 128, lds, acc);
  const int lane = threadIdx.x & 63, w = wave_id();
#pragma unroll
  for (int i = 0; i < TMX; ++i) {
    lds_t* row = lds + (i * 32 + (lane & 31)) * S;
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
        const int col = w * (COLS / 4) + j * 32 + 8 * g + 4 * (lane >> 5);
        *(__attribute__((address_space(3))) u32x2_t*)(row + col * 2) =
            u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
      }
  }
  wait_lgkm0();
  barrier_lds();
  constexpr int CPR = COLS / 8;
  const int width = SWIGLU ? a.N / 2 : a.N, c0 = t.nt * COLS;
  for (int q = threadIdx.x; q < TMX * 32 * CPR; q += NT) {
    const int row = q / CPR, c = c0 + (q % CPR) * 8;
    if (t.m0 + row < t.seg1 && c < width)
      __builtin_nontemporal_store(lds16(lds + row * S + (q % CPR) * 16),
                                  (u32x4_t*)((bf16_t*)a.y + (int64_t)(t.m0 + row) * width + c));
  }
}

template <bool SWIGLU, int EPL>
__global__ __launch_bounds__(NT, 2) void grouped_tile_kernel(GroupedArgs a, int ntiles) {
  extern __shared__ __align__(16) char smem[];
  lds_t* lds = (lds_t*)smem;
  Tile t;
  if (!find_tile<EPL>(a, TM, ntiles, &t)) return;
  const int rows = t.seg1 - t.m0;
  if (rows <= 32) tile_rows<1, SWIGLU>(a, t, lds);
  else if (rows <= 64) tile_rows<2, SWIGLU>(a, t, lds);
  else if (rows <= 96) tile_rows<3, SWIGLU>(a, t, lds);
  else tile_rows<4, SWIGLU>(a, t, lds);
}

// Few rows an expert: tiles of SROWS rows (16, 32 or 48 where there are no more) by
// 64 CB columns, or 32 CB gate and the same up columns.
// Row i of a tile (past the segment its last; its entry with src_of) and where that
// is, and the row of W for its column n (past the last that; SWIGLU: 16 gate, the
// same up, in turn).
__device__ __forceinline__ int index_of(const GroupedArgs& a, const Tile& t, int i) {
  const int r = min(t.m0 + i, t.seg1 - 1);
  return a.src_of ? a.src_of[r] : r;
}
__device__ __forceinline__ const char* row_at(const GroupedArgs& a, int index) {
  const int64_t s = a.src_of ? min(max(index, 0), a.R - 1) / a.k : index;
  return (const char*)a.x + s * a.K * 2;
}
template <bool SWIGLU, int COLS>
__device__ __forceinline__ int64_t col_at(const GroupedArgs& a, const Tile& t, int n) {
  const int64_t mat = (int64_t)t.e * a.N;
  if constexpr (SWIGLU) {
    const int c = min(t.nt * COLS + (n >> 5) * 16 + (n & 15), a.N / 2 - 1);
    return mat + ((n & 16) ? a.N / 2 + c : c);
  } else {
    return mat + min(t.nt * COLS + n, a.N - 1);
  }
}

template <class C, bool SWIGLU>
__device__ __forceinline__ void stream_rows(const GroupedArgs& a, const Tile& t, lds_t* lds) {
  constexpr int COLS = SWIGLU ? C::COLS / 2 : C::COLS, S = COLS * 2 + 16;
  static_assert(C::ROWS * S <= C::LDS && (!SWIGLU || C::CB % 2 == 0), "");
  Stream<C> st;
  st.begin([&](int i) { return index_of(a, t, i); }, [&](int index) { return row_at(a, index); },
           [&](int n) { return col_at<SWIGLU, COLS>(a, t, n); }, a.codes, a.scales, a.K, lds);
  f32x4_t acc[C::RB][C::CB];
  mx4::products<C>(st, a.K / 128, lds, acc);
  const int lane = threadIdx.x & 63, w = wave_id();
#pragma unroll
  for (int b = 0; b < C::RB; ++b) {
    lds_t* row = lds + (16 * b + (lane & 15)) * S + (w * (COLS / 4) + 4 * (lane >> 4)) * 2;
#pragma unroll
    for (int c = 0; c < (SWIGLU ? C::CB / 2 : C::CB); ++c) {
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (SWIGLU) {
          const float gc = clip_gate(acc[b][2 * c][i], a.lim);
          v[i] = gc * sigmoidf_(gc) * clip_up(acc[b][2 * c + 1][i], a.lim);
        } else {
          v[i] = acc[b][c][i];
        }
      }
      *(__attribute__((address_space(3))) u32x2_t*)(row + c * 32) =
          u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    }
  }
  wait_lgkm0();
  barrier_lds();
  constexpr int CPR = COLS / 8;
  const int width = SWIGLU ? a.N / 2 : a.N, c0 = t.nt * COLS;
  for (int i = threadIdx.x; i < C::ROWS * CPR; i += 256) {
    const int row = i / CPR, c = c0 + (i % CPR) * 8;
    if (t.m0 + row < t.seg1 && c < width)
      __builtin_nontemporal_store(lds16(lds + row * S + (i % CPR) * 16),
                                  (u32x4_t*)((bf16_t*)a.y + (int64_t)(t.m0 + row) * width + c));
  }
}

template <int CB> using Rows16 = mx4::Tiles<1, CB, CB == 2 ? 2 : 1>;
template <int CB> using Rows32 = mx4::Tiles<2, CB, CB == 2 ? 2 : 1>;
template <int CB> using Rows48 = mx4::Tiles<3, CB, 1>;
template <int CB> using Rows64 = mx4::Tiles<4, CB, 1>;
using Split16 = mx4::SplitTiles<1, 3>;
using Split32 = mx4::SplitTiles<2, 2>;
constexpr int kSplitLds = std::max(Split16::LDS, Split32::LDS);
template <int CB, int SROWS>
constexpr int kStreamLds = std::max({Rows16<CB>::LDS, Rows32<CB>::LDS, SROWS == 64 ? Rows64<CB>::LDS : 0});

template <int CB, int SROWS, bool SWIGLU, int EPL>
__global__ __launch_bounds__(256) void grouped_stream_kernel(GroupedArgs a, int ntiles) {
  extern __shared__ __align__(16) char smem[];
  lds_t* lds = (lds_t*)smem;
  Tile t;
  if (!find_tile<EPL>(a, SROWS, ntiles, &t)) return;
  const int rows = t.seg1 - t.m0;
  if (rows <= 16) stream_rows<Rows16<CB>, SWIGLU>(a, t, lds);
  else if (SROWS == 32 || rows <= 32) stream_rows<Rows32<CB>, SWIGLU>(a, t, lds);
  else if constexpr (SROWS == 64) {
    if (rows <= 48) stream_rows<Rows48<CB>, SWIGLU>(a, t, lds);
    else stream_rows<Rows64<CB>, SWIGLU>(a, t, lds);
  }
}

// The same where they would leave the chip idle: 32 rows by 64 columns (32 gate,
// the same up), K over the waves.
constexpr int PROWS = 32;

template <class C, bool SWIGLU>
__device__ __forceinline__ void split_rows(const GroupedArgs& a, const Tile& t, lds_t* lds) {
  constexpr int COLS = SWIGLU ? C::COLS / 2 : C::COLS;
  mx4::SplitStream<C> st;
  st.begin([&](int i) { return index_of(a, t, i); }, [&](int index) { return row_at(a, index); },
           [&](int n) { return col_at<SWIGLU, COLS>(a, t, n); }, a.codes, a.scales, a.K, lds);
  f32x4_t acc[C::RB][4];
  // a wave finishes one block of 16 columns, or of gate and up
  const auto keep = [](int w, int c) { return SWIGLU ? (c >> 1) == w : c == w; };
  mx4::split_products<C>(st, a.K / 128, lds, acc, keep);
  const int lane = threadIdx.x & 63, w = wave_id(), width = SWIGLU ? a.N / 2 : a.N;
#pragma unroll
  for (int c = 0; c < (SWIGLU ? 2 : 4); ++c) {
    if (c != w) continue;
    const int col = t.nt * COLS + 16 * c + 4 * (lane >> 4);
#pragma unroll
    for (int b = 0; b < C::RB; ++b) {
      const int r = t.m0 + 16 * b + (lane & 15);
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (SWIGLU) {
          const float gc = clip_gate(acc[b][2 * c][i], a.lim);
          v[i] = gc * sigmoidf_(gc) * clip_up(acc[b][2 * c + 1][i], a.lim);
        } else {
          v[i] = acc[b][c][i];
        }
      }
      if (r < t.seg1 && col < width)  // the width is a multiple of 8
        *(u32x2_t*)((bf16_t*)a.y + (int64_t)r * width + col) =
            u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    }
  }
}

template <bool SWIGLU, int EPL>
__global__ __launch_bounds__(256) void grouped_split_kernel(GroupedArgs a, int ntiles) {
  extern __shared__ __align__(16) char smem[];
  lds_t* lds = (lds_t*)smem;
  Tile t;
  if (!find_tile<EPL>(a, PROWS, ntiles, &t)) return;
  if (t.seg1 - t.m0 <= 16) split_rows<Split16, SWIGLU>(a, t, lds);
  else split_rows<Split32, SWIGLU>(a, t, lds);
}

// A grid of at least `groups`, in two dimensions: one holds fewer than 2^32
// threads along one.
dim3 grid_of(int64_t groups) {
  groups = cdiv(groups, 8) * 8;
  const int64_t gx = std::min<int64_t>(groups, 1 << 22);
  return dim3((unsigned)gx, (unsigned)cdiv(groups, gx));
}

template <int CB, int SROWS, bool SWIGLU, int EPL>
hipError_t run_stream(const LaunchCtx& c, const GroupedArgs& a, int64_t experts) {
  const int ntiles = (int)cdiv(a.N, 64 * CB);
  HIP_RET((allow_smem_once<grouped_stream_kernel<CB, SROWS, SWIGLU, EPL>>(kStreamLds<CB, SROWS>)));
  MOE_LAUNCH(c, "grouped_product", (grouped_stream_kernel<CB, SROWS, SWIGLU, EPL>),
             grid_of((a.R / SROWS + experts) * ntiles), dim3(256), (kStreamLds<CB, SROWS>), a, ntiles);
  return hipSuccess;
}

template <bool SWIGLU, int EPL>
hipError_t run(const LaunchCtx& c, const GroupedArgs& a) {
  const int64_t experts = std::min<int64_t>(a.E, a.R);  // with rows, at most
  const auto groups = [&](int rows, int cols) { return std::max<int64_t>(experts, a.R / rows) * cdiv(a.N, cols); };
  // K over the waves: up to a work-group a CU, and enough of K to share out (us
  // with tiles of 64 by 128 and with these: 8 rows of 8 experts, K = 2048, N =
  // 1536, 192 work-groups, 9.9 and 7.4; 100 rows of one, K = N = 2048, 96, 15.3
  // and 8.6; 16 of 16, 384, 10.1 and 12.3; 4 of one, K = 640, 4.3 and 5.2).
  if (groups(PROWS, 64) <= 256 && a.K >= 1024) {
    const int ntiles = (int)cdiv(a.N, 64);
    HIP_RET((allow_smem_once<grouped_split_kernel<SWIGLU, EPL>>(kSplitLds)));
    MOE_LAUNCH(c, "grouped_product", (grouped_split_kernel<SWIGLU, EPL>), grid_of((a.R / PROWS + experts) * ntiles),
               dim3(256), kSplitLds, a, ntiles);
    return hipSuccess;
  }
  // tiles of 128 rows: more than 48 rows an expert, and one for each CU (us with
  // them and with 64 by 256: 64 rows of 128 experts, K = 2048, N = 1536, 83 and
  // 91, 32 rows 68 and 65; 2000 rows of one, K = N = 4096, 256 work-groups, 64 and
  // 66; 250 rows of 8, 96, 31 and 25)
  const bool tall = a.R > 48 * (int64_t)a.E && groups(TM, TN) >= 256;
  if (!tall) {
    // 64 rows by 256 columns: more than 20 rows an expert, and one for each CU (us
    // with them and with 64 by 128: 44 rows of 128, K = 1536, N = 4096, 122 and 133;
    // 25 of 64, K = 4096, N = 2048, 71 and 75; 16 of 128, K = 2048, N = 1536, 56 and
    // 50; 2 of 128 49 and 41; 250 of 8, 186 work-groups, 25 and 22)
    if (a.R > 20 * (int64_t)a.E && groups(64, 256) >= 256) return run_stream<4, 64, SWIGLU, EPL>(c, a, experts);
    // and 32 by 128 where those are fewer than CUs (75 rows of 8 experts, 108: 17.3
    // and 15.1; 500 of one, K = N = 2048, 128: 18 and 13; 250 of 8, 372: 22 and 28)
    if (groups(64, 128) >= 256) return run_stream<2, 64, SWIGLU, EPL>(c, a, experts);
    return run_stream<2, 32, SWIGLU, EPL>(c, a, experts);
  }
  const int ntiles = (int)cdiv(a.N, TN);
  HIP_RET((allow_smem_once<grouped_tile_kernel<SWIGLU, EPL>>(LDS_BYTES)));
  MOE_LAUNCH(c, "grouped_product", (grouped_tile_kernel<SWIGLU, EPL>), grid_of((a.R / TM + experts) * ntiles), dim3(NT),
             LDS_BYTES, a, ntiles);
  return hipSuccess;
}

}  // namespace

hipError_t launch_grouped(const LaunchCtx& c, GroupedArgs a) {
  // Either order of an expert's tiles reads one operand again from the caches:
  // along the rows' tiles the expert's codes (N K / 2 bytes), along the columns'
  // its rows (2 K each).  The smaller one (1024 rows an expert, N = 1536: 695 us
  // with the codes again, 717 with the rows).
  a.row_major = 4 * (int64_t)a.R >= (int64_t)a.E * a.N;
  if (a.E <= 128) return a.swiglu ? run<true, 2>(c, a) : run<false, 2>(c, a);
  return a.swiglu ? run<true, 16>(c, a) : run<false, 16>(c, a);
}

}  // namespace moe
