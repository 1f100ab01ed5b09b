// Few rows times MXFP4 matrices: the streaming tile of the grouped products and
// of the few-token layer.
//
// Four waves make 16 RB rows by 64 CB columns of W, a wave 16 CB of them, in
// 16x16x32 MFMAs on bf16 (a code times its scale is exact in bfloat16).  What
// bounds it is the stream of codes, moved by direct loads: a stage is H times 128
// values of K (64 bytes of each column, 256 of each row), loaded one stage ahead,
// one barrier a stage, two work-groups a CU (a kernel's LDS is that of the tallest
// tile it may take, 68 or 72 KB).  The K order inside 128 values suits the codes: a
// quarter of a wave takes a 16-byte piece of its column (32 codes, one scale), whose
// four words are four MFMA operands.  The reads of rows, of 64-byte codes and of
// scale words meet each bank twice; LDS is active 18 to 30% of the time so.
//
// What it measured at 33 tokens of 8 of 128 experts, K = 2048, N = 1536 (188 MB of
// codes and scales): 57 us with 32x32x16 products of 32 columns a wave, whose rows
// are read from LDS once for two products; 47 with these, 64 columns a wave; 44
// with three slots of one 128-value stage; 40 with H = 2 and 128 columns a
// work-group, 4.7 TB/s: whole 128-byte lines are asked for (a kernel that only
// loads reads 4.7 TB/s in 64-byte pieces of 256 rows 2 KB apart, and 6.0 in
// 128-byte ones of 128; the two halves of a line in loads of their own: 41).  Where
// more rows leave LDS for 128 values only (RB > 2), wider tiles pay instead.
#pragma once

#include "common.h"
#include "tile.h"

namespace moe {
namespace mx4 {

using namespace tile;

__device__ __forceinline__ void wait_lgkm0() { __builtin_amdgcn_s_waitcnt(0xC07F); }  // lgkmcnt(0) alone

__device__ __forceinline__ u32x4_t lds16(const lds_t* p) {
  return *(const __attribute__((address_space(3))) u32x4_t*)p;
}

// An E8M0 byte as the float whose exponent the conversion takes (0 stands for
// 2^-127, 255 for NaN).
__device__ __forceinline__ float scale_of(uint32_t word, int shift) {
  return __uint_as_float(((word >> shift) & 0xffu) << 23);
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

constexpr int kWaves = 4;

// Two slots of a stage.  The scales are kept apart, four words of a column together
// (512 values), in two buffers: a load of one word from each of 64 columns costs
// the vector memory unit as much as 1 KB of codes.
template <int RB_, int CB_, int H_>
struct Tiles {
  static constexpr int RB = RB_, CB = CB_, H = H_;
  static constexpr int ROWS = 16 * RB, COLS = 64 * CB;
  static constexpr int A = ROWS * 256;
  static constexpr int B = 64 * H;  // bytes of a column's codes, beside each other
  static constexpr int STAGE = H * A + COLS * B;
  static constexpr int SCALES = COLS * 16;
  static constexpr int LDS = 2 * (STAGE + SCALES);
};

// One stage's operands of a wave into registers and its products; `col`: the
// wave's first column in B, whose scale word is at `scales`.  Every read leaves
// before the first product waits for one.
template <int RB, int CB, int BS = 64>
__device__ __forceinline__ void stage_products(const lds_t* A, const lds_t* B, const lds_t* scales, int col,
                                               int scale_stride, f32x4_t (&acc)[RB][CB], int h = 0) {
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  uint32_t word[CB];
  u32x4_t code[CB], av[4][RB];
#pragma unroll
  for (int c = 0; c < CB; ++c) {
    const int n = col + 16 * c + r;
    word[c] = *(const __attribute__((address_space(3))) uint32_t*)(scales + (16 * c + r) * scale_stride);
    if constexpr (BS == 128) code[c] = lds16(B + n * 128 + (((4 * h + q) ^ n) & 7) * 16);
    else code[c] = lds16(B + n * 64 + ((q ^ (n >> 2)) & 3) * 16);
  }
#pragma unroll
  for (int kk = 0; kk < 4; ++kk)
#pragma unroll
    for (int b = 0; b < RB; ++b) av[kk][b] = lds16(A + (16 * b + r) * 256 + (((4 * q + kk) ^ r) & 15) * 16);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int c = 0; c < CB; ++c) {
    const float s = scale_of(word[c], 8 * q);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      const bf16x8_t bv = decode8(code[c][kk], s);
#pragma unroll
      for (int b = 0; b < RB; ++b)
        acc[b][c] =
            __builtin_amdgcn_mfma_f32_16x16x32_bf16(bv, __builtin_bit_cast(bf16x8_t, av[kk][b]), acc[b][c], 0, 0, 0);
    }
  }
}

// This lane's sources: row_at(index_of(i)) is the address of tile row i of the
// activations, col_at(n) the row of W (among all experts') that column n stands for.
template <class C>
struct Stream {
  static constexpr int NC = C::CB * C::H;  // 1 KB loads of codes: 16 / H columns
  const char* pa[C::RB];
  const char* pb[NC];
  const char* ps[C::CB];
  // Sends the first stage's loads: first those of the rows' indices, then the codes'
  // and scales', and the rows' when the indices are there.
  template <class IndexOf, class RowAt, class ColAt>
  __device__ __forceinline__ void begin(IndexOf index_of, RowAt row_at, ColAt col_at, const uint8_t* codes,
                                        const uint8_t* scales, int K, lds_t* lds) {
    const int lane = threadIdx.x & 63, w = wave_id(), units = K / 128;
    int index[C::RB];
#pragma unroll
    for (int i = 0; i < C::RB; ++i) index[i] = index_of(4 * (w + kWaves * i) + (lane >> 4));
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < C::CB; ++i)
      ps[i] = (const char*)scales + col_at(16 * (w * C::CB + i) + (lane >> 2)) * (K / 32);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int n = C::H == 2 ? 8 * (w * NC + i) + (lane >> 3) : 16 * (w * NC + i) + (lane >> 2);
      pb[i] = (const char*)codes + col_at(n) * (K / 2) + (C::H == 2 ? (lane ^ n) & 7 : (lane ^ (n >> 2)) & 3) * 16;
    }
    issue_codes(lds, units);
#pragma unroll
    for (int i = 0; i < C::CB; ++i) this->scales(i, 0, units, lds + 2 * C::STAGE);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < C::RB; ++i) {
      const int r = 4 * (w + kWaves * i) + (lane >> 4);
      pa[i] = row_at(index[i]) + (((lane ^ r) & 15) << 4);
    }
    issue_rows(lds, units);
  }
  // Words 4 g .. of 16 of the wave's columns (past the row's end its last word).
  __device__ __forceinline__ void scales(int i, int g, int stages, lds_t* buffer) const {
    const int word = min(4 * g + (int)(threadIdx.x & 3), stages - 1);
    dma4(ps[i] + 4 * word, buffer + (wave_id() * C::CB + i) * 256);
  }
  // `halves` of H: the last stage may be short.
  __device__ __forceinline__ void issue_codes(lds_t* slot, int halves) {
    const int w = wave_id();
    // a short stage repeats its codes: none are behind
    const int lane = threadIdx.x & 63;
    const int back = halves < C::H ? ((lane ^ (lane >> 3)) & 4) << 4 : 0;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      dma16(pb[i] - back, slot + C::H * C::A + (w * NC + i) * 1024);
      pb[i] += C::B;
    }
  }
  __device__ __forceinline__ void issue_rows(lds_t* slot, int halves) {
    const int w = wave_id();
#pragma unroll
    for (int i = 0; i < C::RB; ++i) {
#pragma unroll
      for (int h = 0; h < C::H; ++h)
        if (h < halves) dma16(pa[i] + 256 * h, slot + h * C::A + (w + kWaves * i) * 1024);
      pa[i] += 256 * C::H;
    }
  }
};

// acc[b][c]: lane l has row 16 b + l % 16; register v the wave's column 16 c +
// 4 (l / 16) + v.  units: K / 128; the first stage is on its way.
template <class C>
__device__ __forceinline__ void products(Stream<C>& st, int units, lds_t* lds, f32x4_t (&acc)[C::RB][C::CB]) {
  constexpr int H = C::H, PER = 4 / H;  // stages a group of scale words
  static_assert(C::CB % PER == 0 || C::CB < PER, "");
  const int w = wave_id(), stages = (units + H - 1) / H;
  lds_t* const words = lds + 2 * C::STAGE;
#pragma unroll
  for (int b = 0; b < C::RB; ++b)
#pragma unroll
    for (int c = 0; c < C::CB; ++c) acc[b][c] = f32x4_t{0, 0, 0, 0};
  for (int p = 0; p < stages; ++p) {
    const int g = p / PER;
    wait_vmcnt<0>();
    wait_lgkm0();  // the slot and the buffer to be filled have been read
    barrier_lds();
    if (p + 1 < stages) {
      // with each stage's loads some of the next group's words
#pragma unroll
      for (int i = 0; i < C::CB; ++i)
        if (p % PER == i % PER) st.scales(i, g + 1, units, words + ((g & 1) ^ 1) * C::SCALES);
      st.issue_codes(lds + ((p & 1) ^ 1) * C::STAGE, units - (p + 1) * H);
      st.issue_rows(lds + ((p & 1) ^ 1) * C::STAGE, units - (p + 1) * H);
    }
    const lds_t* A = lds + (p & 1) * C::STAGE;
    const lds_t* word = words + (g & 1) * C::SCALES + w * C::CB * 256 + (p % PER) * H * 4;
#pragma unroll
    for (int h = 0; h < H; ++h)
      if (h == 0 || p * H + h < units)
        stage_products<C::RB, C::CB, C::B>(A + h * C::A, A + H * C::A, word + h * 4, 16 * C::CB * w, 16, acc, h);
  }
  wait_lgkm0();
  barrier_lds();  // the slots are free
}

// ------------------------------------------------------------- K over the waves
// Where the tiles above are too few to fill the chip: a work-group makes 16 RB
// rows by 64 columns, its waves taking every fourth stage each in a ring of its
// own (no barriers), and their sums meet in LDS, in wave order.
template <int RB_, int NS_>
struct SplitTiles {
  static constexpr int RB = RB_, CB = 4, NS = NS_;
  static constexpr int ROWS = 16 * RB, COLS = 64;
  static constexpr int A = ROWS * 256, CODES = COLS * 64;
  static constexpr int STAGE = A + CODES + 256;
  static constexpr int PARTS = kWaves * RB * CB * 1024;
  static constexpr int LDS = STAGE * NS * kWaves > PARTS ? STAGE * NS * kWaves : PARTS;
};

template <class C>
struct SplitStream {
  static constexpr int NA = 4 * C::RB, LOADS = NA + 5;
  const char* pa[NA];
  const char* pb[4];
  const char* ps;
  // Sends the wave's first stage, as Stream::begin does.
  template <class IndexOf, class RowAt, class ColAt>
  __device__ __forceinline__ void begin(IndexOf index_of, RowAt row_at, ColAt col_at, const uint8_t* codes,
                                        const uint8_t* scales, int K, lds_t* lds) {
    const int lane = threadIdx.x & 63, w = wave_id();
    lds_t* const slot = lds + w * C::NS * C::STAGE;
    int index[NA];
#pragma unroll
    for (int i = 0; i < NA; ++i) index[i] = index_of(4 * i + (lane >> 4));
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = 16 * i + (lane >> 2);
      pb[i] = (const char*)codes + col_at(n) * (K / 2) + (((lane ^ (n >> 2)) & 3) << 4) + w * 64;
    }
    ps = (const char*)scales + col_at(lane) * (K / 32) + w * 4;
    if (w < K / 128) issue_codes(slot);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const int r = 4 * i + (lane >> 4);
      pa[i] = row_at(index[i]) + (((lane ^ r) & 15) << 4) + w * 256;
    }
    if (w < K / 128) issue_rows(slot);
  }
  __device__ __forceinline__ void issue_codes(lds_t* slot) {
    lds_t* const b = slot + C::A;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      dma16(pb[i], b + i * 1024);
      pb[i] += 64 * kWaves;
    }
    dma4(ps, b + C::CODES);
    ps += 4 * kWaves;
  }
  __device__ __forceinline__ void issue_rows(lds_t* slot) {
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      dma16(pa[i], slot + i * 1024);
      pa[i] += 256 * kWaves;
    }
  }
  __device__ __forceinline__ void issue(lds_t* slot) {
    issue_codes(slot);
    issue_rows(slot);
  }
};

// The work-group's sums: each wave gets all rows of the 16-column blocks c with
// keep(wave, c), as products() leaves them; the others' acc hold parts.
template <class C, class Keep>
__device__ __forceinline__ void split_products(SplitStream<C>& st, int stages, lds_t* lds, f32x4_t (&acc)[C::RB][4],
                                               Keep keep) {
  constexpr int NS = C::NS, L = SplitStream<C>::LOADS;
  const int w = wave_id(), lane = threadIdx.x & 63;
  const int mine = (stages - w + kWaves - 1) / kWaves;
  lds_t* const ring = lds + w * NS * C::STAGE;
#pragma unroll
  for (int b = 0; b < C::RB; ++b)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[b][c] = f32x4_t{0, 0, 0, 0};
#pragma unroll
  for (int i = 1; i < NS - 1; ++i)
    if (i < mine) st.issue(ring + i * C::STAGE);
  int slot = 0;
  for (int p = 0; p < mine; ++p) {
    const int behind = mine - 1 - p;
    wait_lgkm0();  // the slot to be filled has been read
    if (behind >= NS - 1) st.issue(ring + (slot == 0 ? NS - 1 : slot - 1) * C::STAGE);
    if (behind >= NS - 1) wait_vmcnt<(NS - 1) * L>();
    else if (NS > 2 && behind == 1) wait_vmcnt<L>();
    else wait_vmcnt<0>();
    asm volatile("" ::: "memory");  // no read moves above the wait
    const lds_t* A = ring + slot * C::STAGE;
    const lds_t* B = A + C::A;
    stage_products<C::RB, 4>(A, B, B + C::CODES, 0, 4, acc);
    asm volatile("" ::: "memory");
    slot = slot + 1 == NS ? 0 : slot + 1;
  }
  wait_lgkm0();
  barrier_lds();  // the rings are free
#pragma unroll
  for (int b = 0; b < C::RB; ++b)
#pragma unroll
    for (int c = 0; c < 4; ++c)
      *(__attribute__((address_space(3))) f32x4_t*)(lds + ((w * C::RB + b) * 4 + c) * 1024 + lane * 16) = acc[b][c];
  wait_lgkm0();
  barrier_lds();
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    if (!keep(w, c)) continue;
#pragma unroll
    for (int b = 0; b < C::RB; ++b) {
      f32x4_t s = {0, 0, 0, 0};
#pragma unroll
      for (int v = 0; v < kWaves; ++v) {
        const f32x4_t x =
            *(const __attribute__((address_space(3))) f32x4_t*)(lds + ((v * C::RB + b) * 4 + c) * 1024 + lane * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] += x[i];
      }
      acc[b][c] = s;
    }
  }
}

}  // namespace mx4
}  // namespace moe
