// Few rows times MXFP4 matrices: the streaming tile of the grouped products and
// of the few-token layer.
//
// Four waves make 16 RB rows by 64 CB columns of W, a wave 16 CB of them, in
// 16x16x32 MFMAs on bf16 (a code times its scale is exact in bfloat16).  What
// bounds it is the stream of codes, so it is kept in flight: a stage is 128
// values of K (64 bytes and four scales of each column, 256 bytes of each row),
// moved by direct loads into a ring of NS slots, NS - 1 ahead, one barrier a
// stage, two or three work-groups a CU.  The K order inside a stage suits the
// codes: a quarter of a wave takes a 16-byte piece of its column (32 codes, one
// scale), whose four words are four MFMA operands.  Next to the stream the LDS
// reads are what costs: each wave reads all rows and its own columns, so it
// takes as many columns as leave enough work-groups (RB CB products for RB + CB
// operands).
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

template <int RB_, int CB_, int NS_>
struct Tiles {
  static constexpr int RB = RB_, CB = CB_, NS = NS_;
  static constexpr int ROWS = 16 * RB, COLS = 64 * CB;
  static constexpr int A = ROWS * 256, CODES = COLS * 64;
  static constexpr int SCALES = 256 * kWaves;  // a word a column, 64 a wave (with 32 columns: twice)
  static constexpr int STAGE = A + CODES + SCALES;
  static constexpr int LDS = STAGE * NS;
};

// One stage's operands of a wave into registers and its products; `col`: the
// wave's first column in B.  Every read leaves before the first product waits
// for one.
template <int RB, int CB>
__device__ __forceinline__ void stage_products(const lds_t* A, const lds_t* B, const lds_t* scales, int col,
                                               f32x4_t (&acc)[RB][CB]) {
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  uint32_t word[CB];
  u32x4_t code[CB], av[4][RB];
#pragma unroll
  for (int c = 0; c < CB; ++c) {
    const int n = col + 16 * c + r;
    word[c] = *(const __attribute__((address_space(3))) uint32_t*)(scales + (16 * c + r) * 4);
    code[c] = lds16(B + n * 64 + ((q ^ (n >> 2)) & 3) * 16);
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

// This lane's sources: row_at(i) is the address of tile row i of the activations,
// col_at(n) the row of W (among all experts') that column n stands for.
template <class C>
struct Stream {
  // 1 KB of rows a load, dealt to the waves; a single KB's other waves load it again
  static constexpr int NA = C::RB, LOADS = C::RB + C::CB + 1;
  const char* pa[NA];
  const char* pb[C::CB];
  const char* ps;
  template <class RowAt, class ColAt>
  __device__ __forceinline__ void init(RowAt row_at, ColAt col_at, const uint8_t* codes, const uint8_t* scales, int K) {
    const int lane = threadIdx.x & 63, w = wave_id();
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const int r = 4 * (w + kWaves * i) + (lane >> 4);
      pa[i] = row_at(r) + (((lane ^ r) & 15) << 4);
    }
#pragma unroll
    for (int i = 0; i < C::CB; ++i) {
      const int n = 16 * (w * C::CB + i) + (lane >> 2);
      pb[i] = (const char*)codes + col_at(n) * (K / 2) + (((lane ^ (n >> 2)) & 3) << 4);
    }
    ps = (const char*)scales + col_at(16 * C::CB * w + (lane & (16 * C::CB - 1))) * (K / 32);
  }
  __device__ __forceinline__ void issue(lds_t* slot) {
    const int w = wave_id();
    lds_t* const b = slot + C::A;
#pragma unroll
    for (int i = 0; i < C::CB; ++i) {
      dma16(pb[i], b + (w * C::CB + i) * 1024);
      pb[i] += 64;
    }
    dma4(ps, b + C::CODES + w * 256);
    ps += 4;
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      dma16(pa[i], slot + (w + kWaves * i) * 1024);
      pa[i] += 256;
    }
  }
};

// acc[b][c]: lane l has row 16 b + l % 16; register v the wave's column 16 c +
// 4 (l / 16) + v.
template <class C>
__device__ __forceinline__ void products(Stream<C>& st, int stages, lds_t* lds, f32x4_t (&acc)[C::RB][C::CB]) {
  constexpr int NS = C::NS, L = Stream<C>::LOADS;
  const int w = wave_id();
#pragma unroll
  for (int b = 0; b < C::RB; ++b)
#pragma unroll
    for (int c = 0; c < C::CB; ++c) acc[b][c] = f32x4_t{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < NS - 1; ++i)
    if (i < stages) st.issue(lds + i * C::STAGE);
  int slot = 0;
  for (int p = 0; p < stages; ++p) {
    // loads land in the order they left: all but those of the stages behind
    const int behind = stages - 1 - p;
    if (behind >= NS - 2) wait_vmcnt<(NS - 2) * L>();
    else if (NS > 3 && behind == 1) wait_vmcnt<L>();
    else wait_vmcnt<0>();
    wait_lgkm0();  // and the slot to be filled has been read
    barrier_lds();
    if (behind >= NS - 1) st.issue(lds + (slot == 0 ? NS - 1 : slot - 1) * C::STAGE);
    const lds_t* A = lds + slot * C::STAGE;
    const lds_t* B = A + C::A;
    stage_products<C::RB, C::CB>(A, B, B + C::CODES + w * 256, 16 * C::CB * w, acc);
    slot = slot + 1 == NS ? 0 : slot + 1;
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
  // At the wave's first stage.
  template <class RowAt, class ColAt>
  __device__ __forceinline__ void init(RowAt row_at, ColAt col_at, const uint8_t* codes, const uint8_t* scales, int K) {
    const int lane = threadIdx.x & 63, w = wave_id();
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const int r = 4 * i + (lane >> 4);
      pa[i] = row_at(r) + (((lane ^ r) & 15) << 4) + w * 256;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = 16 * i + (lane >> 2);
      pb[i] = (const char*)codes + col_at(n) * (K / 2) + (((lane ^ (n >> 2)) & 3) << 4) + w * 64;
    }
    ps = (const char*)scales + col_at(lane) * (K / 32) + w * 4;
  }
  __device__ __forceinline__ void issue(lds_t* slot) {
    lds_t* const b = slot + C::A;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      dma16(pb[i], b + i * 1024);
      pb[i] += 64 * kWaves;
    }
    dma4(ps, b + C::CODES);
    ps += 4 * kWaves;
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      dma16(pa[i], slot + i * 1024);
      pa[i] += 256 * kWaves;
    }
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
  for (int i = 0; i < NS - 1; ++i)
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
    stage_products<C::RB, 4>(A, B, B + C::CODES, 0, acc);
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
