// Loads of matrix rows on their way to MFMA operands without a shared tile:
// each wave loads 16 rows by 128 bytes for itself and turns them in its own
// piece of LDS (the few-token layer and the router's projection, where every
// operand is read once by the wave that needs it).
#pragma once

#include "common.h"
#include "tile.h"

namespace moe {
namespace rowload {

using tile::u32x4_t;

// Loads go through buffer descriptors: a 32-bit offset per lane, and zeros for
// a lane that asks past the end, which is how a K tail becomes exact zeros on
// both operands (every buffer here is below kPast bytes).
constexpr uint32_t kPast = 0xffffff00u;
typedef __amdgpu_buffer_rsrc_t rsrc_t;
__device__ __forceinline__ rsrc_t buffer_of(const void* p, uint64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, (int)(uint32_t)bytes, 0x00020000);
}
// NT: non-temporal, for data that no later load finds in the caches.
template <bool NT = false>
__device__ __forceinline__ u32x4_t load16(rsrc_t r, uint32_t off, bool ok) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, (int)(ok ? off : kPast), 0, NT ? 2 : 0);
}

// An MFMA wants neighbouring lanes to hold neighbouring rows, but a load whose
// neighbouring lanes lie in different rows costs the vector memory unit 64
// cycles, and one whose neighbours are contiguous 25 (measured, 1 KB from the
// caches; 64 cycles for every 1 KB would cap the chip at 9.8 TB/s with the
// activations' loads included).  So a load takes 8 rows of 128 bytes, eight
// lanes a row, and a wave turns the rows around through its own 2 KB of LDS:
// [16 rows][128 bytes], 16-byte chunks XOR-swizzled so that the writes and the
// reads of 16 rows at one chunk are free of bank conflicts.  No barriers: the
// LDS serves one wave's accesses in order.
typedef __attribute__((address_space(3))) char lds_t;
__device__ __forceinline__ int row_chunk(int row, int chunk) { return row * 128 + ((chunk ^ ((row >> 1) & 7)) << 4); }

// 8 half + lane / 8: the row of a 16-row group that this lane loads.
__device__ __forceinline__ int load_row(int half) { return half * 8 + (int)((threadIdx.x & 63) >> 3); }

// 128 bytes at byte `at` of rows at offsets row[0], row[1] (this lane's two
// rows), of which `bytes` exist.
template <bool NT = false>
__device__ __forceinline__ void load_rows(u32x4_t (&v)[2], rsrc_t r, const uint32_t (&row)[2], int at, int bytes) {
  const int off = at + (int)(threadIdx.x & 7) * 16;
#pragma unroll
  for (int h = 0; h < 2; ++h) v[h] = load16<NT>(r, row[h] + off, off < bytes);
}

// Keeps the compiler from moving this lane's LDS accesses past each other: the
// other lanes of the wave read what it writes.  No instruction.
__device__ __forceinline__ void turn_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

__device__ __forceinline__ void put_rows(lds_t* p, const u32x4_t (&v)[2]) {
  const int chunk = threadIdx.x & 7;
  turn_fence();
#pragma unroll
  for (int h = 0; h < 2; ++h)
    *(__attribute__((address_space(3))) u32x4_t*)(p + row_chunk(load_row(h), chunk)) = v[h];
  turn_fence();
}
__device__ __forceinline__ u32x4_t get_chunk(const lds_t* p, int row, int chunk) {
  return *(const __attribute__((address_space(3))) u32x4_t*)(p + row_chunk(row, chunk));
}

// A 16 x 16 float result on its way to be added to other waves': where a lane
// puts rows 4 q .. of its column (16 bytes, as the MFMA leaves them).  A column
// takes 64 bytes, its four pieces permuted so that 16 lanes meet all banks once
// (router forward at 16384 tokens, d = 2048, E = 128: 21.3 us without, 19.8).
__device__ __forceinline__ int part_at(int col, int q) { return col * 16 + ((q ^ (col >> 2)) & 3) * 4; }

}  // namespace rowload
}  // namespace moe
