// The whole layer for a few tokens (T <= kDecodeMaxT), as serving calls it:
//   h = W_gate_up[e] x_t,  a = silu(min(g, L)) clamp(u, -L, L),
//   out_t = sum_j w_tj W_down[e_tj] a,
// with the expert weights in float32, bfloat16, or e4m3 codes with scales
// (128 x 128 float32, or E8M0 per 32 columns) that were laid out once.
//
// What bounds it: every expert that some token selected is read once, 3 I d
// values, and each value meets only that expert's few tokens, so the time is
// the weights' bytes over the memory rate (one token of 8 of 128 experts at d
// = 2048, I = 768: 75 MB).  The layer's 256-row tiles, its sort and its weight
// encoders would cost more than that, so here:
//   * an MFMA's 16 rows are 16 weight rows and its 16 columns are token rows:
//     a weight is loaded once from memory, 128 bytes per row and step ("unit"),
//     and turned into its fragment in the wave's own LDS, whatever the number
//     of tokens;
//   * the K axis of a tile is split over the waves of a work-group and joined
//     in LDS in wave order, so all of a small problem's bytes are in flight
//     at once;
//   * nothing is sorted: each work-group finds its expert's tokens in the ids
//     (at most 256 k of them).
// All sums are float32 in a fixed order, without floating-point atomics.
#include <type_traits>

#include "common.h"
#include "rowload.h"
#include "tile.h"

namespace moe {
namespace {

using namespace rowload;
using tile::u32x4_t;

// ------------------------------------------------------------------- routing
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v == 0.0f) v = 0.0f;  // -0.0 ties with +0.0
  const uint32_t u = __float_as_uint(v);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}

// Largest v over the wave (every lane gets it).  Row rotations by DPP reduce
// each row of 16 lanes, a broadcast of rows joins them in lane 63.
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  auto step = [&](auto ctrl) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl.value, 0xf, 0xf, false);
    v = o > v ? o : v;
  };
  step(std::integral_constant<int, 0x121>{});  // row_ror:1, 2, 4, 8
  step(std::integral_constant<int, 0x122>{});
  step(std::integral_constant<int, 0x124>{});
  step(std::integral_constant<int, 0x128>{});
  step(std::integral_constant<int, 0x142>{});  // row_bcast:15, 31
  step(std::integral_constant<int, 0x143>{});
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// Top k of one token's logits, by one wave: k rounds of a wave-wide maximum;
// among equal logits the lowest index (lane e % 64 holds experts e, e + 64, ...,
// so the first of its registers and then the lowest lane).  The weights are the
// softmax over the selected logits, summed in slot order.  A slot whose logit
// is -inf (a masked expert) is empty: id -1, weight 0.  NaN counts as the
// largest value.  KPL: keys per lane, E <= 64 KPL.
template <int KPL>
struct TopK {
  uint32_t key[KPL];  // 0: taken, or past E
  int id = -1;        // of slot j in lane j % 64
  float ex = 0.0f;    // its unnormalised weight
  float sum = 0.0f;
  template <typename LT>
  __device__ __forceinline__ void load(const LT* __restrict__ row, int E) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      const int e = lane + kWave * i;
      key[i] = 0;
      if (e < E) {
        const float v = to_f32<LT>(row[e]);
        key[i] = v != v ? 0xffffffffu : order_key(v);
      }
    }
  }
  // slots 0 .. k - 1; full(j) is called when slots j - 63 .. j are in the lanes
  // and more follow
  template <class Full>
  __device__ __forceinline__ void select(int k, Full&& full) {
    const int lane = threadIdx.x & 63;
    float top = 0.0f;
    for (int j = 0; j < k; ++j) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < KPL; ++i) m = key[i] > m ? key[i] : m;
      m = wave_max_u32(m);
      int e = 0;
      bool found = false;
#pragma unroll
      for (int i = 0; i < KPL; ++i) {
        const uint64_t eq = __ballot(key[i] == m);
        if (!found && eq) {
          const int l = __builtin_ctzll(eq);
          e = i * kWave + l;
          if (lane == l) key[i] = 0;
          found = true;
        }
      }
      const float l = key_value(m);
      if (j == 0) top = l;
      const bool none = l == -__builtin_huge_valf();
      const float x = none ? 0.0f : expf(l - top);
      sum += x;
      if (lane == (j & 63)) {
        id = none ? -1 : e;
        ex = x;
      }
      if ((j & 63) == 63 && j + 1 < k) full(j);
    }
  }
  __device__ __forceinline__ float weight() const { return id < 0 ? 0.0f : ex / sum; }
};

template <typename LT, int KPL>
__global__ __launch_bounds__(64) void decode_topk_kernel(const LT* __restrict__ logits, int E, int k,
                                                         int32_t* __restrict__ ids, float* __restrict__ w,
                                                         int32_t* __restrict__ mid, float* __restrict__ mw) {
  const int lane = threadIdx.x;
  const int64_t f0 = (int64_t)blockIdx.x * k;
  TopK<KPL> t;
  t.load(logits + (int64_t)blockIdx.x * E, E);
  t.select(k, [&](int j) {
    const int64_t f = f0 + (j & ~63) + lane;
    ids[f] = mid[f] = t.id;
    w[f] = t.ex;
  });
  const int j0 = (k - 1) & ~63;  // the last 64 are still in the lanes
  if (lane < k - j0) {
    const int64_t f = f0 + j0 + lane;
    ids[f] = mid[f] = t.id;
    w[f] = mw[f] = t.weight();
  }
  for (int j = lane; j < j0; j += kWave) {  // each lane reads back its own stores
    const int64_t f = f0 + j;
    const float v = ids[f] < 0 ? 0.0f : w[f] / t.sum;
    w[f] = mw[f] = v;
  }
}

// Given ids: a slot outside [0, E) is empty (mid = -1).  An expert named twice
// by one token keeps its first slot, with the weights added in slot order.
__global__ __launch_bounds__(64) void decode_ids_kernel(const int32_t* __restrict__ ids,
                                                        const float* __restrict__ w, int E, int k,
                                                        int32_t* __restrict__ mid, float* __restrict__ mw) {
  __shared__ int first[kMaxExperts];
  const int lane = threadIdx.x;
  const int64_t f0 = (int64_t)blockIdx.x * k;
  for (int e = lane; e < E; e += kWave) first[e] = k;
  __syncthreads();
  for (int j = lane; j < k; j += kWave) {
    const int e = ids[f0 + j];
    if (e >= 0 && e < E) atomicMin(&first[e], j);
  }
  __syncthreads();
  int twice = 0;
  for (int j = lane; j < k; j += kWave) {
    const int e = ids[f0 + j];
    twice |= e >= 0 && e < E && first[e] != j;
  }
  const bool any_twice = __syncthreads_or(twice);
  for (int j = lane; j < k; j += kWave) {
    const int e = ids[f0 + j];
    const bool mine = e >= 0 && e < E && first[e] == j;
    float v = mine ? w[f0 + j] : 0.0f;
    if (mine && any_twice)
      for (int i = j + 1; i < k; ++i)
        if (ids[f0 + i] == e) v += w[f0 + i];
    mid[f0 + j] = mine ? e : -1;
    mw[f0 + j] = v;
  }
}

// ------------------------------------------------------------ weight formats
// A unit is 128 bytes of each of 16 weight rows.  UK: values of K per unit; BV:
// 16-byte operands of a token's matching activations per lane; NF: MFMAs.
enum WFormat { WF_F32 = 0, WF_BF16 = 1, WF_FP8 = 2, WF_MX = 3 };
template <int F> struct Fmt {  // coded: 128 codes, 4 MFMAs of 32
  typedef bf16_t act;
  typedef bf16x8_t frag;
  static constexpr int UK = 128, BV = 4, NF = 4;
};
template <> struct Fmt<WF_F32> {
  typedef float act;
  typedef float frag;
  static constexpr int UK = 32, BV = 2, NF = 8;
};
template <> struct Fmt<WF_BF16> {
  typedef bf16_t act;
  typedef bf16x8_t frag;
  static constexpr int UK = 64, BV = 2, NF = 2;
};

// A unit's weights in flight, and its scale bytes: `mx` holds, in lane 4 r + i,
// row r's four scale bytes of unit i of a batch of up to four units.
template <int F>
__device__ __forceinline__ uint32_t mx_words(const void* s, int row4, int K, int unit) {
  if constexpr (F == WF_MX) return ((const uint32_t*)s)[(int64_t)row4 * (K >> 7) + min(unit, (K >> 7) - 1)];
  return 0;
}

// The NF / 2 MFMA operands of 16 bytes of a weight row, chunk 4 c + q of its
// unit.  Codes become bfloat16 exactly (e4m3 has four significant bits); an
// E8M0 scale is a power of two and rides on the conversion, which takes it from
// the exponent field alone: byte 0 arrives as the bits of +0 and stands for 2^-127.
// Exact down to bfloat16's smallest numbers (2^-133).  mx: the row's four scale
// bytes of this unit.
template <int F>
__device__ __forceinline__ void chunk_frags(typename Fmt<F>::frag* fr, u32x4_t a, uint32_t mx, int c, int q) {
  if constexpr (F == WF_F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) fr[i] = __uint_as_float(a[i]);
  } else if constexpr (F == WF_BF16) {
    fr[0] = __builtin_bit_cast(bf16x8_t, a);
  } else {
    // its 16 codes lie in block 2 c + q / 2
    const float s = F == WF_MX ? __uint_as_float(((mx >> (16 * c + 8 * (q >> 1))) & 0xffu) << 23) : 1.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      u32x4_t o;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t word = a[2 * h + i];
        o[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(word, s, false));
        o[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(word, s, true));
      }
      fr[h] = __builtin_bit_cast(bf16x8_t, o);
    }
  }
}
// All of a unit's: this lane's row is col, its chunks are q and 4 + q.
template <int F>
__device__ __forceinline__ void to_frags(typename Fmt<F>::frag (&fr)[Fmt<F>::NF], const lds_t* p, uint32_t mx, int q,
                                         int col) {
#pragma unroll
  for (int c = 0; c < 2; ++c) chunk_frags<F>(fr + c * (Fmt<F>::NF / 2), get_chunk(p, col, c * 4 + q), mx, c, q);
}

// The activations of 16 tokens that meet a unit's weights: the same values of
// K, 128 bytes a token, or 256 beside codes.  Tokens 8.. come from r1, and are
// neither loaded nor stored with `eight` (their columns hold anything and are
// dropped).
template <int F> constexpr int kActHalves = F >= WF_FP8 ? 2 : 1;
template <int F>
__device__ __forceinline__ void load_acts(u32x4_t (&v)[kActHalves<F>][2], rsrc_t r, rsrc_t r1,
                                          const uint32_t (&row)[2], const bool (&live)[2], int unit, int bytes,
                                          bool eight) {
#pragma unroll
  for (int h = 0; h < kActHalves<F>; ++h) {
    const int off = (unit * kActHalves<F> + h) * 128 + (int)(threadIdx.x & 7) * 16;
    v[h][0] = load16(r, row[0] + off, live[0] && off < bytes);
    if (!eight) v[h][1] = load16(r1, row[1] + off, live[1] && off < bytes);
  }
}
template <int F>
__device__ __forceinline__ void put_acts(lds_t* p, const u32x4_t (&v)[kActHalves<F>][2], bool eight) {
  const int chunk = threadIdx.x & 7;
  turn_fence();
#pragma unroll
  for (int h = 0; h < kActHalves<F>; ++h) {
    *(__attribute__((address_space(3))) u32x4_t*)(p + h * 2048 + row_chunk(load_row(0), chunk)) = v[h][0];
    if (!eight) *(__attribute__((address_space(3))) u32x4_t*)(p + h * 2048 + row_chunk(load_row(1), chunk)) = v[h][1];
  }
  turn_fence();
}
// The BV / 2 operands that meet weight chunk 4 c + q, and all of a unit's.
template <int F>
__device__ __forceinline__ void chunk_acts(u32x4_t* b, const lds_t* p, int c, int q, int col) {
  if constexpr (F >= WF_FP8) {
#pragma unroll
    for (int v = 0; v < 2; ++v) b[v] = get_chunk(p + c * 2048, col, 2 * q + v);
  } else {
    b[0] = get_chunk(p, col, 4 * c + q);
  }
}
template <int F>
__device__ __forceinline__ void get_acts(u32x4_t (&b)[Fmt<F>::BV], const lds_t* p, int q, int col) {
#pragma unroll
  for (int c = 0; c < 2; ++c) chunk_acts<F>(b + c * (Fmt<F>::BV / 2), p, c, q, col);
}

// s + the products of N operands (a unit's: NF of them), unscaled.
template <int F, int N = Fmt<F>::NF>
__device__ __forceinline__ f32x4_t unit_dot(f32x4_t s, const typename Fmt<F>::frag* fr, const u32x4_t* b) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (F == WF_F32)
      s = __builtin_amdgcn_mfma_f32_16x16x4f32(fr[i], __uint_as_float(b[i >> 2][i & 3]), s, 0, 0, 0);
    else
      s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fr[i], __builtin_bit_cast(bf16x8_t, b[i]), s, 0, 0, 0);
  }
  return s;
}

// acc += the same; sb: the block scale of WF_FP8 (a unit is one 128-wide block).
template <int F>
__device__ __forceinline__ void unit_mma(f32x4_t& acc, const typename Fmt<F>::frag (&fr)[Fmt<F>::NF],
                                         const u32x4_t (&b)[Fmt<F>::BV], float sb) {
  if constexpr (F == WF_FP8) {
    const f32x4_t s = unit_dot<F>(f32x4_t{0, 0, 0, 0}, fr, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = fmaf(sb, s[i], acc[i]);
  } else {
    acc = unit_dot<F>(acc, fr, b);
  }
}

// Blockwise scale of row n and unit `unit` (past K: any) of one matrix [N, K]
// of an expert.  Loaded with the weights it belongs to: a load of its own at
// the time of use waits for memory again.
template <int F>
__device__ __forceinline__ float block_scale_of(const void* s, int n, int K, int unit) {
  if constexpr (F == WF_FP8) return ((const float*)s)[(int64_t)(n >> 7) * (K >> 7) + min(unit, (K >> 7) - 1)];
  return 1.0f;
}

__device__ __forceinline__ float swiglu(float g, float u, float lim) {
  const float gc = clip_gate(g, lim);
  return gc * sigmoidf_(gc) * clip_up(u, lim);
}

// The weighted activation on its way to the down product.  The bf16 MFMA takes
// bf16 operands, and one rounding to bf16 here would be as large an error as the
// output's own; so bf16 calls keep two planes, the value rounded and what that
// left, rounded (2^-17 of the value is lost), and both are multiplied.  Their
// sums are kept apart until join_planes: where an infinite weight meets the
// second plane, 0 inf or a rest of the other sign would make a NaN of the
// formula's infinity.
__device__ __forceinline__ int64_t aw_plane(const DecodeArgs& a) { return (int64_t)a.T * a.k * a.I; }
template <typename AT>
__device__ __forceinline__ void put_aw(const DecodeArgs& a, int64_t at, float v0, float v1) {
  if constexpr (sizeof(AT) == 4) {
    *(f32x2_t*)((float*)a.aw + at) = f32x2_t{v0, v1};
  } else {
    const float h0 = bf2f(f2bf(v0)), h1 = bf2f(f2bf(v1));
    // beside an infinity or NaN the rest would be NaN; h carries it alone
    const float l0 = fabsf(h0) < __builtin_huge_valf() ? v0 - h0 : 0.0f;
    const float l1 = fabsf(h1) < __builtin_huge_valf() ? v1 - h1 : 0.0f;
    *(uint32_t*)((bf16_t*)a.aw + at) = pack_bf16x2(h0, h1);
    *(uint32_t*)((bf16_t*)a.aw + aw_plane(a) + at) = pack_bf16x2(l0, l1);
  }
}

// The sum over both planes.
__device__ __forceinline__ float join_planes(float main, float rest) {
  return fabsf(main) < __builtin_huge_valf() ? main + rest : main;
}

// The same routing inside the gate/up kernel, for a token or a few: every
// work-group does it for itself, which costs it less than another launch and
// the way through memory (T = 1, the case above: 24.5 us with a launch
// for it, 23.3 without).
constexpr int kInlineT = 8, kInlineSlots = 256, kInlineE = 128;
struct InlineRoute {
  int32_t mid[kInlineSlots];
  float mw[kInlineSlots];
};
__host__ __device__ inline bool inline_route_fits(int T, int k, int E) {
  return T <= kInlineT && k <= kWave && T * k <= kInlineSlots && E <= kInlineE;
}

// NW waves (at least a thread per slot).  The first work-group leaves the
// results in memory.
template <int NW>
__device__ __forceinline__ void route_inline(InlineRoute& r, const DecodeArgs& a) {
  static_assert(NW * 64 >= kInlineSlots, "a thread per slot");
  const int lane = threadIdx.x & 63, k = a.k;
  const bool first_group = blockIdx.x == 0 && blockIdx.y == 0;
  if (a.logits) {
    for (int t = tile::wave_id(); t < a.T; t += NW) {
      TopK<2> top;
      if (a.logits_f32) top.load((const float*)a.logits + (int64_t)t * a.E, a.E);
      else top.load((const bf16_t*)a.logits + (int64_t)t * a.E, a.E);
      top.select(k, [](int) {});
      if (lane < k) {
        const int f = t * k + lane;
        const float w = top.weight();
        r.mid[f] = top.id;
        r.mw[f] = w;
        if (first_group) {
          a.ids[f] = a.mid[f] = top.id;
          a.w[f] = a.mw[f] = w;
        }
      }
    }
  } else if ((int)threadIdx.x < a.T * k) {  // as decode_ids_kernel
    const int f = threadIdx.x, j = f % k, f0 = f - j;
    const int e = a.ids[f];
    bool mine = e >= 0 && e < a.E;
    for (int i = 0; i < j; ++i) mine &= a.ids[f0 + i] != e;
    float v = mine ? a.w[f] : 0.0f;
    if (mine)
      for (int i = j + 1; i < k; ++i)
        if (a.ids[f0 + i] == e) v += a.w[f0 + i];
    r.mid[f] = mine ? e : -1;
    r.mw[f] = v;
    if (first_group) {
      a.mid[f] = mine ? e : -1;
      a.mw[f] = v;
    }
  }
  __syncthreads();
}

// ------------------------------------------------------- an expert's tokens
// Work item -> expert.  With at least as many experts as slots, item i is
// slot i, and only the first slot of an expert works on it; otherwise item e
// is expert e.  -1: nothing to do.  Uniform over the work-group.
__device__ __forceinline__ int item_expert(const int32_t* mid, int item, int R, int E) {
  if (R > E) return item;
  const int e = mid[item];
  if (e < 0) return -1;
  int earlier = 0;
  for (int f = threadIdx.x; f < item; f += blockDim.x) earlier |= mid[f] == e;
  return __syncthreads_or(earlier) ? -1 : e;
}

struct Rows {  // an expert's tokens in token order
  int slot[kDecodeMaxT];
  float w[kDecodeMaxT];
  int part[4];
};

// Finds the slots that chose expert e, a thread per token (at least
// kDecodeMaxT threads): count() returns their number, list() then fills rows
// in token order.  What a caller loads in between is in flight meanwhile (a
// barrier does not wait for loads).
struct Finder {
  int slot;
  float w;
  uint64_t has;
  __device__ __forceinline__ int count(Rows& rows, const int32_t* mid, const float* mw, int e, int T, int k) {
    const int t = threadIdx.x, wave = t >> 6;
    slot = -1;
    for (int j0 = 0; j0 < k; j0 += 8) {  // eight loads at a time
      int v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = mid[min(t * k + j0 + i, T * k - 1)];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (t < T && j0 + i < k && v[i] == e) slot = t * k + j0 + i;  // at most one (see decode_ids_kernel)
    }
    w = slot >= 0 ? mw[slot] : 0.0f;
    has = __ballot(slot >= 0);
    if (wave < 4 && (t & 63) == 0) rows.part[wave] = __popcll(has);
    __syncthreads();
    return rows.part[0] + rows.part[1] + rows.part[2] + rows.part[3];
  }
  __device__ __forceinline__ void list(Rows& rows) const {
    const int t = threadIdx.x, wave = t >> 6;
    int r = __popcll(has & ((1ull << (t & 63)) - 1));
#pragma unroll
    for (int i = 0; i < 3; ++i) r += i < wave ? rows.part[i] : 0;
    if (slot >= 0) {
      rows.slot[r] = slot;
      rows.w[r] = w;
    }
    __syncthreads();
  }
};

// ------------------------------------------------------------ gate/up product
// One work-group: TB times 16 gate rows and the same up rows of one expert, for
// all of its tokens, NBMAX blocks of 16 a pass; the NW waves take batches of UN units of K in turn.
template <int F, int TB, int UN>
struct GuWeights {  // UN units of the tile's gate and up rows, in flight
  u32x4_t g[TB][UN][2], u[TB][UN][2];
  uint32_t mg[TB], mu[TB];
  float sg[UN], su[UN];  // blockwise scales (a tile lies in one block of rows)
};

template <int TB>
struct GuTile {  // where a lane finds them
  rsrc_t w;
  const void* sc;
  uint32_t g[TB][2], u[TB][2];  // offsets of this lane's gate and up rows
  int row4;                     // row whose scale bytes it loads, and 16 on
  int n0;
};

template <int F, bool NT, int TB, int UN>
__device__ __forceinline__ void load_gu(GuWeights<F, TB, UN>& w, const GuTile<TB>& t, int I, int K, int base) {
  const int bytes = F >= WF_FP8 ? K : K * (int)sizeof(typename Fmt<F>::act);
#pragma unroll
  for (int i = 0; i < UN; ++i) {
#pragma unroll
    for (int b = 0; b < TB; ++b) {
      load_rows<NT>(w.g[b][i], t.w, t.g[b], (base + i) * 128, bytes);
      load_rows<NT>(w.u[b][i], t.w, t.u[b], (base + i) * 128, bytes);
    }
    w.sg[i] = block_scale_of<F>(t.sc, t.n0, K, base + i);
    w.su[i] = block_scale_of<F>(t.sc, I + t.n0, K, base + i);
  }
#pragma unroll
  for (int b = 0; b < TB; ++b) {
    w.mg[b] = mx_words<F>(t.sc, t.row4 + 16 * b, K, base + (int)(threadIdx.x & 3));
    w.mu[b] = mx_words<F>(t.sc, I + t.row4 + 16 * b, K, base + (int)(threadIdx.x & 3));
  }
}

template <int F, int NW, int TB, int NBMAX>
constexpr size_t gu_smem() {  // per wave: gate, up, activations; then the waves' parts
  const size_t work = (size_t)NW * (4096 + 2048 * kActHalves<F>), parts = (size_t)NW * NBMAX * TB * 2048;
  return work > parts ? work : parts;
}

// The tokens r0 .. r0 + 16 NB of the expert.  w holds the first units.
template <int F, bool NT, int NW, int TB, int UN, int NB>
__device__ __forceinline__ void gateup_rows(const DecodeArgs& a, const Rows& rows, int r0, int n, bool again,
                                            GuWeights<F, TB, UN>& w, const GuTile<TB>& t, char* smem) {
  typedef typename Fmt<F>::act AT;
  const int lane = threadIdx.x & 63, wave = tile::wave_id(), q = lane >> 4, col = lane & 15;
  const int K = a.d;
  const int units = (K + Fmt<F>::UK - 1) / Fmt<F>::UK;
  const int bytes = K * (int)sizeof(AT);
  const rsrc_t xb = buffer_of(a.x, (uint64_t)a.T * bytes);
  const bool eight = NB == 1 && n - r0 <= 8;
  lds_t* lw = (lds_t*)smem + wave * (4096 + 2048 * kActHalves<F>);
  uint32_t xr[NB][2];
  bool live[NB][2];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = r0 + b * 16 + load_row(h);
      live[b][h] = r < n;
      xr[b][h] = (uint32_t)(rows.slot[live[b][h] ? r : n - 1] / a.k) * bytes;
    }
  f32x4_t ag[NB][TB], au[NB][TB];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int m = 0; m < TB; ++m) ag[b][m] = au[b][m] = f32x4_t{0, 0, 0, 0};
  constexpr int UB = NB == 1 ? UN : 1;  // units whose activations are in flight together
  for (int base = wave * UN; base < units; base += NW * UN) {
    if (base != wave * UN || again) load_gu<F, NT>(w, t, a.I, K, base);
#pragma unroll
    for (int i0 = 0; i0 < UN; i0 += UB) {
      u32x4_t xv[UB][NB][kActHalves<F>][2];
#pragma unroll
      for (int i = 0; i < UB; ++i)
#pragma unroll
        for (int b = 0; b < NB; ++b) load_acts<F>(xv[i][b], xb, xb, xr[b], live[b], base + i0 + i, bytes, eight);
      __builtin_amdgcn_sched_barrier(0);  // all loads leave before the first product waits
#pragma unroll
      for (int i = 0; i < UB; ++i) {
        u32x4_t xf[NB][Fmt<F>::BV];
#pragma unroll
        for (int m = 0; m < TB; ++m) {
          put_rows(lw, w.g[m][i0 + i]);
          put_rows(lw + 2048, w.u[m][i0 + i]);
          uint32_t mg = 0, mu = 0;
          if constexpr (F == WF_MX) {
            mg = (uint32_t)__shfl((int)w.mg[m], col * 4 + i0 + i, kWave);
            mu = (uint32_t)__shfl((int)w.mu[m], col * 4 + i0 + i, kWave);
          }
          typename Fmt<F>::frag fr[Fmt<F>::NF];
          to_frags<F>(fr, lw, mg, q, col);
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            if (m == 0) {
              put_acts<F>(lw + 4096, xv[i][b], eight);
              get_acts<F>(xf[b], lw + 4096, q, col);
            }
            unit_mma<F>(ag[b][m], fr, xf[b], w.sg[i0 + i]);
          }
          to_frags<F>(fr, lw + 2048, mu, q, col);
#pragma unroll
          for (int b = 0; b < NB; ++b) unit_mma<F>(au[b][m], fr, xf[b], w.su[i0 + i]);
        }
      }
    }
  }
  // parts [wave][b][tile of 16 rows][gate, up][col][16 rows], over the waves'
  // work space
  float* red = (float*)smem;
  __syncthreads();
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int m = 0; m < TB; ++m) {
      float* p = red + ((wave * NB + b) * TB + m) * 512 + part_at(col, q);
      *(f32x4_t*)p = ag[b][m];
      *(f32x4_t*)(p + 256) = au[b][m];
    }
  __syncthreads();
  for (int o = threadIdx.x; o < NB * TB * 128; o += NW * 64) {
    // neighbouring threads: neighbouring pairs of rows of all TB tiles, then tokens
    const int m = (o & 7) * 2, tb = (o >> 3) % TB, c = o / (8 * TB) & 15, b = o / (128 * TB);
    const int r = r0 + b * 16 + c, row = t.n0 + tb * 16 + m;
    if (r < n && row < a.I) {  // I is a multiple of 8: both rows are in or out
      f32x2_t g = {0, 0}, u = {0, 0};
#pragma unroll
      for (int v = 0; v < NW; ++v) {
        const float* p = red + ((v * NB + b) * TB + tb) * 512 + part_at(c, m >> 2) + (m & 3);
        const f32x2_t pg = *(const f32x2_t*)p, pu = *(const f32x2_t*)(p + 256);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          g[i] += pg[i];
          u[i] += pu[i];
        }
      }
      const float w = rows.w[r];
      put_aw<AT>(a, (int64_t)rows.slot[r] * a.I + row, w * swiglu(g[0], u[0], a.lim), w * swiglu(g[1], u[1], a.lim));
    }
  }
  __syncthreads();
}

template <int F, bool NT, int NBMAX, int NW, int TB, int UN, bool INLINE = false>
__global__ __launch_bounds__(NW * 64) void decode_gateup_kernel(DecodeArgs a) {
  static_assert(UN <= 4, "mx_words holds four units");
  static_assert(NW * 64 >= kDecodeMaxT, "Finder takes a thread per token");
  __shared__ Rows rows;
  __shared__ __align__(16) char smem[gu_smem<F, NW, TB, NBMAX>()];
  const int32_t* mid = a.mid;
  const float* mw = a.mw;
  if constexpr (INLINE) {
    __shared__ InlineRoute route;
    route_inline<NW>(route, a);
    mid = route.mid;
    mw = route.mw;
  }
  const int e = __builtin_amdgcn_readfirstlane(item_expert(mid, blockIdx.y, a.T * a.k, a.E));
  if (e < 0) return;
  const int lane = threadIdx.x & 63;
  Finder find;
  const int n = find.count(rows, mid, mw, e, a.T, a.k);
  if (n == 0) return;
  GuTile<TB> t;
  t.n0 = blockIdx.x * 16 * TB;
  const int rowb = a.d * (F >= WF_FP8 ? 1 : (int)sizeof(typename Fmt<F>::act));
  const uint64_t wbytes = (uint64_t)2 * a.I * rowb;
  t.w = buffer_of((const char*)a.w_gate_up + e * wbytes, wbytes);
#pragma unroll
  for (int b = 0; b < TB; ++b)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = min(t.n0 + b * 16 + load_row(h), a.I - 1);  // rows past I repeat the last and are dropped
      t.g[b][h] = (uint32_t)row * rowb;
      t.u[b][h] = (uint32_t)(a.I + row) * rowb;
    }
  t.row4 = t.n0 + (lane >> 2);  // read for WF_MX, where I is a multiple of 128
  const char* sc = (const char*)a.s_gate_up;
  if (F == WF_FP8) sc += (int64_t)e * (2 * a.I / 128) * (a.d / 128) * 4;
  if (F == WF_MX) sc += (int64_t)e * 2 * a.I * (a.d / 32);
  t.sc = sc;
  GuWeights<F, TB, UN> w;
  load_gu<F, NT>(w, t, a.I, a.d, tile::wave_id() * UN);
  find.list(rows);
  if constexpr (NBMAX == 1) {
    gateup_rows<F, NT, NW, TB, UN, 1>(a, rows, 0, n, false, w, t, smem);
  } else {
    const int first = blockIdx.z * 16 * NBMAX;
    for (int r0 = first; r0 < n; r0 += gridDim.z * 16 * NBMAX) {
      if (n - r0 <= 16) gateup_rows<F, NT, NW, TB, UN, 1>(a, rows, r0, n, r0 != first, w, t, smem);
      else gateup_rows<F, NT, NW, TB, UN, NBMAX>(a, rows, r0, n, r0 != first, w, t, smem);
    }
  }
}

// ---------------------------------------------- down product, up to 32 slots
// One work-group: 8 rows of d for all tokens; the waves take batches of the
// (expert, unit of I) pairs, and the combine is the sum itself (aw carries the
// weights).  The experts are found in the lanes of each wave, slot f in lane f,
// without LDS or barriers.  An MFMA's rows and columns 0 .. 7 are the tile's
// rows and the tokens at the first half of a unit, 8 .. 15 the same rows and
// tokens at the second half; the two diagonal blocks of its result are the
// sums, the others are dropped.  (T = 1, the case above: 23.1 us with tiles of
// 16 rows, 22.4 with these.)  Sixteen waves with six units each in flight hold
// all of that case's pairs, 8 experts by 12 units, at once; codes have half the
// units and, beside them, twice the registers of activations: four.
constexpr int kDownWaves = 16;

template <int F>
__global__ __launch_bounds__(kDownWaves * 64) void decode_down_small_kernel(DecodeArgs a) {
  typedef typename Fmt<F>::act AT;
  constexpr int WORK = 2048 + 2048 * kActHalves<F>, UN = F >= WF_FP8 ? 4 : 6;
  __shared__ __align__(16) char work[kDownWaves * WORK];  // then the parts [2 waves][8 tokens][8 rows]
  const int lane = threadIdx.x & 63, wave = tile::wave_id(), q = lane >> 4, col = lane & 15;
  const int r8 = col & 7, half = col >> 3;
  const int R = a.T * a.k;
  const int mine = lane < R ? a.mid[lane] : -1;
  bool first = mine >= 0;
  for (int f = 0; f < R; ++f) first &= f >= lane || __builtin_amdgcn_readlane(mine, f) != mine;
  const uint64_t firsts = __ballot(first);
  const int nact = __popcll(firsts);
  const int K = a.I, n0 = blockIdx.x * 8;
  const int units = (K + Fmt<F>::UK - 1) / Fmt<F>::UK;
  const int abytes = F >= WF_FP8 ? K : K * (int)sizeof(AT), bbytes = K * (int)sizeof(AT);
  const uint64_t wbytes = (uint64_t)a.d * abytes;
  const uint32_t wrow = (uint32_t)min(n0 + load_row(0), a.d - 1) * abytes;
  constexpr int P = F == WF_F32 ? 1 : 2;  // planes of aw
  rsrc_t xb[P];
#pragma unroll
  for (int p = 0; p < P; ++p) xb[p] = buffer_of((const AT*)a.aw + p * aw_plane(a), (uint64_t)R * bbytes);
  lds_t* lw = (lds_t*)work + wave * WORK;
  const int total = nact * units;
  const uint64_t slots = a.k == 64 ? ~0ull : (1ull << a.k) - 1;  // a token's slots
  f32x4_t acc[P];  // a plane's sums each
#pragma unroll
  for (int p = 0; p < P; ++p) acc[p] = f32x4_t{0, 0, 0, 0};
  for (int base = wave * UN; base < total; base += kDownWaves * UN) {
    u32x4_t wv[UN], xv[UN][P][kActHalves<F>];
    uint32_t mx[UN];
    float sb[UN];
    bool on_expert[UN];
    int idx = base / units, unit = base - idx * units;
    uint64_t rest = firsts;
    for (int i = 0; i < idx; ++i) rest &= rest - 1;
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      const bool on = base + i < total;  // uniform in the wave
      const int e = on ? __builtin_amdgcn_readlane(mine, __builtin_ctzll(rest)) : 0;
      const uint64_t has = __ballot(mine == e);
      const int off = unit * 128 + (lane & 7) * 16;
      wv[i] = load16(buffer_of((const char*)a.w_down + e * wbytes, wbytes), wrow + off, on && off < abytes);
      const int t = load_row(0);
      const uint64_t ts = t < a.T ? (has >> (t * a.k)) & slots : 0;
      const uint32_t xrow = (uint32_t)(t * a.k + (ts ? __builtin_ctzll(ts) : 0)) * bbytes;
#pragma unroll
      for (int h = 0; h < kActHalves<F>; ++h) {
        const int o = (unit * kActHalves<F> + h) * 128 + (lane & 7) * 16;
#pragma unroll
        for (int p = 0; p < P; ++p) xv[i][p][h] = load16(xb[p], xrow + o, on && ts && o < bbytes);
      }
      on_expert[i] = on && r8 < a.T && ((has >> (r8 * a.k)) & slots);
      const char* sc = (const char*)a.s_down;
      if (F == WF_FP8) sc += (int64_t)e * (a.d / 128) * (K / 128) * 4;
      if (F == WF_MX) sc += (int64_t)e * a.d * (K / 32);
      mx[i] = F == WF_MX ? ((const uint32_t*)sc)[(int64_t)(n0 + r8) * (K >> 7) + unit] : 0;
      sb[i] = block_scale_of<F>(sc, n0, K, unit);
      if (on && ++unit == units) {
        unit = 0;
        rest &= rest - 1;
      }
    }
    __builtin_amdgcn_sched_barrier(0);  // all loads leave before the first product waits
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      const int chunk = lane & 7;
      turn_fence();
      *(__attribute__((address_space(3))) u32x4_t*)(lw + row_chunk(load_row(0), chunk)) = wv[i];
      turn_fence();
      typename Fmt<F>::frag fr[Fmt<F>::NF / 2];
      chunk_frags<F>(fr, get_chunk(lw, r8, 4 * half + q), mx[i], half, q);
#pragma unroll
      for (int p = 0; p < P; ++p) {
        turn_fence();
#pragma unroll
        for (int h = 0; h < kActHalves<F>; ++h)
          *(__attribute__((address_space(3))) u32x4_t*)(lw + 2048 + h * 2048 + row_chunk(load_row(0), chunk)) =
              xv[i][p][h];
        turn_fence();
        u32x4_t xf[Fmt<F>::BV / 2];
        chunk_acts<F>(xf, lw + 2048, half, q, r8);
        const f32x4_t s = unit_dot<F, Fmt<F>::NF / 2>(f32x4_t{0, 0, 0, 0}, fr, xf);
#pragma unroll
        for (int m = 0; m < 4; ++m) acc[p][m] = on_expert[i] ? fmaf(sb[i], s[m], acc[p][m]) : acc[p][m];
      }
    }
  }
  if constexpr (P == 2) {
#pragma unroll
    for (int m = 0; m < 4; ++m) acc[0][m] = join_planes(acc[0][m], acc[1][m]);
  }
  float* red = (float*)work;
  __syncthreads();
  if ((q >> 1) == half) *(f32x4_t*)(red + ((wave * 2 + half) * 8 + r8) * 8 + (q & 1) * 4) = acc[0];
  __syncthreads();
  if (threadIdx.x < 64) {
    const int t = threadIdx.x >> 3, m = threadIdx.x & 7;
    if (t < a.T) {  // d is a multiple of 8
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < 2 * kDownWaves; ++w) v += red[(w * 8 + t) * 8 + m];
      ((AT*)a.out)[(int64_t)t * a.d + n0 + m] = from_f32<AT>(v);
    }
  }
}

// --------------------------------------------- down product, more tokens
// One wave: 16 TB rows of d of one expert for its tokens, all of I, or with KS
// its fourth of I, joined in LDS; the products go to y [T k, d] in float32,
// which decode_combine_kernel sums in slot order.
constexpr int kDownRowWaves = 4;

template <int TB>
struct DownTile {
  rsrc_t w;
  const void* sc;
  uint32_t row[TB][2];  // offsets of this lane's rows
  int row4, n0;
};

template <int F, bool NT, int TB, int UN, bool KS, int NB, bool EIGHT = false>
__device__ __forceinline__ void down_rows(const DecodeArgs& a, const Rows& rows, int r0, int n, const DownTile<TB>& t,
                                          lds_t* lw, float* red) {
  typedef typename Fmt<F>::act AT;
  const int lane = threadIdx.x & 63, q = lane >> 4, col = lane & 15;
  const int K = a.I;
  const int units = (K + Fmt<F>::UK - 1) / Fmt<F>::UK;
  const int abytes = F >= WF_FP8 ? K : K * (int)sizeof(AT), bbytes = K * (int)sizeof(AT);
  const rsrc_t xb = buffer_of(a.aw, (uint64_t)a.T * a.k * bbytes);
  const rsrc_t xl = F == WF_F32 ? xb : buffer_of((const AT*)a.aw + aw_plane(a), (uint64_t)a.T * a.k * bbytes);
  // P passes over a unit's weights, one for each plane of aw; with EIGHT (at most
  // 8 rows) columns 8 .. are the same rows' second plane instead
  static_assert(!EIGHT || (F != WF_F32 && NB == 1), "");
  constexpr int P = F == WF_F32 || EIGHT ? 1 : 2;
  uint32_t xr[NB][2];
  bool live[NB][2];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = r0 + b * 16 + load_row(EIGHT ? 0 : h);
      live[b][h] = r < n;
      xr[b][h] = (uint32_t)rows.slot[live[b][h] ? r : n - 1] * bbytes;
    }
  f32x4_t acc[P][NB][TB];  // a plane's sums each
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int m = 0; m < TB; ++m) acc[p][b][m] = f32x4_t{0, 0, 0, 0};
  constexpr int UB = NB == 1 ? UN : 1;
  const int wave = tile::wave_id();
  for (int base = KS ? wave * UN : 0; base < units; base += (KS ? kDownRowWaves : 1) * UN) {
    u32x4_t wv[TB][UN][2];
    float sb[UN];
#pragma unroll
    for (int i = 0; i < UN; ++i) {
#pragma unroll
      for (int m = 0; m < TB; ++m) load_rows<NT>(wv[m][i], t.w, t.row[m], (base + i) * 128, abytes);
      sb[i] = block_scale_of<F>(t.sc, t.n0, K, base + i);
    }
    uint32_t mx[TB];
#pragma unroll
    for (int m = 0; m < TB; ++m) mx[m] = mx_words<F>(t.sc, t.row4 + 16 * m, K, base + (lane & 3));
#pragma unroll
    for (int i0 = 0; i0 < UN; i0 += UB) {
      u32x4_t xv[UB][NB][P][kActHalves<F>][2];
#pragma unroll
      for (int i = 0; i < UB; ++i)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int p = 0; p < P; ++p)
            load_acts<F>(xv[i][b][p], p ? xl : xb, p || EIGHT ? xl : xb, xr[b], live[b], base + i0 + i, bbytes, false);
      __builtin_amdgcn_sched_barrier(0);  // all loads leave before the first product waits
#pragma unroll
      for (int i = 0; i < UB; ++i) {
        u32x4_t xf[NB][P][Fmt<F>::BV];
#pragma unroll
        for (int m = 0; m < TB; ++m) {
          typename Fmt<F>::frag fr[Fmt<F>::NF];
          put_rows(lw, wv[m][i0 + i]);
          uint32_t code = 0;
          if constexpr (F == WF_MX) code = (uint32_t)__shfl((int)mx[m], col * 4 + i0 + i, kWave);
          to_frags<F>(fr, lw, code, q, col);
#pragma unroll
          for (int b = 0; b < NB; ++b) {
#pragma unroll
            for (int p = 0; p < P; ++p) {
              if (m == 0) {
                put_acts<F>(lw + 2048, xv[i][b][p], false);
                get_acts<F>(xf[b][p], lw + 2048, q, col);
              }
              unit_mma<F>(acc[p][b][m], fr, xf[b][p], sb[i0 + i]);
            }
          }
        }
      }
    }
  }
  if constexpr (EIGHT) {  // columns 8 .. belong to the columns eight before
#pragma unroll
    for (int m = 0; m < TB; ++m)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        acc[0][0][m][v] = join_planes(acc[0][0][m][v], __shfl_xor(acc[0][0][m][v], 8, kWave));
  } else if constexpr (P == 2) {
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int m = 0; m < TB; ++m)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[0][b][m][v] = join_planes(acc[0][b][m][v], acc[1][b][m][v]);
  }
  if constexpr (KS) {  // parts [wave][b][16 tokens][16 rows], over the waves' work space
    static_assert(TB == 1, "a part is 16 rows");
    __syncthreads();
#pragma unroll
    for (int b = 0; b < NB; ++b) *(f32x4_t*)(red + (wave * NB + b) * 256 + part_at(col, q)) = acc[0][b][0];
    __syncthreads();
    for (int o = threadIdx.x; o < NB * 64; o += kDownRowWaves * 64) {
      const int r = r0 + (o >> 2), row = t.n0 + (o & 3) * 4;
      const float* p = red + (o >> 6) * 256 + part_at((o >> 2) & 15, o & 3);
      f32x4_t s = *(const f32x4_t*)p;
#pragma unroll
      for (int w = 1; w < kDownRowWaves; ++w) {
        const f32x4_t v = *(const f32x4_t*)(p + w * NB * 256);
#pragma unroll
        for (int m = 0; m < 4; ++m) s[m] += v[m];
      }
      if (r < n && row < a.d) *(f32x4_t*)(a.y + (int64_t)rows.slot[r] * a.d + row) = s;
    }
    __syncthreads();
    return;
  }
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int r = r0 + b * 16 + col;
#pragma unroll
    for (int m = 0; m < TB; ++m) {
      const int row = t.n0 + 16 * m + q * 4;
      if (r < n && row < a.d)  // d is a multiple of 8: four rows are in or out together
        *(f32x4_t*)(a.y + (int64_t)rows.slot[r] * a.d + row) = acc[0][b][m];
    }
  }
}

// The wide blockwise form is held to three waves a SIMD: it would take 174
// registers and leave two (16 tokens, e4m3 above: 46 us with two, 42 with three).
template <int F, bool NT, int TB, int UN, bool KS>
__global__ __launch_bounds__(kDownRowWaves * 64, F == WF_FP8 && TB == 2 ? 3 : 1) void decode_down_rows_kernel(DecodeArgs a) {
  static_assert(kDownRowWaves * 64 >= kDecodeMaxT, "Finder takes a thread per token");
  __shared__ Rows rows;
  __shared__ __align__(16) char work[kDownRowWaves * (2048 + 2048 * kActHalves<F>)];
  const int e = __builtin_amdgcn_readfirstlane(item_expert(a.mid, blockIdx.y, a.T * a.k, a.E));
  if (e < 0) return;
  Finder find;
  const int n = find.count(rows, a.mid, a.mw, e, a.T, a.k);
  find.list(rows);
  DownTile<TB> t;
  const int lane = threadIdx.x & 63, wave = tile::wave_id();
  t.n0 = (KS ? (int)blockIdx.x : (int)blockIdx.x * kDownRowWaves + wave) * 16 * TB;
  if (n == 0 || t.n0 >= a.d) return;  // the whole work-group with KS; else no barrier follows
  const int rowb = a.I * (F >= WF_FP8 ? 1 : (int)sizeof(typename Fmt<F>::act));
  const uint64_t wbytes = (uint64_t)a.d * rowb;
  t.w = buffer_of((const char*)a.w_down + e * wbytes, wbytes);
#pragma unroll
  for (int m = 0; m < TB; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) t.row[m][h] = (uint32_t)min(t.n0 + 16 * m + load_row(h), a.d - 1) * rowb;
  t.row4 = t.n0 + (lane >> 2);  // read for WF_MX, where d is a multiple of 128
  const char* sc = (const char*)a.s_down;
  if (F == WF_FP8) sc += (int64_t)e * (a.d / 128) * (a.I / 128) * 4;
  if (F == WF_MX) sc += (int64_t)e * a.d * (a.I / 32);
  t.sc = sc;
  lds_t* lw = (lds_t*)work + wave * (2048 + 2048 * kActHalves<F>);
  for (int r0 = blockIdx.z * 32; r0 < n; r0 += gridDim.z * 32) {
    if (F != WF_F32 && n - r0 <= 8)
      down_rows<F, NT, TB, UN, KS, 1, F != WF_F32>(a, rows, r0, n, t, lw, (float*)work);
    else if (n - r0 <= 16) down_rows<F, NT, TB, UN, KS, 1>(a, rows, r0, n, t, lw, (float*)work);
    else down_rows<F, NT, TB, UN, KS, 2>(a, rows, r0, n, t, lw, (float*)work);
  }
}

// out[t] = sum of the token's live slots of y, in slot order; one rounding.
template <typename AT>
__global__ __launch_bounds__(256) void decode_combine_kernel(DecodeArgs a) {
  const int c = blockIdx.x * 256 + threadIdx.x, t = blockIdx.y;
  if (c * 4 >= a.d) return;
  f32x4_t acc = {0, 0, 0, 0};
  const int64_t f0 = (int64_t)t * a.k;
  for (int j0 = 0; j0 < a.k; j0 += 8) {  // eight loads at a time
    bool live[8];
    f32x4_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) live[i] = j0 + i < a.k && a.mid[f0 + min(j0 + i, a.k - 1)] >= 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = f32x4_t{0, 0, 0, 0};
      if (live[i]) v[i] = *(const f32x4_t*)(a.y + (f0 + j0 + i) * a.d + c * 4);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int m = 0; m < 4; ++m) acc[m] += v[i][m];
  }
  AT* o = (AT*)a.out + (int64_t)t * a.d + c * 4;
  if constexpr (sizeof(AT) == 4) *(f32x4_t*)o = acc;
  else *(uint2*)o = uint2{pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3])};
}

int work_items(const DecodeArgs& a) { return a.T * a.k > a.E ? a.E : a.T * a.k; }
int64_t gu_groups(const DecodeArgs& a) { return cdiv(a.I, 16) * work_items(a); }

// Whether work-groups of 32 rows (a wave's, in the down product) leave four for
// each CU.  Twice the rows halve what is read of the activations; fewer groups
// leave CUs idle at the end.  Above, us with 16 and 32 rows at 256 tokens by the
// experts (with one plane of aw to write; two add 2 to 6): gate/up bf16 128 151
// and 137, 64 (1536 groups) 94 and 86, 32 (768) 51 and 55; mxfp8, 200 tokens,
// 128 experts 97 and 82, 8 (192) 20 and 25.
bool wide_gateup(const DecodeArgs& a) { return cdiv(a.I, 32) * work_items(a) >= 1024; }

// For the down product also two tokens an expert, below which its activations
// are little beside its weights (us with 16 and 32 rows, mxfp8, 200 tokens 69
// and 55; e4m3, 16 of 8 of 64 experts, d = 4096, I = 1024 49 and 43; bf16, 256
// tokens 107 and 95, 64 67 both ways; 32 experts, 512 groups: 27 and 30).
bool wide_down(const DecodeArgs& a) {
  return cdiv(a.d, 32 * kDownRowWaves) * work_items(a) >= 1024 && a.T * a.k >= 2 * work_items(a);
}

// Work-groups that an expert's tokens are split over, 32 at a time, where the
// experts and rows alone leave CUs free: each then reads the weights again,
// from the caches, instead of passing over them for one block after another
// (256 tokens of 2 of 8 experts, d = 2048, I = 768, bf16: gate/up 31 us without
// and 23, down 19 and 13; 219 tokens, 2 experts, d = 192, I = 784: 15 and 7, 51
// and 10.  Up to 512 or 2048 work-groups instead of 1024: the first case's
// gate/up 35 and 25).
unsigned token_split(const DecodeArgs& a, int64_t groups) {
  const int64_t most = cdiv(a.T, 32), want = 1024 / groups;
  return (unsigned)(want < 1 ? 1 : want < most ? want : most);
}

// Whether the weights that the tokens may select exceed the last-level cache.
// Nothing of them is left there for the next call then, and non-temporal loads
// keep them from displacing what this call reads again (64 tokens of 8 of 128
// experts above: 221 us without, 204 with).  Below that size they cost the
// reuse, also where other layers' weights were used since the last call (256
// tokens of 2 of 8 experts of the same size, 75 MB read twice: 44 us without and
// 56 with them on one layer's weights, 48 and 57 on those of 16 layers in turn;
// one token of all 8 experts 22 and 23, and 26 both ways).
template <int F>
bool past_cache(const DecodeArgs& a) {
  constexpr int64_t kLastLevelCache = int64_t(256) << 20;
  const int64_t value = F >= WF_FP8 ? 1 : sizeof(typename Fmt<F>::act);
  return work_items(a) * int64_t(3) * a.I * a.d * value > kLastLevelCache;
}

template <int F, bool NT>
hipError_t run_gateup(const LaunchCtx& c, const DecodeArgs& a) {
  const dim3 grid((unsigned)cdiv(a.I, 16), (unsigned)work_items(a));
  constexpr int UN = F >= WF_FP8 ? 2 : 4;
  if (a.T > 16 && wide_gateup(a)) {
    // units of K at a time: coded weights one (two leave room for fewer waves: 84
    // us and 111 at 200 tokens), the others two (137 both ways at 256, at 64 125
    // and with one 131)
    constexpr int UNW = F >= WF_FP8 ? 1 : 2;
    const dim3 wide((unsigned)cdiv(a.I, 32), grid.y);
    MOE_LAUNCH(c, "decode_gateup", (decode_gateup_kernel<F, NT, 2, 4, 2, UNW>), wide, dim3(4 * 64), 0, a);
  } else if (a.T > 16) {
    const dim3 split(grid.x, grid.y, token_split(a, gu_groups(a)));
    // a work-group per CU or fewer: eight waves (57 tokens of both of 2 experts,
    // d = 3792, I = 648, float32, 164 groups: 31 us with four and 26; 175 tokens,
    // 5 experts, d = 960, I = 272, 510 groups: 8.1 and 9.4)
    if (gu_groups(a) * split.z <= 256)
      MOE_LAUNCH(c, "decode_gateup", (decode_gateup_kernel<F, NT, 2, 8, 1, 2>), split, dim3(8 * 64), 0, a);
    else
      MOE_LAUNCH(c, "decode_gateup", (decode_gateup_kernel<F, NT, 2, 4, 1, 2>), split, dim3(4 * 64), 0, a);
  }
  // As many work-groups as fit beside each other, two per CU: eight waves each,
  // so that all bytes are in flight at once (T = 1 above, 384 work-groups: 24.7
  // us with eight, 26.3 with four).  More: four, of which more fit (T = 2, 768:
  // 38.7 us with eight, 36.1 with four; 16 tokens of 8 of 64 experts, d = 4096,
  // I = 1024, e4m3: 150 and 139).
  else if (gu_groups(a) <= 512 && a.route_inline)
    MOE_LAUNCH(c, "decode_gateup", (decode_gateup_kernel<F, NT, 1, 8, 1, UN, true>), grid, dim3(8 * 64), 0, a);
  else if (gu_groups(a) <= 512)
    MOE_LAUNCH(c, "decode_gateup", (decode_gateup_kernel<F, NT, 1, 8, 1, UN>), grid, dim3(8 * 64), 0, a);
  else if (a.route_inline)
    MOE_LAUNCH(c, "decode_gateup", (decode_gateup_kernel<F, NT, 1, 4, 1, UN, true>), grid, dim3(4 * 64), 0, a);
  else
    MOE_LAUNCH(c, "decode_gateup", (decode_gateup_kernel<F, NT, 1, 4, 1, UN>), grid, dim3(4 * 64), 0, a);
  return hipSuccess;
}

template <int F, bool NT>
hipError_t run_down(const LaunchCtx& c, const DecodeArgs& a) {
  if (decode_one_down(a.T, a.k)) {
    MOE_LAUNCH(c, "decode_down", decode_down_small_kernel<F>, dim3((unsigned)(a.d / 8)), dim3(kDownWaves * 64), 0, a);
    return hipSuccess;
  }
  constexpr int UN = F >= WF_FP8 ? 2 : 4;
  const unsigned items = (unsigned)work_items(a);
  if (wide_down(a)) {
    const dim3 grid((unsigned)cdiv(a.d, 32 * kDownRowWaves), items);
    MOE_LAUNCH(c, "decode_down", (decode_down_rows_kernel<F, NT, 2, UN / 2, false>), grid, dim3(kDownRowWaves * 64), 0, a);
  } else {
    const unsigned tiles = (unsigned)cdiv(a.d, 16 * kDownRowWaves);
    const dim3 grid(tiles, items, token_split(a, (int64_t)tiles * items));
    // a work-group per CU or fewer: each of its waves takes a fourth of I instead
    // of 16 rows (20 tokens, 4 experts, d = 224, I = 952, float32: 11.2 us
    // without and 6.0; 219 tokens, 2 experts, d = 192, I = 784: 10.3 and 5.1; up
    // to 1024, 256 tokens of 2 of 8 experts, d = 2048, I = 768: 12.5 and 15.1)
    if ((int64_t)tiles * items * grid.z <= 256) {
      const dim3 split((unsigned)cdiv(a.d, 16), items, grid.z);
      MOE_LAUNCH(c, "decode_down", (decode_down_rows_kernel<F, NT, 1, UN, true>), split, dim3(kDownRowWaves * 64), 0, a);
    } else {
      MOE_LAUNCH(c, "decode_down", (decode_down_rows_kernel<F, NT, 1, UN, false>), grid, dim3(kDownRowWaves * 64), 0, a);
    }
  }
  const dim3 cg((unsigned)cdiv(a.d, 1024), (unsigned)a.T);
  if constexpr (F == WF_F32) MOE_LAUNCH(c, "decode_combine", decode_combine_kernel<float>, cg, dim3(256), 0, a);
  else MOE_LAUNCH(c, "decode_combine", decode_combine_kernel<bf16_t>, cg, dim3(256), 0, a);
  return hipSuccess;
}

template <int F>
hipError_t run(const LaunchCtx& c, const DecodeArgs& a) {
  if (past_cache<F>(a)) {
    HIP_RET((run_gateup<F, true>(c, a)));
    return run_down<F, true>(c, a);
  }
  HIP_RET((run_gateup<F, false>(c, a)));
  return run_down<F, false>(c, a);
}

}  // namespace

hipError_t launch_decode(const LaunchCtx& c, DecodeArgs a, int weights) {
  // 8 tokens above, 48 work-groups a slot: 103 us with each routing for itself, 98
  // with a launch before; 4 tokens: 58.9 both ways
  a.route_inline = inline_route_fits(a.T, a.k, a.E) && gu_groups(a) <= 1024;
#define TOPK(LT, KPL)                                                                                   \
  MOE_LAUNCH(c, "decode_route", (decode_topk_kernel<LT, KPL>), dim3((unsigned)a.T), dim3(64), 0,        \
             (const LT*)a.logits, a.E, a.k, a.ids, a.w, a.mid, a.mw)
#define TOPK_E(LT)                    \
  if (a.E <= 128) TOPK(LT, 2);        \
  else if (a.E <= 512) TOPK(LT, 8);   \
  else TOPK(LT, 16)
  if (a.route_inline) {
    // the gate/up kernel's
  } else if (!a.logits) {
    MOE_LAUNCH(c, "decode_route", decode_ids_kernel, dim3((unsigned)a.T), dim3(64), 0, a.ids, a.w, a.E, a.k, a.mid,
               a.mw);
  } else if (a.logits_f32) {
    TOPK_E(float);
  } else {
    TOPK_E(bf16_t);
  }
#undef TOPK_E
#undef TOPK
  if (weights == 1) return run<WF_FP8>(c, a);
  if (weights == 2) return run<WF_MX>(c, a);
  return a.dtype == F32 ? run<WF_F32>(c, a) : run<WF_BF16>(c, a);
}

}  // namespace moe
