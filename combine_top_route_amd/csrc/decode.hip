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
//     a weight is loaded once from memory straight into its fragment, 128
//     bytes per row and step ("unit"), whatever the number of tokens;
//   * the K axis of a tile is split over the waves of a work-group and joined
//     in LDS in wave order, so all of a small problem's bytes are in flight
//     at once;
//   * nothing is sorted: each work-group finds its expert's tokens in the ids
//     (at most 256 k of them).
// All sums are float32 in a fixed order; there are no atomics.
#include <type_traits>

#include "common.h"
#include "tile.h"

namespace moe {
namespace {

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

// Top k of one token's logits, one wave per token: k rounds of a wave-wide
// maximum; among equal logits the lowest index (lane e % 64 holds experts e,
// e + 64, ..., so the first of its registers and then the lowest lane).  The
// weights are the softmax over the selected logits, summed in slot order.  A
// slot whose logit is -inf (a masked expert) is empty: id -1, weight 0.  NaN
// counts as the largest value.  KPL: keys per lane, E <= 64 KPL.
template <typename LT, int KPL>
__global__ __launch_bounds__(64) void decode_topk_kernel(const LT* __restrict__ logits, int E, int k,
                                                         int32_t* __restrict__ ids, float* __restrict__ w,
                                                         int32_t* __restrict__ mid, float* __restrict__ mw) {
  const int lane = threadIdx.x, t = blockIdx.x;
  const LT* row = logits + (int64_t)t * E;
  uint32_t key[KPL];  // 0: taken, or past E
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    const int e = lane + kWave * i;
    key[i] = 0;
    if (e < E) {
      const float v = to_f32<LT>(row[e]);
      key[i] = v != v ? 0xffffffffu : order_key(v);
    }
  }
  float top = 0.0f, sum = 0.0f;
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
    const float ex = none ? 0.0f : expf(l - top);
    sum += ex;
    if (lane == (j & 63)) {
      const int64_t f = (int64_t)t * k + j;
      ids[f] = mid[f] = none ? -1 : e;
      w[f] = ex;
    }
  }
  for (int j = lane; j < k; j += kWave) {  // each lane reads back its own stores
    const int64_t f = (int64_t)t * k + j;
    const float v = ids[f] < 0 ? 0.0f : w[f] / sum;
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
// A unit is 128 bytes of each of 16 weight rows; lane l holds row l % 16, bytes
// 16 q and 64 + 16 q with q = l / 16.  UK: values of K per unit; BV: 16-byte
// loads of a token's matching activations per lane; NF: MFMA operands.
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

// Loads go through buffer descriptors: a 32-bit offset per lane, and zeros for
// a lane that asks past the end, which is how a K tail becomes exact zeros on
// both operands (every buffer here is below kPast bytes).
constexpr uint32_t kPast = 0xffffff00u;
typedef __amdgpu_buffer_rsrc_t rsrc_t;
__device__ __forceinline__ rsrc_t buffer_of(const void* p, uint64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, (int)(uint32_t)bytes, 0x00020000);
}
__device__ __forceinline__ u32x4_t load16(rsrc_t r, uint32_t off, bool ok) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, (int)(ok ? off : kPast), 0, 0);
}

// This lane's 32 bytes of a weight row's unit; row: the row's offset plus 16 q,
// bytes: the row's length.
__device__ __forceinline__ void load_a(u32x4_t (&a)[2], rsrc_t r, uint32_t row, int unit, int q, int bytes) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int off = unit * 128 + c * 64;
    a[c] = load16(r, row + off, off + q * 16 < bytes);
  }
}

// The activations that meet load_a's bytes: the same values of K.  row: the
// token's offset.
template <int F>
__device__ __forceinline__ void load_b(u32x4_t (&b)[Fmt<F>::BV], rsrc_t r, uint32_t row, int unit, int q, int bytes) {
#pragma unroll
  for (int v = 0; v < Fmt<F>::BV; ++v) {
    const int off = F >= WF_FP8 ? unit * 256 + (v >> 1) * 128 + q * 32 + (v & 1) * 16 : unit * 128 + v * 64 + q * 16;
    b[v] = load16(r, row + off, off < bytes);
  }
}

// MFMA operands of a unit's weights.  Codes become bfloat16 exactly (e4m3 has
// four significant bits); an E8M0 scale is a power of two and rides on the
// conversion, also exactly down to bfloat16's smallest numbers (2^-133).
// mx: the row's four scale bytes of this unit.
template <int F>
__device__ __forceinline__ void to_frags(typename Fmt<F>::frag (&fr)[Fmt<F>::NF], const u32x4_t (&a)[2], uint32_t mx,
                                         int q) {
  if constexpr (F == WF_F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) fr[i] = __uint_as_float(a[i >> 2][i & 3]);
  } else if constexpr (F == WF_BF16) {
#pragma unroll
    for (int c = 0; c < 2; ++c) fr[c] = __builtin_bit_cast(bf16x8_t, a[c]);
  } else {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      // this lane's 16 codes of chunk c lie in block 2 c + q / 2
      const float s =
          F == WF_MX ? __uint_as_float(((mx >> (16 * c + 8 * (q >> 1))) & 0xffu) << 23) : 1.0f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        u32x4_t o;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t word = a[c][2 * h + i];
          o[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(word, s, false));
          o[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(word, s, true));
        }
        fr[2 * c + h] = __builtin_bit_cast(bf16x8_t, o);
      }
    }
  }
}

// s + the unit's weights times the unit's activations, unscaled.
template <int F>
__device__ __forceinline__ f32x4_t unit_dot(f32x4_t s, const typename Fmt<F>::frag (&fr)[Fmt<F>::NF],
                                            const u32x4_t (&b)[Fmt<F>::BV]) {
#pragma unroll
  for (int i = 0; i < Fmt<F>::NF; ++i) {
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

// Scales of one matrix [N, K] of an expert: blockwise fp32 [N/128, K/128], or
// E8M0 bytes [N, K/32].
template <int F>
__device__ __forceinline__ float block_scale_of(const void* s, int64_t n, int K, int unit) {
  if constexpr (F == WF_FP8) return ((const float*)s)[(n >> 7) * (K >> 7) + unit];
  return 1.0f;
}
template <int F>
__device__ __forceinline__ uint32_t mx_word_of(const void* s, int64_t n, int K, int unit) {
  if constexpr (F == WF_MX) return ((const uint32_t*)s)[n * (K >> 7) + unit];
  return 0;
}

__device__ __forceinline__ float swiglu(float g, float u, float lim) {
  const float gc = clip_gate(g, lim);
  return gc * sigmoidf_(gc) * clip_up(u, lim);
}

// ------------------------------------------------------- an expert's tokens
// Work item -> expert.  With at least as many experts as slots, item i is
// slot i, and only the first slot of an expert works on it; otherwise item e
// is expert e.  -1: nothing to do.  Uniform over the work-group.
__device__ __forceinline__ int item_expert(const int32_t* __restrict__ mid, int item, int R, int E) {
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

// Fills `rows` with the slots that chose expert e; returns their number.  At
// least 256 threads.
__device__ __forceinline__ int find_rows(Rows& rows, const int32_t* __restrict__ mid, const float* __restrict__ mw,
                                         int e, int T, int k) {
  const int t = threadIdx.x, wave = t >> 6;
  int slot = -1;
  if (t < T)
    for (int j = 0; j < k; ++j)
      if (mid[t * k + j] == e) slot = t * k + j;  // at most one (see decode_ids_kernel)
  const uint64_t has = __ballot(slot >= 0);
  if (wave < 4 && (t & 63) == 0) rows.part[wave] = __popcll(has);
  __syncthreads();
  int before = 0, n = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    before += i < wave ? rows.part[i] : 0;
    n += rows.part[i];
  }
  if (slot >= 0) {
    const int r = before + __popcll(has & ((1ull << (t & 63)) - 1));
    rows.slot[r] = slot;
    rows.w[r] = mw[slot];
  }
  __syncthreads();
  return n;
}

// ------------------------------------------------------------ gate/up product
// One work-group: 16 gate rows and the same 16 up rows of one expert, for all
// of its tokens; the NW waves take the units of K in turn, UN at a time.
template <int F, int UN>
struct GuWeights {  // UN units of this lane's gate and up row, in flight
  u32x4_t g[UN][2], u[UN][2];
  uint32_t mg[UN], mu[UN];
};

template <int F, int NW, int UN>
__device__ __forceinline__ void load_gu(GuWeights<F, UN>& w, rsrc_t wr, const void* sc, int I, int K, int row,
                                        int base, int q) {
  const int units = (K + Fmt<F>::UK - 1) / Fmt<F>::UK;
  const int bytes = F >= WF_FP8 ? K : K * (int)sizeof(typename Fmt<F>::act);
  const uint32_t g = (uint32_t)row * bytes + q * 16, u = (uint32_t)(I + row) * bytes + q * 16;
#pragma unroll
  for (int i = 0; i < UN; ++i) {
    const int unit = base + i * NW, us = min(unit, units - 1);
    load_a(w.g[i], wr, g, unit, q, bytes);
    load_a(w.u[i], wr, u, unit, q, bytes);
    w.mg[i] = mx_word_of<F>(sc, row, K, us);
    w.mu[i] = mx_word_of<F>(sc, I + row, K, us);
  }
}

// The tokens r0 .. r0 + 16 NB of the expert.  w holds the first units; UB
// units' activations are loaded at a time (they come from the caches).
template <int F, int NW, int UN, int NB, int UB>
__device__ __forceinline__ void gateup_rows(const DecodeArgs& a, const Rows& rows, int r0, int n,
                                            GuWeights<F, UN>& w, rsrc_t wr, const void* sc, int n0, int row,
                                            float* red) {
  typedef typename Fmt<F>::act AT;
  const int lane = threadIdx.x & 63, wave = tile::wave_id(), q = lane >> 4, col = lane & 15;
  const int K = a.d;
  const int units = (K + Fmt<F>::UK - 1) / Fmt<F>::UK;
  const int bytes = K * (int)sizeof(AT);
  const rsrc_t xb = buffer_of(a.x, (uint64_t)a.T * bytes);
  uint32_t xr[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int r = min(r0 + b * 16 + col, n - 1);  // columns past the last token repeat it and are dropped
    xr[b] = (uint32_t)(rows.slot[r] / a.k) * bytes;
  }
  f32x4_t ag[NB], au[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) ag[b] = au[b] = f32x4_t{0, 0, 0, 0};
  for (int base = wave; base < units; base += NW * UN) {
    if (base != wave || r0) load_gu<F, NW, UN>(w, wr, sc, a.I, K, row, base, q);
#pragma unroll
    for (int i0 = 0; i0 < UN; i0 += UB) {
      u32x4_t xv[UB][NB][Fmt<F>::BV];
#pragma unroll
      for (int i = 0; i < UB; ++i)
#pragma unroll
        for (int b = 0; b < NB; ++b) load_b<F>(xv[i][b], xb, xr[b], base + (i0 + i) * NW, q, bytes);
      __builtin_amdgcn_sched_barrier(0);  // all loads leave before the first product waits
#pragma unroll
      for (int i = 0; i < UB; ++i) {
        const int us = min(base + (i0 + i) * NW, units - 1);
        const float sg = block_scale_of<F>(sc, n0, K, us), su = block_scale_of<F>(sc, a.I + n0, K, us);
        typename Fmt<F>::frag fr[Fmt<F>::NF];
        to_frags<F>(fr, w.g[i0 + i], w.mg[i0 + i], q);
#pragma unroll
        for (int b = 0; b < NB; ++b) unit_mma<F>(ag[b], fr, xv[i][b], sg);
        to_frags<F>(fr, w.u[i0 + i], w.mu[i0 + i], q);
#pragma unroll
        for (int b = 0; b < NB; ++b) unit_mma<F>(au[b], fr, xv[i][b], su);
      }
    }
  }
  // red [wave][2 b + gate/up][col][16 rows]
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    float* p = red + ((wave * NB + b) * 2 * 16 + col) * 16 + q * 4;
    *(f32x4_t*)p = ag[b];
    *(f32x4_t*)(p + 256) = au[b];
  }
  __syncthreads();
  for (int o = threadIdx.x; o < NB * 256; o += NW * 64) {
    const int b = o >> 8, c = (o >> 4) & 15, m = o & 15;
    const int r = r0 + b * 16 + c;
    if (r < n && n0 + m < a.I) {
      float g = 0.0f, u = 0.0f;
#pragma unroll
      for (int v = 0; v < NW; ++v) {
        const float* p = red + ((v * NB + b) * 2 * 16 + c) * 16 + m;
        g += p[0];
        u += p[256];
      }
      ((AT*)a.aw)[(int64_t)rows.slot[r] * a.I + n0 + m] = from_f32<AT>(rows.w[r] * swiglu(g, u, a.lim));
    }
  }
  __syncthreads();
}

template <int F, int NBMAX, int NW, int UN>
__global__ __launch_bounds__(NW * 64) void decode_gateup_kernel(DecodeArgs a) {
  __shared__ Rows rows;
  __shared__ float red[NW * NBMAX * 512];
  const int e = __builtin_amdgcn_readfirstlane(item_expert(a.mid, blockIdx.y, a.T * a.k, a.E));
  if (e < 0) return;
  const int lane = threadIdx.x & 63, q = lane >> 4;
  const int n0 = blockIdx.x * 16;
  const int row = min(n0 + (lane & 15), a.I - 1);  // rows past I repeat the last and are dropped
  const int64_t wb = F >= WF_FP8 ? 1 : sizeof(typename Fmt<F>::act);
  const uint64_t wbytes = (uint64_t)2 * a.I * a.d * wb;
  const rsrc_t wr = buffer_of((const char*)a.w_gate_up + e * wbytes, wbytes);
  const char* sc = (const char*)a.s_gate_up;
  if (F == WF_FP8) sc += (int64_t)e * (2 * a.I / 128) * (a.d / 128) * 4;
  if (F == WF_MX) sc += (int64_t)e * 2 * a.I * (a.d / 32);
  const int n = find_rows(rows, a.mid, a.mw, e, a.T, a.k);
  if (n == 0) return;
  GuWeights<F, UN> w;
  load_gu<F, NW, UN>(w, wr, sc, a.I, a.d, row, tile::wave_id(), q);
  constexpr int UB1 = F >= WF_FP8 ? (UN > 2 ? 2 : UN) : UN;
  if constexpr (NBMAX == 1) {
    gateup_rows<F, NW, UN, 1, UB1>(a, rows, 0, n, w, wr, sc, n0, row, red);
  } else {
    for (int r0 = 0; r0 < n; r0 += 64) {
      const int left = n - r0;
      if (left <= 16) gateup_rows<F, NW, UN, 1, UB1>(a, rows, r0, n, w, wr, sc, n0, row, red);
      else if (left <= 32) gateup_rows<F, NW, UN, 2, (UB1 + 1) / 2>(a, rows, r0, n, w, wr, sc, n0, row, red);
      else gateup_rows<F, NW, UN, 4, 1>(a, rows, r0, n, w, wr, sc, n0, row, red);
    }
  }
}

// ---------------------------------------------- down product, up to 16 tokens
// One work-group: 16 rows of d for all tokens and all experts.  An MFMA's
// columns are the tokens, so one accumulator runs over every (expert, unit of
// I) pair, and the combine is the sum itself (aw carries the weights).  aw is
// rounded to the activations' type like the layer's, for the MFMA's operand.
constexpr int kDownWaves = 16;

template <int F>
__global__ __launch_bounds__(kDownWaves * 64) void decode_down_kernel(DecodeArgs a) {
  typedef typename Fmt<F>::act AT;
  extern __shared__ __align__(16) char smem[];
  float* red = (float*)smem;                              // [waves][16 tokens][16 rows]
  int* active = (int*)(red + kDownWaves * 256);           // [E] experts with tokens
  uint16_t* tab = (uint16_t*)(active + a.E);              // [E][T] slot of the token + 1, 0: none
  __shared__ int counts[kDownWaves];
  const int lane = threadIdx.x & 63, wave = tile::wave_id(), q = lane >> 4, col = lane & 15;
  const int R = a.T * a.k, cells = a.E * a.T;
  for (int i = threadIdx.x; i < cells; i += kDownWaves * 64) tab[i] = 0;
  __syncthreads();
  for (int f = threadIdx.x; f < R; f += kDownWaves * 64) {
    const int e = a.mid[f], t = f / a.k;
    if (e >= 0) tab[e * a.T + t] = (uint16_t)(f - t * a.k + 1);
  }
  __syncthreads();
  // E <= 1024 threads: expert e is thread e
  bool on = false;
  if ((int)threadIdx.x < a.E)
    for (int t = 0; t < a.T; ++t) on |= tab[threadIdx.x * a.T + t] != 0;
  const uint64_t has = __ballot(on);
  if (lane == 0) counts[wave] = __popcll(has);
  __syncthreads();
  int before = 0, nact = 0;
  for (int i = 0; i < kDownWaves; ++i) {
    before += i < wave ? counts[i] : 0;
    nact += counts[i];
  }
  if (on) active[before + __popcll(has & ((1ull << lane) - 1))] = threadIdx.x;
  __syncthreads();

  const int K = a.I, n0 = blockIdx.x * 16;
  const int row = min(n0 + col, a.d - 1);
  const int units = (K + Fmt<F>::UK - 1) / Fmt<F>::UK;
  const int abytes = F >= WF_FP8 ? K : K * (int)sizeof(AT), bbytes = K * (int)sizeof(AT);
  const uint64_t wbytes = (uint64_t)a.d * abytes;
  const uint32_t wrow = (uint32_t)row * abytes + q * 16;
  const rsrc_t xb = buffer_of(a.aw, (uint64_t)a.T * a.k * bbytes);
  const int total = nact * units;
  constexpr int UN = 4;
  f32x4_t acc = {0, 0, 0, 0};
  for (int base = wave; base < total; base += kDownWaves * UN) {
    u32x4_t wv[UN][2], xv[UN][Fmt<F>::BV];
    uint32_t mx[UN];
    float sb[UN];
    bool on_expert[UN];
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      const int p = base + i * kDownWaves;
      const bool live = p < total;  // uniform in the wave
      const int idx = live ? p / units : 0, unit = live ? p - idx * units : 0;
      const int e = __builtin_amdgcn_readfirstlane(active[idx]);
      const int j = col < a.T ? tab[e * a.T + col] : 0;
      const bool mine = on_expert[i] = live && j != 0;
      load_a(wv[i], buffer_of((const char*)a.w_down + e * wbytes, wbytes), wrow, unit, q, live ? abytes : 0);
      load_b<F>(xv[i], xb, (uint32_t)(col * a.k + j - 1) * bbytes, unit, q, mine ? bbytes : 0);
      const char* sc = (const char*)a.s_down;
      if (F == WF_FP8) sc += (int64_t)e * (a.d / 128) * (K / 128) * 4;
      if (F == WF_MX) sc += (int64_t)e * a.d * (K / 32);
      mx[i] = mx_word_of<F>(sc, row, K, unit);
      sb[i] = block_scale_of<F>(sc, n0, K, unit);
    }
    __builtin_amdgcn_sched_barrier(0);  // all loads leave before the first product waits
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      typename Fmt<F>::frag fr[Fmt<F>::NF];
      to_frags<F>(fr, wv[i], mx[i], q);
      // a lane's results are its own column's: a token takes nothing from an
      // expert that it did not choose, whatever that expert's weights hold
      const f32x4_t s = unit_dot<F>(f32x4_t{0, 0, 0, 0}, fr, xv[i]);
#pragma unroll
      for (int m = 0; m < 4; ++m) acc[m] = on_expert[i] ? fmaf(sb[i], s[m], acc[m]) : acc[m];
    }
  }
  *(f32x4_t*)(red + (wave * 16 + col) * 16 + q * 4) = acc;
  __syncthreads();
  for (int o = threadIdx.x; o < 256; o += kDownWaves * 64) {
    const int t = o >> 4, m = o & 15;
    if (t < a.T && n0 + m < a.d) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kDownWaves; ++w) v += red[(w * 16 + t) * 16 + m];
      ((AT*)a.out)[(int64_t)t * a.d + n0 + m] = from_f32<AT>(v);
    }
  }
}

// --------------------------------------------- down product, more tokens
// One wave: 16 rows of d of one expert for its tokens, all of I; the products
// go to y [T k, d] in float32, which decode_combine_kernel sums in slot order.
constexpr int kDownRowWaves = 4;

template <int F, int NB, int UN>
__device__ __forceinline__ void down_rows(const DecodeArgs& a, const Rows& rows, int r0, int n, rsrc_t wr,
                                          const void* sc, int n0, int row) {
  typedef typename Fmt<F>::act AT;
  const int lane = threadIdx.x & 63, q = lane >> 4, col = lane & 15;
  const int K = a.I;
  const int units = (K + Fmt<F>::UK - 1) / Fmt<F>::UK;
  const int abytes = F >= WF_FP8 ? K : K * (int)sizeof(AT), bbytes = K * (int)sizeof(AT);
  const uint32_t wrow = (uint32_t)row * abytes + q * 16;
  const rsrc_t xb = buffer_of(a.aw, (uint64_t)a.T * a.k * bbytes);
  uint32_t xr[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) xr[b] = (uint32_t)rows.slot[min(r0 + b * 16 + col, n - 1)] * bbytes;
  f32x4_t acc[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) acc[b] = f32x4_t{0, 0, 0, 0};
  for (int base = 0; base < units; base += UN) {
    u32x4_t wv[UN][2], xv[UN][NB][Fmt<F>::BV];
    uint32_t mx[UN];
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      load_a(wv[i], wr, wrow, base + i, q, abytes);
      mx[i] = mx_word_of<F>(sc, row, K, min(base + i, units - 1));
#pragma unroll
      for (int b = 0; b < NB; ++b) load_b<F>(xv[i][b], xb, xr[b], base + i, q, bbytes);
    }
    __builtin_amdgcn_sched_barrier(0);  // all loads leave before the first product waits
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      typename Fmt<F>::frag fr[Fmt<F>::NF];
      to_frags<F>(fr, wv[i], mx[i], q);
      const float sb = block_scale_of<F>(sc, n0, K, min(base + i, units - 1));
#pragma unroll
      for (int b = 0; b < NB; ++b) unit_mma<F>(acc[b], fr, xv[i][b], sb);
    }
  }
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int r = r0 + b * 16 + col;
    if (r < n && n0 + q * 4 < a.d)  // d is a multiple of 8: four rows are in or out together
      *(f32x4_t*)(a.y + (int64_t)rows.slot[r] * a.d + n0 + q * 4) = acc[b];
  }
}

template <int F>
__global__ __launch_bounds__(kDownRowWaves * 64) void decode_down_rows_kernel(DecodeArgs a) {
  __shared__ Rows rows;
  const int e = __builtin_amdgcn_readfirstlane(item_expert(a.mid, blockIdx.y, a.T * a.k, a.E));
  if (e < 0) return;
  const int n = find_rows(rows, a.mid, a.mw, e, a.T, a.k);
  const int n0 = (blockIdx.x * kDownRowWaves + tile::wave_id()) * 16;
  if (n == 0 || n0 >= a.d) return;  // no barrier follows
  const int row = min(n0 + (int)(threadIdx.x & 15), a.d - 1);
  const int64_t wb = F >= WF_FP8 ? 1 : sizeof(typename Fmt<F>::act);
  const uint64_t wbytes = (uint64_t)a.d * a.I * wb;
  const rsrc_t wr = buffer_of((const char*)a.w_down + e * wbytes, wbytes);
  const char* sc = (const char*)a.s_down;
  if (F == WF_FP8) sc += (int64_t)e * (a.d / 128) * (a.I / 128) * 4;
  if (F == WF_MX) sc += (int64_t)e * a.d * (a.I / 32);
  for (int r0 = 0; r0 < n; r0 += 64) {
    const int left = n - r0;
    if (left <= 16) down_rows<F, 1, 4>(a, rows, r0, n, wr, sc, n0, row);
    else if (left <= 32) down_rows<F, 2, 2>(a, rows, r0, n, wr, sc, n0, row);
    else down_rows<F, 4, 1>(a, rows, r0, n, wr, sc, n0, row);
  }
}

// out[t] = sum of the token's live slots of y, in slot order; one rounding.
template <typename AT>
__global__ __launch_bounds__(256) void decode_combine_kernel(DecodeArgs a) {
  const int c = blockIdx.x * 256 + threadIdx.x, t = blockIdx.y;
  if (c * 4 >= a.d) return;
  f32x4_t acc = {0, 0, 0, 0};
  for (int j = 0; j < a.k; ++j) {
    const int64_t f = (int64_t)t * a.k + j;
    if (a.mid[f] >= 0) {
      const f32x4_t v = *(const f32x4_t*)(a.y + f * a.d + c * 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] += v[i];
    }
  }
  AT* o = (AT*)a.out + (int64_t)t * a.d + c * 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = from_f32<AT>(acc[i]);
}

template <int F>
hipError_t run(const LaunchCtx& c, const DecodeArgs& a) {
  const int R = a.T * a.k;
  const unsigned items = (unsigned)(R > a.E ? a.E : R);
  const dim3 gu((unsigned)cdiv(a.I, 16), items);
  constexpr int UN = F >= WF_FP8 ? 2 : 4;
  if (a.T <= 16) {
    MOE_LAUNCH(c, "decode_gateup", (decode_gateup_kernel<F, 1, 8, UN>), gu, dim3(8 * 64), 0, a);
    const size_t smem = kDownWaves * 1024 + (size_t)a.E * 4 + (size_t)a.E * a.T * 2;  // at most 52 KB
    MOE_LAUNCH(c, "decode_down", decode_down_kernel<F>, dim3((unsigned)cdiv(a.d, 16)), dim3(kDownWaves * 64), smem, a);
    return hipSuccess;
  }
  MOE_LAUNCH(c, "decode_gateup", (decode_gateup_kernel<F, 4, 4, UN / 2>), gu, dim3(4 * 64), 0, a);
  MOE_LAUNCH(c, "decode_down", decode_down_rows_kernel<F>, dim3((unsigned)cdiv(a.d, 16 * kDownRowWaves), items),
             dim3(kDownRowWaves * 64), 0, a);
  const dim3 cg((unsigned)cdiv(a.d, 1024), (unsigned)a.T);
  if constexpr (F == WF_F32) MOE_LAUNCH(c, "decode_combine", decode_combine_kernel<float>, cg, dim3(256), 0, a);
  else MOE_LAUNCH(c, "decode_combine", decode_combine_kernel<bf16_t>, cg, dim3(256), 0, a);
  return hipSuccess;
}

}  // namespace

hipError_t launch_decode(const LaunchCtx& c, const DecodeArgs& a, const void* logits, int logits_dtype, int32_t* ids,
                         float* w, int weights) {
#define TOPK(LT, KPL)                                                                                   \
  MOE_LAUNCH(c, "decode_route", (decode_topk_kernel<LT, KPL>), dim3((unsigned)a.T), dim3(64), 0,        \
             (const LT*)logits, a.E, a.k, ids, w, a.mid, a.mw)
#define TOPK_E(LT)                    \
  if (a.E <= 128) TOPK(LT, 2);        \
  else if (a.E <= 512) TOPK(LT, 8);   \
  else TOPK(LT, 16)
  if (!logits)
    MOE_LAUNCH(c, "decode_route", decode_ids_kernel, dim3((unsigned)a.T), dim3(64), 0, ids, w, a.E, a.k, a.mid, a.mw);
  else if (logits_dtype == F32) {
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
