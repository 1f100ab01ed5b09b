// Shared definitions of the HIP kernels (gfx950) and the host launchers.
#pragma once

#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

typedef uint16_t bf16_t;  // bfloat16 storage
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

enum DType { F32 = 0, BF16 = 1 };

constexpr int kWave = 64;

__device__ __forceinline__ float bf2f(bf16_t u) { return __uint_as_float((uint32_t)u << 16); }

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

// float -> bfloat16, round to nearest even (v_cvt_pk_bf16_f32).
__device__ __forceinline__ bf16_t f2bf(float f) { return __builtin_bit_cast(bf16_t, (__bf16)f); }

// Two floats -> packed bfloat16 pair (lo in bits 0..15), one instruction.
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const f32x2_t v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<bf16_t>(bf16_t v) { return bf2f(v); }

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ bf16_t from_f32<bf16_t>(float v) { return f2bf(v); }

// Logistic function with the hardware exp2 and reciprocal (about 1 ulp each).
__device__ __forceinline__ float sigmoidf_(float z) { return __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }

// Clamped SwiGLU (DeepSeek V4's, as "Mario/overlap moe kernel integration"
// names it in its commit on activations.ClampedSilu): a = silu(min(g, lim))
// * clamp(u, -lim, lim).  lim = +inf gives the plain SwiGLU, bit for bit
// (min and max with +-inf leave finite values unchanged).  In the backward
// a gradient passes only where its clamp is inactive (at lim inclusive).
// One median-of-three each (v_med3_f32): fminf / fmaxf in IEEE mode cost a
// canonicalising max per operand on top of the min and max themselves.  The
// gate's lower bound -inf comes from an opaque move: with a literal -inf the
// compiler turns the median back into that min-with-canonicalise pair.
__device__ __forceinline__ float opaque_neg_inf() {
  float v;
  asm("s_mov_b32 %0, 0xff800000" : "=s"(v));
  return v;
}
__device__ __forceinline__ float clamp_gate(float g, float lim) {
  return __builtin_amdgcn_fmed3f(g, opaque_neg_inf(), lim);
}
__device__ __forceinline__ float clamp_up(float u, float lim) { return __builtin_amdgcn_fmed3f(u, -lim, lim); }

// The same clamps where a NaN has to come through (a comparison with NaN is
// false; the median above may drop it).
__device__ __forceinline__ float clip_gate(float g, float lim) { return g > lim ? lim : g; }
__device__ __forceinline__ float clip_up(float u, float lim) { return u > lim ? lim : (u < -lim ? -lim : u); }

__host__ __device__ constexpr int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A grid of at least `blocks` (each of up to 1024 threads), and a block's number in
// it: one dimension of a grid holds fewer than 2^32 threads.
constexpr int kFold = 21;
inline dim3 folded_grid(int64_t blocks) {
  const int64_t x = blocks < (1 << kFold) ? blocks : 1 << kFold;
  return dim3((unsigned)x, (unsigned)cdiv(blocks, x));
}
__device__ __forceinline__ int64_t folded_block() { return ((int64_t)blockIdx.y << kFold) + blockIdx.x; }

// Order of a row GEMM's tiles within an expert.  Either order re-reads one
// operand once per group of tiles that runs together: taken N-tile-major,
// the token rows (once per N tile); taken row-tile-major, the weight (once
// per group of row tiles).  The re-read operand should be the one that
// stays in the caches, the smaller: row-tile-major when the token operand's
// distinct bytes exceed the weight's (as for a GPU's expert-parallel share,
// few experts with many rows), else N-tile-major.
inline int rows_tile_order(int64_t token_bytes, int64_t weight_bytes) { return token_bytes > weight_bytes; }

// ----------------------------------------------------------------------------
// Host side: every launcher enqueues through MOE_LAUNCH, which checks the
// launch status and, while the API layer is timing kernels, hands the
// dispatch a start and a stop event: the runtime stamps them with the
// kernel's own start and end, with no extra packets on the stream.
// ----------------------------------------------------------------------------
struct LaunchCtx {
  hipStream_t stream;
  // while timing: the events to attach to the named kernel's dispatch (both
  // null when none are available)
  void (*events)(const char* name, hipEvent_t* start, hipEvent_t* stop);
};

#define MOE_LAUNCH(ctx, name, kernel, grid, block, shmem, ...)                               \
  do {                                                                                       \
    hipEvent_t _start = nullptr, _stop = nullptr;                                            \
    if ((ctx).events) (ctx).events(name, &_start, &_stop);                                   \
    if (_start)                                                                              \
      hipExtLaunchKernelGGL(kernel, grid, block, shmem, (ctx).stream, _start, _stop, 0,     \
                            __VA_ARGS__);                                                    \
    else                                                                                     \
      hipLaunchKernelGGL(kernel, grid, block, shmem, (ctx).stream, __VA_ARGS__);             \
    hipError_t _e = hipGetLastError();                                                       \
    if (_e != hipSuccess) return _e;                                                         \
  } while (0)

#define HIP_RET(...)                        \
  do {                                      \
    hipError_t _r = (__VA_ARGS__);          \
    if (_r != hipSuccess) return _r;        \
  } while (0)

// ---------------------------------------------------------------- routing
// Tile table sizes: row tiles of the grouped GEMMs (expert-aligned).
constexpr int kRowTile = 256;
// Flat entries handled by one wave in the counting sort.
constexpr int kSortChunk = 1024;
constexpr int kMaxExperts = 1024;  // the C ABI rejects E outside [1, kMaxExperts]

hipError_t launch_topk(const LaunchCtx& c, const void* logits, int logits_dtype, int T, int E,
                       int k, int32_t* ids, float* w);
// counts / offsets / permutation from ids. hist: [ceil(R/kSortChunk), E] int32 scratch.
hipError_t launch_sort(const LaunchCtx& c, const int32_t* ids, int T, int E, int k,
                       int32_t* hist, int32_t* counts, int32_t* offsets, int32_t* row_of,
                       int32_t* src_of);
// GEMM schedule from offsets: tile_off [E+1] (row tiles of kRowTile per expert,
// prefix-summed), order [E] (experts by descending row count, ties by id) and,
// when blk_off is not null, blk_off [E+1] (runs of kTokBlock rows per expert,
// prefix-summed: the token blocks of the fp8 weight-gradient operands).
constexpr int kTokBlock = 128;
// tiles (optional) [tile_off[E]]: per row tile {expert, first row, end of the
// expert's segment, 0}.
// Per expert: row-tile offsets (tile_off, and tiles when non-null), order
// (experts by row count, largest first), xorder when non-null (the weight
// gradients' experts per XCD: slot s of XCD x at 8 s + x, -1 when empty; 8
// ceil(E/8) entries) and blk_off when non-null (128-row token blocks).
hipError_t launch_schedule(const LaunchCtx& c, const int32_t* offsets, int E, int32_t* tile_off,
                           int32_t* order, int32_t* xorder, int32_t* blk_off, int4* tiles);
// Upper bound of the row-tile count.
inline int64_t max_row_tiles(int64_t R, int64_t E) { return R / kRowTile + E; }

// ---------------------------------------------------------------- row passes
// xp[r] = x[src_of[r] / k]; rows of 4 or 8 KB are written as a scatter
// through row_of (x read once), others gathered through src_of.
hipError_t launch_permute(const LaunchCtx& c, const char* name, int dtype, const void* x,
                          const int32_t* src_of, const int32_t* row_of,
                          int R, int k, int d, void* xp);
// Masked experts' slots: those whose logit (of expert ids[t*k+j]) is -inf.
struct CombineMask {
  const void* logits;  // [T, E], float32 or bf16
  const int32_t* ids;  // [T, k]
  int E;
  bool f32;
};
// out[t] = sum_j (w ? w[t*k+j] : 1) * rows[row_of[t*k+j]], without the masked slots
// where there is a mask.
hipError_t launch_combine(const LaunchCtx& c, const char* name, int dtype, const void* rows,
                          const int32_t* row_of, const float* w, int T, int k, int d, void* out,
                          const CombineMask* mask = nullptr);
// bf16 SwiGLU backward per row from G [R,I] and H [R,2I]: dH [R,2I] and the
// row's top-k-weight gradient dw [R] = <G, silu(g) u>.
// lim: the SwiGLU clamp (+inf: none).
hipError_t launch_swiglu_bwd(const LaunchCtx& c, const void* G, const void* H, const float* topk_w,
                             const int32_t* src_of, int R, int I, float lim, void* dH, float* dw);
// tok[r] = src_of[r] / k: the token of each expert-sorted row.
hipError_t launch_tok_of(const LaunchCtx& c, const int32_t* src_of, int R, int k, int32_t* tok);
// d_topk_w[t,j] = sum_b dwp[row_of[t*k+j]*nblk + b]; dlogits (optional).
hipError_t launch_topk_grad(const LaunchCtx& c, const float* dwp, int nblk, const int32_t* row_of,
                            const int32_t* ids, const float* w, int T, int k, int E,
                            float* d_topk_w, void* dlogits, int logits_dtype);

// ------------------------------------------------- 8-bit activation checkpoint
// (save8.hip) H [R, 2I] as e4m3 codes with one E8M0 scale per 32 columns of
// either half: codes [R, 2I], scales [R, 2 ceil(I/32)].
inline int64_t save8_scales(int64_t I) { return 2 * cdiv(I, 32); }
// codes and scales from H, and (aw non-null) the weighted SwiGLU output.
hipError_t launch_save8(const LaunchCtx& c, int dtype, const void* H, const float* topk_w, const int32_t* src_of,
                        int R, int I, float lim, void* aw, uint8_t* codes, uint8_t* scales);
// SwiGLU backward from them and G [R, I]: dH, dw [R] = <G, a>, aw (may be null).
hipError_t launch_swiglu_bwd8(const LaunchCtx& c, int dtype, const void* G, const uint8_t* codes,
                              const uint8_t* scales, const float* topk_w, const int32_t* src_of, int R, int I,
                              float lim, void* dH, void* aw, float* dw);
// A checkpoint in place of the backward's H and Aw: aw is then written.
struct Save8 {
  const uint8_t* codes;
  const uint8_t* scales;
  void* aw;  // [R, I] workspace
};

// ---------------------------------------------------------------- GEMMs
struct LayerArgs {
  int T, d, E, k, I, R;
  int dtype;
  const void* x;
  const void* w_gate_up;
  const void* w_down;
  const float* topk_w;
  const int32_t* offsets;
  const int32_t* src_of;
  const int32_t* row_of;
  const int32_t* tile_off;  // [E+1], kRowTile tiles
  const int4* tiles;        // [tile_off[E]] row-tile descriptors
  const int32_t* order;     // [E] experts by row count, largest first
  const int32_t* xorder;    // [8 ceil(E/8)] weight-gradient slot s of XCD x at 8 s + x (-1: empty)
  const int32_t* tok_of;    // [R] token of each sorted row (backward only)
  float swiglu_lim;         // SwiGLU clamp limit, +inf for the plain SwiGLU
  bool persistent;          // bf16 row GEMMs as persistent kernels
};

// Forward GEMMs write H [R,2I] (gate|up, may be null), Aw [R,I] = w_row *
// silu(gate) * up (each row already carries its top-k weight) and Yw [R,d] =
// Aw W_down^T, so the combine is a plain sum of each token's k rows.  Yw ==
// null: the gate/up GEMM alone (the recomputing backward).
// bf16 MFMA path.  codes and scales (non-null): H's 8-bit checkpoint instead of H.
hipError_t bf16_fwd_gemms(const LaunchCtx& c, const LayerArgs& a, void* H, void* Aw, void* Yw,
                          uint8_t* codes = nullptr, uint8_t* scales = nullptr);
// backward outputs dH [R,2I], dXp [R,d], dwp [R, bf16_dw_blocks(I)] fp32, dW_gu, dW_d.
// s8 (non-null): the checkpoint that stands for H and Aw (both null then).
hipError_t bf16_bwd_gemms(const LaunchCtx& c, const LayerArgs& a, const void* dout,
                          const void* H, const void* Aw, void* dH, void* dXp, float* dwp,
                          void* dW_gu, void* dW_d, const Save8* s8 = nullptr);

// Number of per-row partials of <G, a> that the down dgrad writes (dwp [R, n]).
int bf16_dw_blocks(int I);
int f32_dw_blocks(int I);

// float32 path (plain FMA kernels, unfused epilogues).  forward needs H.
hipError_t f32_fwd_gemms(const LaunchCtx& c, const LayerArgs& a, void* H, void* Aw, void* Yw);
// backward needs G [R,I] fp32 scratch.
hipError_t f32_bwd_gemms(const LaunchCtx& c, const LayerArgs& a, const void* dout,
                         const void* H, const void* Aw, void* dH, void* dXp, float* dwp,
                         void* dW_gu, void* dW_d, float* G, const Save8* s8 = nullptr);

// ------------------------------------------------------------------ router
// (router.hip) The router's projection and its gradients.
struct RouterPlan {
  int64_t run_tokens, runs;  // dw is summed in `runs` parts of run_tokens tokens
};
RouterPlan router_plan(int64_t T, int64_t d, int64_t E, int dtype);
struct RouterArgs {
  int T, d, E;
  int dtype, logits_dtype;
  const void* x;        // [T, d]
  const void* w;        // [E, d]
  const void* dlogits;  // [T, E], backward
  const void* dx_in;    // [T, d] or null
  void* dx;             // [T, d]
  void* dw;             // [E, d]
  float* parts;         // [runs, E, d] workspace
  int64_t run_tokens;
  int runs;
  // set by the launcher
  int d_blocks, e_blocks, dw_groups, dx_eblocks, dx_blocks, dx_tokens, dx_groups;
  bool dx_first;
};
hipError_t launch_router_fwd(const LaunchCtx& c, const RouterArgs& a, void* logits);
hipError_t launch_router_bwd(const LaunchCtx& c, RouterArgs a);

// ------------------------------------------------------------------- norms
// (norm.hip) The norms around a block with its gate and residual scale.
struct NormArgs {
  int64_t T;
  int d;
  int dtype;
  int gate_kind;       // moe_gate_kind
  float scale, eps, inv_d;
  const void* x;       // forward: [T, d]
  const void* y;       // [T, d] or null
  const void* w_post;  // [d] or null
  const void* gate;    // [d] or [T] by gate_kind
  const void* w_next;  // [d] or null
  void* z;             // forward's outputs (null: not made)
  void* h;
  const void* dz;      // backward: [T, d] or null
  const void* dh;      // with w_next
  const void* z_in;    // with w_next
  void* dx;
  void* dy;            // null: no block
  void* dw_post;
  void* dgate;
  void* dw_next;
  float* parts;        // [groups, 2, d] workspace
};
// Work-groups of the backward.
int64_t norm_bwd_groups(int64_t T, int64_t d, int dtype);
hipError_t launch_norm_fwd(const LaunchCtx& c, const NormArgs& a);
hipError_t launch_norm_bwd(const LaunchCtx& c, const NormArgs& a);

// ------------------------------------------------------------ few tokens
// The whole layer for up to kDecodeMaxT tokens (decode.hip).
constexpr int kDecodeMaxT = 256;
// Whether the down products of all experts are summed in one kernel (at most 32
// slots of 8 tokens); otherwise the products of each slot go through memory and
// a combine kernel (d = 2048, where its d / 8 work-groups are one per CU, I = 768,
// 8 of 128 experts, bf16: 2 tokens 12.6 us for the down product in one kernel; 4
// tokens 19.2 and 17.7 + 4.0; 8 tokens, 64 slots, 36.4 and 28.7 + 4.0).  A smaller
// d leaves CUs without a work-group (7 tokens, 21 slots, d = 1000, float32: 8 us).
inline bool decode_one_down(int64_t T, int64_t k) { return T <= 8 && T * k <= 32; }
struct DecodeArgs {
  int T, d, E, k, I;
  int dtype;              // of x, out and aw (and of uncoded weights)
  float lim;              // SwiGLU clamp limit, +inf for the plain SwiGLU
  const void* x;          // [T, d]
  const void* w_gate_up;  // [E, 2I, d] in dtype, or e4m3 codes, or e2m1 codes [E, 2I, d/2]
  const void* s_gate_up;  // coded: fp32 [E, 2I/128, d/128] or E8M0 [E, 2I, d/32]
  const void* w_down;     // [E, d, I]
  const void* s_down;     // fp32 [E, d/128, I/128] or E8M0 [E, d, I/32]
  void* out;              // [T, d]
  const void* logits;     // [T, E], or null: ids and w are inputs
  int32_t* ids;           // [T, k]
  float* w;               // [T, k]
  bool logits_f32;
  bool route_inline;      // set by the launcher: the gate/up kernel routes
  int32_t* mid;           // [T, k] workspace: expert of the slot, -1 for an empty or merged slot
  float* mw;              // [T, k] workspace: its weight
  void* aw;               // [T k, I] workspace: weighted SwiGLU output per live slot, float32 or two bf16 planes
  float* y;               // [T k, d] workspace: down products per live slot, where they are not summed at once
};
// weights: moe_weight_format.
hipError_t launch_decode(const LaunchCtx& c, DecodeArgs a, int weights);

// ------------------------------------------------------- grouped products
// (grouped.hip) Expert-sorted rows times their experts' MXFP4 matrices.
struct GroupedArgs {
  int R, k, E, N, K;       // R: rows there are, at most
  bool swiglu;             // W = [gate; up]: y [R, N / 2]
  float lim;               // SwiGLU clamp limit, +inf for the plain SwiGLU
  const void* x;           // [R / k, K] with src_of, else [R, K]
  const int32_t* offsets;  // [E + 1]
  const int32_t* src_of;   // [R] or null
  const uint8_t* codes;    // [E, N, K / 2]
  const uint8_t* scales;   // [E, N, K / 32]
  void* y;                 // [R, N or N / 2]
  bool row_major;          // set by the launcher: tile order within an expert
};
hipError_t launch_grouped(const LaunchCtx& c, GroupedArgs a);

// ---------------------------------------------------------------- fp8 path
// Block quantisation to e4m3 (quant_fp8.hip).  Two formats: blockwise (fp32
// scales; rows 1 x 128, weights 128 x 128, tokens 128-row runs) and MX
// (E8M0 scale bytes; rows 1 x 32, weights 1 x 32 along K and, transposed,
// along N, tokens 32-row blocks inside the 128-row runs).  Scale buffers are
// typed void*: fp32 values or E8M0 bytes.
//   rows:   src [rows, C] -> q [rows, C], s [rows, C/128] fp32 or [rows, C/32] bytes;
//           run_major: the 32-bit words [C/128, rows] instead; with row_of
//           (and k), the words [C/128, rows k] of the expert-sorted rows
//           row_of[r k + j] that gather token row r;
//   weight: W [E, N, K] -> q [E, N, K] and/or qt [E, K, N]; blockwise scales
//           s [E, N/128, K/128] / st [E, K/128, N/128]; MX s [E, N, K/32] /
//           st [E, K, N/32], or with run_major the words [E, K/128, N] /
//           [E, N/128, K];
//   tok:    128-row runs of each expert's segment, written transposed q [C,
//           128 nblk_max], one 32-bit scale word per run and column [C,
//           nblk_max] (an fp32 scale, or four E8M0 codes).
hipError_t launch_quant_rows(const LaunchCtx& c, const char* name, const void* src, int64_t ld,
                             int64_t rows, int C, uint8_t* q, void* s, bool mx, bool run_major,
                             const int32_t* row_of = nullptr, int k = 1);
hipError_t launch_quant_weight(const LaunchCtx& c, const char* name, const void* W, int E, int N,
                               int K, uint8_t* q, float* s, uint8_t* qt, float* st);
hipError_t launch_quant_weight_mx(const LaunchCtx& c, const char* name, const void* W, int E, int N,
                                  int K, uint8_t* q, uint8_t* s, uint8_t* qt, uint8_t* st, bool run_major);
// run_major: scale words [run][C] (as the weight-gradient GEMMs read them)
// instead of [C][nblk_max]
hipError_t launch_quant_tok(const LaunchCtx& c, const char* name, const void* src, int64_t ld,
                            const int32_t* src_of, int kdiv, int C, const int32_t* offsets,
                            const int32_t* blk_off, int E, int nblk_max, uint8_t* q, void* s,
                            bool mx, bool run_major);

// MXFP4 (quant_mxfp4.hip): src bf16, a multiple of 32 values -> e2m1 codes, two a
// byte, and an E8M0 byte per 32.
hipError_t launch_quant_mxfp4(const LaunchCtx& c, const void* src, int64_t values, uint8_t* q, uint8_t* s);

// fp8 path's SwiGLU backward: from an fp32 G [R,I] and H, dH (bf16-rounded,
// never stored) in two e4m3 encodings: row codes dhq [R,2I] with scale words
// run-major dhs [2I/128, R], and the transposed token blocks of
// launch_quant_tok (run_major) in q / s; per-row partials of <G, a> into dw
// [R, I/128] (I % 128 == 0).
hipError_t launch_swiglu_bwd_tok(const LaunchCtx& c, const float* G, const void* H, const float* topk_w,
                                 const int32_t* src_of, int R, int I, float lim, const int32_t* offsets,
                                 const int32_t* blk_off, int E, int nblk_max, float* dw, uint8_t* dhq,
                                 void* dhs, uint8_t* q, void* s, bool mx);

// Weight codes the backward's data gradients read, left in `saved` by the
// fp8 forward: blockwise the forward encodings (one scale per 128 x 128
// block either way), MX the transposed encodings (blocks along the other
// axis).
struct Fp8Saved {
  uint8_t* wd_dgq; void* wd_dgs;    // codes and scales: blockwise [E,d,I], MX [E,I,d]
  uint8_t* wgu_dgq; void* wgu_dgs;  // blockwise [E,2I,d], MX [E,d,2I]
};
// Workspace of the fp8 forward: quantised x, weights and Aw with their scales.
struct Fp8Fwd {
  bool mx;                     // MXFP8 rather than blockwise
  uint8_t* xq; void* xs;       // codes [T,d]; scale words [d/128, R] per expert-sorted row
  uint8_t* wguq; void* wgus;   // [E,2I,d]
  uint8_t* wdq; void* wds;     // [E,d,I]
  uint8_t* awq; void* aws;     // codes [R,I]; scale words run-major [I/128, R]
  Fp8Saved sv;                 // written when saving for the backward (else null)
};
// Workspace of the fp8 backward.  tqa/tsa and tqb/tsb hold the two
// token-blocked operands of one weight gradient at a time
// ([max(d,2I)] and [max(I,d)] rows of 128 nblk_max bytes).
struct Fp8Bwd {
  bool mx;
  bool quant_weights;           // encode the weights into sv first
                                // (no fp8 forward ran)
  uint8_t* doutq; void* douts;  // codes [T,d]; scale words [d/128, R] per expert-sorted row
  Fp8Saved sv;                  // from the forward's saved buffer
  uint8_t* dhq; void* dhs;      // codes [R,2I]; scale words run-major [2I/128, R]
  uint8_t* tqa; void* tsa;
  uint8_t* tqb; void* tsb;
  float* G;                     // [R,I] the down dgrad's output
  const int32_t* blk_off;       // [E+1]
  int nblk_max;
};
int fp8_dw_blocks(int I);
// Same outputs as the bf16 path; H and Aw are stored in bf16.
hipError_t fp8_fwd_gemms(const LaunchCtx& c, const LayerArgs& a, const Fp8Fwd& q, void* H, void* Aw,
                         void* Yw);
hipError_t fp8_bwd_gemms(const LaunchCtx& c, const LayerArgs& a, const Fp8Bwd& q, const void* dout,
                         const void* H, const void* Aw, void* dXp, float* dwp, void* dW_gu, void* dW_d);

}  // namespace moe
