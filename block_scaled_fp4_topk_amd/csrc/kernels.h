// Internal launcher interface between the C-ABI layer (api.cpp) and the HIP
// kernels.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/moefp4.h"

namespace moefp4 {

constexpr int kMaxExperts = 512;

// The router's selection (moefp4_gate): E routed experts, bias [E] or null.
struct GateSel {
  int E, top_k, shared, scoring, renorm;
  float scale;
  const float* bias;
};
constexpr int kGateMaxTopK = 64;   // one lane per selected expert
// Most tokens the dot form is used for, with bfloat16 and with FP32 weights
// (which the tiled form splits first).  Both forms, dot / tiled, with the
// selection, for 256 experts, us:
//                     8 tokens   16         32         64
//   bf16, H = 6144   10.6/10.8  11.1/10.9  13.4/11.2
//         H = 2048    9.2/8.6    9.6/8.7   10.6/9.0
//   FP32, H = 6144   10.7/20.9  11.0/20.8  13.8/21.0  17.5/21.9
//         H = 2048    9.2/13.0   9.6/12.9  10.6/13.2  13.1/13.9
// The borders move little with the number of experts.  H = 6144 / 2048: bf16, 8
// tokens, 64 experts 9.6/9.7 and 8.4/7.6, 512 experts 12.3/12.8 and 10.9/10.7;
// FP32, 64 tokens, 64 experts 10.5/16.7 and 9.0/11.6, 512 experts 27.1/28.3 and
// 19.1/17.5 (128 tokens of 64 experts 13.1/17.2, of 512 44.3/28.5).
constexpr int kGateDotMax = 8, kGateDotMaxF32 = 64;

// Logits of T tokens: one dot product per expert and token (dot), or a tiled
// product with K split in `parts` of `per` stages.  part_bytes: the logits
// [parts][T][ld] float32, most_bytes: the most that T or fewer tokens need for
// them; planes_bytes: FP32 weights as bfloat16 planes.
struct GatePlan {
  bool dot;
  int per, parts, ld;
  size_t planes_bytes, part_bytes, most_bytes;
};
GatePlan gate_plan(int T, int E, int H, bool w_f32);
hipError_t launch_gate(const GatePlan& p, const GateSel& g, const void* w, bool w_f32, const uint16_t* x, int T, int H,
                       uint16_t* planes, float* part, int32_t* ids, float* wts, hipStream_t s);

// Tile of activation rows processed by one grouped-GEMM workgroup.
struct RouteOut {
  int32_t* counts;         // [E]
  int32_t* offsets;        // [E+1]
  int32_t* sorted_assign;  // [A]
  int32_t* slot_of;        // [A]
  int32_t* tiles;          // [2 * max_tiles] (expert, first row)
  int32_t* ntiles;         // [1]
  int32_t* flags;          // [1] dropped assignments
  uint32_t* zero_words;    // optional [n_zero] words cleared by the route kernel
  int n_zero;
  // optional: per-token fp16 staging scale of bf16 rows x [T, H] (row_scale
  // null: not computed); row_scale[t] = 2**p_t with p_t chosen so the row
  // maximum times 2**-p_t lies in [2**14, 2**15)
  const uint16_t* x;
  int T, H;
  float* row_scale;
  // optional (with row_scale): the rows themselves converted, fp16(x * 2**-p_t)
  // [T, H] (exact: 8 significant bits inside the fp16 range)
  uint16_t* x16;
  // optional: FP8 + UE8M0 per 32 quantisation of bf16 rows x [T, H] into
  // x8 [T, H] and xsf [T, H/32] (x8 null: not computed); x_fp4: MXFP4
  // (E2M1 + UE8M0 per 32) instead, x8 [T, H/2]
  uint8_t* x8;
  uint8_t* xsf;
  bool x_fp4;
  // multi-workgroup form (nchunks > 0): chunks of `chunk` assignments and a
  // [nchunks][E + 1] int32 scratch for their histograms / starts
  int nchunks, chunk;
  int32_t* hist;
};

// Assignments per chunk of the multi-workgroup route (T * k above
// kRouteSingleMax uses it).
constexpr int kRouteSingleMax = 8192;
constexpr int kRouteMaxChunks = 64;
inline int route_chunk(long long A) {
  long long c = (A + kRouteMaxChunks - 1) / kRouteMaxChunks;
  c = (c + 1023) / 1024 * 1024;
  return (int)(c < 4096 ? 4096 : c);
}

hipError_t launch_route(const int32_t* topk_ids, int A, int E, int tile_m, const RouteOut& o,
                        hipStream_t s);

// bf16 [T, H] -> E4M3 [T, H] + UE8M0 [T, H/32]: per 32 elements e =
// ceil(log2(amax / 448)) (amax == 0: e = -127), clamped to [-127, 127],
// codes RNE(x / 2**e), sign kept.  fp4: MXFP4 instead, E2M1 [T, H/2] (two
// per byte, even element low) with e = ceil(log2(amax / 6)).  H % 32 == 0.
hipError_t launch_quantize_act(const uint16_t* x, long long T, int H, uint8_t* xq, uint8_t* xsf,
                               bool fp4, hipStream_t s);

// bf16 [T, H] -> fp16 [T, H] * 2**-p_t with p_t chosen per row so the row
// maximum lands in [2**14, 2**15); scale[t] = 2**p_t.
hipError_t launch_rows_to_f16(const uint16_t* x, int T, int H, uint16_t* x16, float* scale,
                              hipStream_t s);

// The whole layer for a few tokens in two launches (layer.hip).  T <= 8,
// H % 256 == 0, H <= 6144, I % 256 == 0, I * H < 2^31, at most 16 experts per
// token (shared ones among them), E = routed + shared <= 512.
// Up to 8 tokens with group16, 2 with group32 weights.  Both forms, captured
// in a graph, two launches / gate + forward, us:
//                                     T = 1      2        4          8        16
//   256 experts, H 6144, I 2048, g16: 58/65    86/89    132/143   238/259   412/399
//                                g32: 54/63    79/77    135/136   231/223   379/343
//   128 experts, H 4096, I 1536, g16: 39/50    55/57     80/97    126/146   188/194
//                                g32: 35/45    48/53     78/72    117/108   171/151
//    64 experts, H 2048, I 768,  g16: 31/34    34/36     42/42     52/46     61/58
//                                g32: 27/32    31/34     35/35     45/39     56/45
// (Beyond the limits: measured in a form that took 16 tokens of either.  FC2
// takes a few instructions more per weight than the decode tiles, two products
// with group32; without a graph gate + forward has five launches more to
// enqueue.)
constexpr int kFewTokens = 8, kFewTokensG32 = 2;
constexpr int kFewMaxH = 6144;
constexpr int kFewMaxK = 16;
struct FewArgs {
  GateSel g;              // E: routed experts
  int T, H, I, w13_order;
  bool g16, w_f32, out_f32;
  const uint16_t* x;      // [T, H] bf16
  const void* gate_w;
  const uint8_t *w13, *w13_sf, *w2, *w2_sf;
  const float *w13_gs, *w2_gs;
  void* out;
  int32_t* ids;           // optional outputs [T, top_k + shared]
  float* wts;
  // workspace
  int32_t* flags;         // [2] places without an expert, waits past their limit
  float* logits;          // [T][ld]
  int ld;
  uint16_t* x16;          // group16: x as fp16 * 2**-p [T, H] ...
  float* xs;              // ... and 2**p [T]
  uint16_t* h;            // [T * k][I] fp16 in blocks of 16 with a shared exponent (group16), or bf16 high and low
                          // parts [2][T * k][I] (group32)
  int8_t* hexp;           // group16: [T * k][I / 16] exponents
  int32_t* sync;          // [few_sync_words]
  float* part;            // [workgroups][2][64 lanes][8] partial outputs
  int nwg;
  int looks;              // at FC1's counters before a wait is given up
};
// About a microsecond each, 0.3 s in all.  (Counted, not timed: a clock goes on
// while the queue is switched out for another process's.)
constexpr int kFewLooks = 1 << 18;
// launch 2's counters: a queue and a count of finished items per XCD, a line
// each, then one word per 32 outputs
constexpr int kFewQueues = 8, kFewLine = 32;
constexpr int few_sync_words(int H) { return 2 * kFewQueues * kFewLine + H / 32; }
hipError_t launch_few(const FewArgs& a, hipStream_t s);
// CUs of the current device (the workgroups of the persistent kernels)
int cu_count();

// The projection with adapters (project.hip).  K % 256 == 0, N % 16 == 0, R a
// multiple of 8 up to 128, N * K < 2^32, T < 2^24.
// Most tokens of the form for few tokens; beyond, the tiled product.  Both at
// N = 4096, K = 6144, group16 without adapters: 64 tokens 14.8 us against 23.4
// us, 128 tokens 23.7 against 27.6; N = 1968, K = 2048: 128 tokens 11.7 against
// 15.2.  (256 tokens in the few form: 117 us against 35.)
constexpr int kProjectFew = 128;
// u by dot products (every token reads its adapter's A for itself), or with
// matrix instructions, the tokens grouped by adapter?  Whole calls, dot / grouped,
// us: K = 6144, rank 16, 512 tokens (50 M) 68/70, 700 (69 M) 106/100; rank 64,
// 128 tokens (50 M) 41/55, 200 (79 M) 58/53; K = 2048, rank 8, 512 tokens (8 M)
// 27/39, 4096 (67 M) 69/72, 8192 (134 M) 117/100.
inline bool project_dot(long long T, long long K, long long R) { return T * K * R <= (64ll << 20); }
struct ProjectArgs {
  int T, N, K, L, R;   // L = 0: no adapters
  bool g16, out_f32;
  const uint16_t* x;   // [T, K] bf16
  const uint8_t *w, *w_sf;
  const float* w_gs;   // [1] or null
  const uint16_t *a, *b;  // [L, R, K], [L, N, R] bf16
  const int32_t* id;      // [T]
  const float* scale;     // [L]
  void* out;
  // workspace
  uint16_t* x16;  // few tokens: x as the products read it (fp16 * 2**-p for group16)
  float* xs;      // few tokens, group16: 2**p [T]
  float* u;       // [ku][T, R]
  int ku;
  float* part;    // [parts][T, N] of the tiled product
  RouteOut route; // u by matrix instructions: tokens grouped by adapter, tiles of 32
  int32_t* ids;   // [T] what they are grouped by
  const int32_t* order;  // [T] tokens in that order (route.sorted_assign), or null
};
// The tiled product: tokens per workgroup, parts of K and their 64-element
// stages.
struct ProjectGemm {
  int tt, per, parts;
};
// parts of K in which u is computed
int project_u_parts(long long T, long long K, long long R);
ProjectGemm project_gemm_plan(long long T, long long N, long long K);
// The most rows that u and the tiled product's parts (0: it has one) take for T
// or fewer tokens.
long long project_u_rows(long long T, long long K, long long R);
long long project_part_rows(long long T, long long N, long long K);
hipError_t launch_project(const ProjectArgs& a, hipStream_t s);

// Products grouped by expert (moe_fp4_grouped, _dx, _dw).  form 0: p = x [M, K],
// q = W [E, N, K], out [M, N]; 1: p = dy [M, N], q = W, out [M, K]; 2: p = dy,
// q = x, out [E, N, K].
struct GroupedArgs {
  int M, E, N, K;
  int gran;           // 0: bfloat16 weights; 16, 32: FP4 (w, w_sf, w_gs in place of q)
  int out_f32, accumulate;
  int stream;         // the output is larger than the caches (set by launch_grouped, as parts is)
  int parts, group, many;  // of every sum; consecutive tiles per XCD; tiles per workgroup
  float* part;        // [parts][outputs] where parts > 1
  const uint16_t *p, *q;
  const uint8_t *w, *w_sf;
  const float* w_gs;
  const int32_t* offsets;
  void* out;
};
// The form of a product: few 1, 2: the stream of the weights with 16 or 32 rows
// per workgroup; else many > 0: so many tiles of 64 x 128 per workgroup, or tiles
// of tile x tile outputs (64: 64 x 128), the sums in parts.
struct GroupedPlan { int few, tile, parts, many, far; };
GroupedPlan grouped_plan(int form, long long M, long long E, long long N, long long K, int gran);
// The most floats that the parts of M or fewer rows take.
long long grouped_part_floats(int form, long long M, long long E, long long N, long long K);
hipError_t launch_grouped(const GroupedArgs& a, int form, hipStream_t s);

// Block norms (moe_fp4_block_norm, _grad).  gate_kind 0: none, 1: [H], 2: [T],
// 3: [T, H]; gate_act 1: sigmoid.
struct NormArgs {
  long long T;
  int H, h_f32, post_f32, pre_f32, gate_f32, gate_kind, gate_act;
  float scale, h_scale, eps;
  const void *h, *y, *post_w, *gate, *pre_w;
  void *h_out, *n;
  const void *dh, *dn;
  void *d_h, *d_y, *d_gate;
  float *d_post_w, *d_pre_w;
  float* part;  // [3][norm_grad_parts][H]
};
constexpr int kNormMostH = 16384;
int norm_grad_parts(long long T, int H);
hipError_t launch_block_norm(const NormArgs& a, hipStream_t s);
hipError_t launch_block_norm_grad(const NormArgs& a, hipStream_t s);

struct FcArgs {
  const uint8_t* w;          // [E, N, K/2]
  const uint8_t* wsf;        // [E, N, K/gran]
  const float* gs;           // [E] or null
  const void* act;           // FC1: x or x16 [T, K]; FC2: h [A, K]
  const uint8_t* act_sf;     // A8: [rows, K/32] UE8M0
  const float* act_scale;    // A16 group16 FC1: per token 2**p
  const uint32_t* hmax_in;   // A16 group16 FC2: per slot max |h| bits
  const int32_t* tiles;
  const int32_t* ntiles;
  const int32_t* counts;
  const int32_t* offsets;
  const int32_t* sorted_assign;
  int K, N, I, H, top_k, w13_order;
  void* h_out;               // FC1: h [A, I] (bf16 or fp8)
  uint8_t* h_sf_out;         // FC1 A8: [A, I/32]
  uint32_t* hmax_out;        // FC1 A16 group16: per slot max |h| bits
  float* y_out;              // FC2: [A, H]
};

// 64-row expert tiles (bf16 activations with more than 16 assignments per
// active expert, and FP8 activations at shapes the prefill GEMM does not take)
hipError_t launch_fc1_a16(const FcArgs& a, int gran, int max_tiles, hipStream_t s);
hipError_t launch_fc2_a16(const FcArgs& a, int gran, int max_tiles, hipStream_t s);
hipError_t launch_fc1_a8(const FcArgs& a, int max_tiles, hipStream_t s);
hipError_t launch_fc2_a8(const FcArgs& a, int max_tiles, hipStream_t s);

// Decode-shaped FC kernels (expert tiles of <= 16 activation rows); mode 0:
// bf16 x group16, 1: bf16 x group32, 2: FP8 x group32, 3: MXFP4 x group32
// (act [rows, K/2], h written as MXFP4).  Needs K % 256 == 0,
// I % 64 == 0 (FC1) and H % 128 == 0 (FC2).
hipError_t launch_fc_decode(const FcArgs& a, int mode, bool fc1, int max_tiles, hipStream_t s);

// Single-launch decode (FC1 + SwiGLU + h quantisation, then FC2) in one
// persistent kernel.  Each expert tile's FC1 and FC2 items run on one XCD
// (tile t on XCD t % nx), taken from that XCD's queue in order (every FC1
// item before any FC2 item), so h passes from FC1 to FC2 through the XCD's
// own L2: an FC1 item waits for its stores and bumps done[t]; an FC2 item
// waits until done[t] counts every FC1 row block of its tile, then drops its
// CU's L1 lines.  queue [nx] and done [max_tiles] are zeroed by the route
// launch (which also clears *err); err counts waits that exceeded their
// time limit (the kernel then finishes with wrong results instead of
// hanging).
struct DecodeSync {
  int32_t* queue;
  int32_t* done;
  int32_t* err;
  int nx;            // XCDs (workgroups read their XCD id from the hardware)
  int nblk1, nblk2;  // FC1 / FC2 row blocks per tile
};
hipError_t launch_fc_decode_fused(const FcArgs& a1, const FcArgs& a2, int mode, const DecodeSync& y,
                                  hipStream_t s);
// words of the DecodeSync queue + done counters for max_tiles tiles
inline int decode_sync_words(int max_tiles) { return 8 + max_tiles; }
// XCDs of the current device (32 CUs each on MI355X), 1..8
int xcd_count();

// Prefill-shaped FP8 x FP4 grouped GEMMs on 128-row expert tiles (direct-
// to-LDS pipelined, 512 weight rows per work item); a4: MXFP4 activations
// (act [rows, K/2], h written as MXFP4).  Needs H % 512 == 0, I % 512 == 0
// and 32-bit row offsets.  prep: weights in the GEMM layout of
// launch_prepare_gemm.
hipError_t launch_fc_gemm_a8(const FcArgs& a, bool fc1, bool a4, bool prep, int max_tiles, hipStream_t s);

// RAW group32 weights [E, N, K/2] + [E, N, K/32] -> the GEMM layout of the
// prefill kernels (moe_fp4_prepare_gemm_weights); N, K multiples of 512,
// N * K / 32 < 2^31.
hipError_t launch_prepare_gemm(const uint8_t* src, const uint8_t* src_sf, uint8_t* dst, uint8_t* dst_sf,
                               int64_t E, int64_t N, int64_t K, bool w13, int w13_order, hipStream_t s);

// Group16 weights (E2M1 + E4M3 [E, N, K/16] + global scale gs [E] or null)
// -> the same GEMM layout with group32 UE8M0 scales, gs folded in
// (moe_fp4_prepare_gemm_weights_g16): bit-identical to launch_requant_g16_g32
// followed by launch_prepare_gemm.  N, K multiples of 512, N * K / 32 < 2^31.
hipError_t launch_requant_prepare_gemm(const uint8_t* src, const uint8_t* src_sf, const float* gs, uint8_t* dst,
                                       uint8_t* dst_sf, int64_t E, int64_t N, int64_t K, bool w13, int w13_order,
                                       hipStream_t s);

// out[t, :] = sum_j w[t, j] * y[slot_of[t*k + j], :]  (f32, or rounded to bf16)
hipError_t launch_combine(const float* y, const int32_t* slot_of, const float* topk_w, int T,
                          int k, int H, void* out, bool out_f32, hipStream_t s);

// Register-only loop of the block-scaled MFMA (FP4 x FP8, or FP4 x FP4 with
// a4): blocks x 4 waves x iters x 32 instructions of 2*16*16*128 flops.
hipError_t launch_mfma_peak(bool a4, int iters, int blocks, float* sink, hipStream_t s);

hipError_t launch_requant_g16_g32(const uint8_t* src, const uint8_t* src_sf, const float* gs,
                                  uint8_t* dst, uint8_t* dst_sf, int64_t E, int64_t N, int64_t K,
                                  hipStream_t s);

}  // namespace moefp4
