// A projection over block-scaled FP4 weights with low-rank adapters of many
// requests beside it: y[t] = W x[t] + s_l B_l (A_l x[t]), l = the token's
// adapter (none for ids outside [0, L)).
//
//  1. project_prep: x as the products read it, and for few tokens the low-rank
//     activations u = s_l A_l x (one workgroup per token and 4 ranks).
//     group16 weights multiply in fp16, x as fp16 * 2**-p (exact down to 2**-24
//     of the row's maximum); group32 weights in bfloat16, x as it is.
//     (More tokens: project_shrink computes u with matrix instructions.)
//  2. up to 64 tokens, project_few: the FP4 stream bounds it (an N x K matrix
//     is read once for N K / 2 bytes).  A workgroup owns 16 output rows, its 8
//     waves an eighth of K each; the weights come as whole 128-byte lines into
//     registers, all requested before the first is used.
//     more, project_gemm: matrix instructions bound it.  128 rows x 128 tokens
//     per workgroup; the weights are decoded once per workgroup into LDS,
//     beside x's tile, double-buffered.
//  u stays FP32 up to the product with B: added in FP32 (few), or split into a
//  high and a low bfloat16 (16 bits) for the matrix instructions (gemm).
//  An adapter's product is added to its own tokens only (not multiplied by
//  zero elsewhere), so that its infinities or NaN stay with them.
#include "common.h"
#include "kernels.h"

#include <type_traits>

namespace moefp4 {

namespace {

__device__ __forceinline__ uint32_t bf16_bits(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

// ---------------------------------------------------------------------------
// 1. preparation

// Element k (a multiple of 8) of token t in the order project_few's lanes
// read: [16-token group][256-element chunk][j][q][token][8] for k % 256 =
// 64 q + 8 j + (0 .. 7).
__device__ __forceinline__ size_t frag_at(int t, int k, int K) {
  const int c = k >> 8, q = (k >> 6) & 3, j = (k >> 3) & 7;
  return ((((size_t)(t >> 4) * (K >> 8) + c) * 8 + j) * 64 + q * 16 + (t & 15)) * 8;
}

// One token's row by 256 threads.  F16: to fp16 * 2**-p with *scale = 2**p;
// FRAG: in fragment order, else in place order.
template <bool F16, bool FRAG>
__device__ __forceinline__ void prep_row(const ProjectArgs& a, int t, uint32_t* s_max) {
  const int tid = threadIdx.x, K = a.K;
  const uint16_t* row = a.x + (size_t)t * K;
  float inv = 1.0f;
  if (F16) {
    uint32_t m = 0;
    for (int i = tid * 8; i < K; i += 2048) {
      const uint4 v = *reinterpret_cast<const uint4*>(row + i);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t lo = (w[j] & 0x7FFFu) << 16, hi = w[j] & 0x7FFF0000u;
        m = lo > m ? lo : m;
        m = hi > m ? hi : m;
      }
    }
    for (int d = 32; d >= 1; d >>= 1) {
      const uint32_t y = __shfl_xor(m, d, 64);
      m = y > m ? y : m;
    }
    if ((tid & 63) == 0) s_max[tid >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; ++w) m = s_max[w] > m ? s_max[w] : m;
    int p = m ? (int)(m >> 23) - 127 - 14 : 0;
    p = p < -110 ? -110 : p;
    inv = __builtin_ldexpf(1.0f, -p);
    if (tid == 0) a.xs[t] = __builtin_ldexpf(1.0f, p);
  }
  for (int i = tid * 8; i < K; i += 2048) {
    const uint4 v = *reinterpret_cast<const uint4*>(row + i);
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if (F16) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const _Float16 lo = (_Float16)(bf16_to_f32(w[j] & 0xFFFFu) * inv);
        const _Float16 hi = (_Float16)(bf16_to_f32(w[j] >> 16) * inv);
        w[j] = (uint32_t)__builtin_bit_cast(uint16_t, lo) | ((uint32_t)__builtin_bit_cast(uint16_t, hi) << 16);
      }
    }
    const size_t at = FRAG ? frag_at(t, i, K) : (size_t)t * K + i;
    *reinterpret_cast<uint4*>(a.x16 + at) = uint4{w[0], w[1], w[2], w[3]};
  }
}

constexpr int kShrinkRanks = 4;  // ranks per workgroup of the dot form

// u[t][r0 .. r0 + 4) = s_l A_l x[t] by 256 threads.
__device__ __forceinline__ void shrink_dot(const ProjectArgs& a, int t, int r0, float* s_red) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, K = a.K;
  const int l = a.id[t];
  if ((unsigned)l >= (unsigned)a.L) return;
  const uint16_t* row = a.x + (size_t)t * K;
  const uint16_t* A = a.a + ((size_t)l * a.R + r0) * K;
  float acc[kShrinkRanks] = {};
  for (int k = tid * 8; k < K; k += 2048) {
    const uint4 xv = *reinterpret_cast<const uint4*>(row + k);
    uint4 av[kShrinkRanks];
#pragma unroll
    for (int r = 0; r < kShrinkRanks; ++r) av[r] = *reinterpret_cast<const uint4*>(A + (size_t)r * K + k);
    const uint32_t x[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
    for (int r = 0; r < kShrinkRanks; ++r) {
      const uint32_t w[4] = {av[r].x, av[r].y, av[r].z, av[r].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[r] = __builtin_fmaf(u2f(x[i] << 16), u2f(w[i] << 16), acc[r]);
        acc[r] = __builtin_fmaf(u2f(x[i] & 0xFFFF0000u), u2f(w[i] & 0xFFFF0000u), acc[r]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kShrinkRanks; ++r) {
    for (int d = 32; d >= 1; d >>= 1) acc[r] += __shfl_xor(acc[r], d, 64);
    if (lane == 0) s_red[wave * kShrinkRanks + r] = acc[r];
  }
  __syncthreads();
  if (tid < kShrinkRanks)
    a.u[(size_t)t * a.R + r0 + tid] = a.scale[l] * ((s_red[tid] + s_red[kShrinkRanks + tid]) +
                                                    (s_red[2 * kShrinkRanks + tid] + s_red[3 * kShrinkRanks + tid]));
}

// Workgroups [0, prep): a token's row each; then (shrink) one per token and
// 4 ranks.
template <bool F16, bool FRAG>
__global__ __launch_bounds__(256) void project_prep_kernel(ProjectArgs a, int prep) {
  __shared__ uint32_t s_max[4];
  __shared__ float s_red[4 * kShrinkRanks];
  const int b = blockIdx.x;
  if (b < prep) {
    prep_row<F16, FRAG>(a, b, s_max);
  } else {
    const int nr = a.R / kShrinkRanks, i = b - prep;
    shrink_dot(a, i / nr, (i % nr) * kShrinkRanks, s_red);
  }
}

// u of many tokens with matrix instructions: 16 tokens per workgroup, K split
// over its 4 waves, every adapter that occurs among the 16 in turn (runs of one
// request's tokens: one or two), 16 ranks at a time.
__global__ __launch_bounds__(256) void project_shrink_kernel(ProjectArgs a) {
  __shared__ v4f s_part[4][8][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, q = lane >> 4, K = a.K, R = a.R;
  const int t = blockIdx.x * 16 + r16;
  const int tc = t < a.T ? t : a.T - 1;
  const int id = t < a.T ? a.id[t] : -1;
  uint64_t left = __ballot((unsigned)id < (unsigned)a.L && q == 0);
  const uint16_t* xr = a.x + (size_t)tc * K + 8 * q;
  const int k0 = wave * (K >> 2), k1 = k0 + (K >> 2);  // (K is a multiple of 256)
  const int nt = (R + 15) >> 4;
  while (left) {
    const int l = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
    left &= ~__ballot(id == l);
    v4f acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = v4f{0.f, 0.f, 0.f, 0.f};
    const uint16_t* A = a.a + (size_t)l * R * K + 8 * q;
    for (int k = k0; k < k1; k += 64) {
      v8bf B[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) B[s] = *reinterpret_cast<const v8bf*>(xr + k + 32 * s);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (i < nt) {
          const int r = min(16 * i + r16, R - 1);  // (ranks past R are not stored)
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const v8bf w = *reinterpret_cast<const v8bf*>(A + (size_t)r * K + k + 32 * s);
            acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, B[s], acc[i], 0, 0, 0);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < nt) s_part[wave][i][lane] = acc[i];
    __syncthreads();
    // lane: ranks 16 i + 4 q .. + 3, token r16; the waves share the rank tiles
    for (int i = wave; i < nt; i += 4) {
      const v4f s = (s_part[0][i][lane] + s_part[1][i][lane]) + (s_part[2][i][lane] + s_part[3][i][lane]);
      const int r = 16 * i + 4 * q;
      if (id == l && r < R)
        *reinterpret_cast<v4f*>(a.u + (size_t)t * R + r) = s * a.scale[l];
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// 2a. few tokens

// 16 rows x 256 K of weights: instruction j holds rows 8 j + lane / 8, bytes
// 16 (lane & 7) of the chunk's 128; s: the scales of row r16, K [64 q, + 64).
struct WTile {
  u32x4 c[2];
  uint32_t s;
};

// NG: 16-token groups; NC: chunks of K in flight per wave.
template <int MODE, int NG, int NC>
__global__ __launch_bounds__(512, 2) void project_few_kernel(ProjectArgs a) {
  __shared__ float4 s_red[8][NG][64];
  __shared__ __attribute__((aligned(16))) uint8_t s_turn[8][2048];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, q = lane >> 4, K = a.K;
  const int n0 = blockIdx.x * 16, nch = K >> 8;
  const uint32_t rowb = K >> 1, rows = MODE == 0 ? K >> 4 : K >> 5;
  const uint8_t* codes = a.w + (size_t)n0 * rowb;
  const uint8_t* sf = a.w_sf + (size_t)n0 * rows;
  const uint32_t o0 = (lane >> 3) * rowb + 16 * (lane & 7), step8 = 8 * rowb;
  const uint32_t f0 = r16 * rows + (MODE == 0 ? 4 * q : 2 * q);
  // (no load is conditional: chunks past the end repeat the last one, and
  // their products are not added)
  auto load = [&](int c, WTile& w) __attribute__((always_inline)) {
    c = c < nch ? c : nch - 1;
    w.c[0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(codes + o0 + c * 128));
    w.c[1] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(codes + o0 + step8 + c * 128));
    if (MODE == 0) w.s = *reinterpret_cast<const uint32_t*>(sf + f0 + c * 16);
    else w.s = *reinterpret_cast<const uint16_t*>(sf + f0 + c * 8);
  };
  WTile w[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) load(wave + 8 * i, w[i]);

  // the adapters' part of output (row rn, token rt + 32 p), while the weights come
  const int rn = tid & 15, rt = tid >> 4;
  constexpr int NP = (NG + 1) / 2;
  float lora[NP];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    lora[p] = 0.0f;
    const int t = rt + 32 * p;
    if (a.L > 0 && t < a.T) {
      const int l = a.id[t];
      if ((unsigned)l < (unsigned)a.L) {
        const uint16_t* B = a.b + ((size_t)l * a.N + n0 + rn) * a.R;
        const float* u = a.u + (size_t)t * a.R;
        for (int r = 0; r < a.R; r += 8) {
          const uint4 v = *reinterpret_cast<const uint4*>(B + r);
          const float4 ua = *reinterpret_cast<const float4*>(u + r), ub = *reinterpret_cast<const float4*>(u + r + 4);
          float s = lora[p];
          s = __builtin_fmaf(u2f(v.x << 16), ua.x, s);
          s = __builtin_fmaf(u2f(v.x & 0xFFFF0000u), ua.y, s);
          s = __builtin_fmaf(u2f(v.y << 16), ua.z, s);
          s = __builtin_fmaf(u2f(v.y & 0xFFFF0000u), ua.w, s);
          s = __builtin_fmaf(u2f(v.z << 16), ub.x, s);
          s = __builtin_fmaf(u2f(v.z & 0xFFFF0000u), ub.y, s);
          s = __builtin_fmaf(u2f(v.w << 16), ub.z, s);
          s = __builtin_fmaf(u2f(v.w & 0xFFFF0000u), ub.w, s);
          lora[p] = s;
        }
      }
    }
  }

  v4f acc[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) acc[g] = v4f{0.f, 0.f, 0.f, 0.f};
  uint8_t* turn = s_turn[wave];
  const int wr = lane >> 3, seg = lane & 7;
  const uint32_t tw0 = wr * 128 + 16 * (seg ^ (wr >> 1)), tw1 = (wr + 8) * 128 + 16 * (seg ^ ((wr + 8) >> 1));
  const uint32_t tr0 = r16 * 128 + 16 * ((2 * q) ^ (r16 >> 1)), tr1 = r16 * 128 + 16 * ((2 * q + 1) ^ (r16 >> 1));
  const u32x4* xf = reinterpret_cast<const u32x4*>(a.x16) + lane;
  for (int c0 = 0; c0 < nch; c0 += 8 * NC) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = c0 + wave + 8 * i;
      asm volatile("" : "+v"(w[i].c[0]), "+v"(w[i].c[1]), "+v"(w[i].s));
      // the codes turned into operand order through the wave's own LDS
      *reinterpret_cast<u32x4*>(turn + tw0) = w[i].c[0];
      *reinterpret_cast<u32x4*>(turn + tw1) = w[i].c[1];
      const u32x4 c4[2] = {*reinterpret_cast<const u32x4*>(turn + tr0), *reinterpret_cast<const u32x4*>(turn + tr1)};
      const uint32_t sc = w[i].s;
      if (c < nch) {
        u32x4 A[8];
        if constexpr (MODE == 0) {
          const v2h lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(sc, 1.0f, false);
          const v2h hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(sc, 1.0f, true);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const _Float16 s = j < 2 ? lo[0] : j < 4 ? lo[1] : j < 6 ? hi[0] : hi[1];
            A[j] = __builtin_bit_cast(u32x4, dq8_f16(c4[j >> 2][j & 3], v2h{s, s}));
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            A[j] = __builtin_bit_cast(u32x4, dq8_bf16(c4[j >> 2][j & 3], ue8m0_to_f32((sc >> (8 * (j >> 2))) & 0xFFu)));
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const u32x4* xc = xf + ((size_t)g * nch + c) * 512;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const u32x4 b = xc[64 * j];
            if constexpr (MODE == 0)
              acc[g] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, A[j]), __builtin_bit_cast(v8h, b),
                                                              acc[g], 0, 0, 0);
            else
              acc[g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, A[j]),
                                                               __builtin_bit_cast(v8bf, b), acc[g], 0, 0, 0);
          }
        }
      }
      if (c0 + 8 * NC < nch) load(c + 8 * NC, w[i]);
    }
  }
#pragma unroll
  for (int g = 0; g < NG; ++g) s_red[wave][g][lane] = float4{acc[g][0], acc[g][1], acc[g][2], acc[g][3]};
  __syncthreads();
  const float gs = a.w_gs ? a.w_gs[0] : 1.0f;
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int t = rt + 32 * p;
    if (t >= a.T) continue;
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < 8; ++v)
      s += reinterpret_cast<const float*>(&s_red[v][t >> 4][(t & 15) + 16 * (rn >> 2)])[rn & 3];
    s = __builtin_fmaf(s, gs * (MODE == 0 ? a.xs[t] : 1.0f), lora[p]);
    const size_t at = (size_t)t * a.N + n0 + rn;
    if (a.out_f32) static_cast<float*>(a.out)[at] = s;
    else static_cast<uint16_t*>(a.out)[at] = (uint16_t)bf16_bits(s);
  }
}

// ---------------------------------------------------------------------------
// 2b. many tokens

constexpr int kTile = 128;  // weight rows and tokens per workgroup
constexpr int kGK = 64;     // K elements per stage

// LDS rows of 128 bytes; 16-byte segment s of row r sits at s ^ ((r >> 1) & 7),
// so that the 16 rows a lane group reads touch all 64 banks.
__device__ __forceinline__ int pswz(int r) { return (r >> 1) & 7; }

template <int MODE>
__global__ __launch_bounds__(256, 2) void project_gemm_kernel(ProjectArgs a, int row_tiles) {
  // x and the decoded weights of a stage, two stages
  __shared__ __attribute__((aligned(16))) uint8_t s_x0[kTile * 128], s_x1[kTile * 128];
  __shared__ __attribute__((aligned(16))) uint8_t s_w[2][kTile * 128];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, q = lane >> 4, K = a.K, N = a.N, T = a.T;
  const int n0 = (blockIdx.x % row_tiles) * kTile, t0 = (blockIdx.x / row_tiles) * kTile;
  const int wn = (wave & 1) * 64, wt = (wave >> 1) * 64;
  const uint16_t* xsrc = MODE == 0 ? a.x16 : a.x;

  // x rows by direct loads to LDS, eight whole 128-byte rows per instruction
  // (rows past T repeat the last one: their results are not stored)
  auto stage_x = [&](int s, uint8_t* lds) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 32 * wave + 8 * i + (lane >> 3);
      const int t = min(t0 + r, T - 1);
      const uint16_t* src = xsrc + (size_t)t * K + s * kGK + 8 * ((lane & 7) ^ pswz(r));
      __builtin_amdgcn_global_load_lds(src, lds + (32 * wave + 8 * i) * 128, 16, 0, 0);
    }
  };
  // weights: thread = (row, half); of every two stages (64 bytes of a row) its
  // 16 bytes of each stage's 32, and the scales of their K
  const int wrow = tid >> 1, half = tid & 1;
  const int nrow = min(n0 + wrow, N - 1);
  const uint8_t* wsrc = a.w + (size_t)nrow * (K >> 1) + 16 * half;
  const uint8_t* ssrc = a.w_sf + (size_t)nrow * (MODE == 0 ? K >> 4 : K >> 5);
  struct Raw { u32x4 c[2]; uint64_t s; };
  auto load_w = [&](int s2, Raw& r) __attribute__((always_inline)) {  // stages 2 s2, 2 s2 + 1
    r.c[0] = *reinterpret_cast<const u32x4*>(wsrc + s2 * 64);
    r.c[1] = *reinterpret_cast<const u32x4*>(wsrc + s2 * 64 + 32);
    if (MODE == 0) r.s = *reinterpret_cast<const uint64_t*>(ssrc + s2 * 8);
    else r.s = *reinterpret_cast<const uint32_t*>(ssrc + s2 * 4);
  };
  auto decode = [&](const Raw& r, int par, uint8_t* lds) __attribute__((always_inline)) {
    const u32x4 c = r.c[par];
    uint8_t* row = lds + wrow * 128;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u32x4 v;
      if constexpr (MODE == 0) {
        // K 32 half + 8 j of the stage: scale byte 4 par + 2 half + j / 2
        const uint32_t b = (uint32_t)(r.s >> (8 * (4 * par + 2 * half + (j >> 1)))) & 0xFFu;
        v = __builtin_bit_cast(u32x4, dq8_f16(c[j], e4m3_to_h2(b)));
      } else {
        const uint32_t b = (uint32_t)(r.s >> (8 * (2 * par + half))) & 0xFFu;
        v = __builtin_bit_cast(u32x4, dq8_bf16(c[j], ue8m0_to_f32(b)));
      }
      *reinterpret_cast<u32x4*>(row + 16 * ((4 * half + j) ^ pswz(wrow))) = v;
    }
  };

  v4f acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](const uint8_t* sx, const uint8_t* sw) __attribute__((always_inline)) {
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      u32x4 B[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = wt + 16 * j + r16;
        B[j] = *reinterpret_cast<const u32x4*>(sx + r * 128 + 16 * ((4 * ks + q) ^ pswz(r)));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = wn + 16 * i + r16;
        const u32x4 A = *reinterpret_cast<const u32x4*>(sw + r * 128 + 16 * ((4 * ks + q) ^ pswz(r)));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (MODE == 0)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, A), __builtin_bit_cast(v8h, B[j]),
                                                               acc[i][j], 0, 0, 0);
          else
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, A),
                                                                __builtin_bit_cast(v8bf, B[j]), acc[i][j], 0, 0, 0);
        }
      }
    }
  };

  const int n2 = K / (2 * kGK);  // pairs of stages (K is a multiple of 256)
  Raw cur, nxt;
  stage_x(0, s_x0);
  load_w(0, cur);
  decode(cur, 0, s_w[0]);
  // every wave waits for its own direct loads before the barrier that hands
  // them to the others (the barrier itself does not: the compiler waits where
  // this wave reads LDS, behind it)
  auto handover = [&]() __attribute__((always_inline)) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
  };
  for (int p = 0; p < n2; ++p) {
    handover();  // stage 2 p is in LDS; every wave is past stage 2 p - 1
    stage_x(2 * p + 1, s_x1);
    load_w(min(p + 1, n2 - 1), nxt);
    decode(cur, 1, s_w[1]);
    multiply(s_x0, s_w[0]);
    handover();  // stage 2 p + 1 is in LDS; every wave is past stage 2 p
    if (p + 1 < n2) {
      stage_x(2 * p + 2, s_x0);
      decode(nxt, 0, s_w[0]);
    }
    multiply(s_x1, s_w[1]);
    cur = nxt;
  }

  // scales, then the adapters that occur among each 16 tokens, then the output
  const float gs = a.w_gs ? a.w_gs[0] : 1.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int t = t0 + wt + 16 * j + r16;
    const float cs = gs * (MODE == 0 && t < T ? a.xs[t] : 1.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i][j] *= cs;
    if (a.L > 0) {
      const int id = t < T ? a.id[t] : -1;
      uint64_t left = __ballot((unsigned)id < (unsigned)a.L && q == 0);
      while (left) {
        const int l = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        const bool mine = id == l;
        left &= ~__ballot(mine);
        v4f add[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) add[i] = v4f{0.f, 0.f, 0.f, 0.f};
        for (int r0 = 0; r0 < a.R; r0 += 32) {
          const int r = r0 + 8 * q;
          v8bf hi = {}, lo = {};
          if (mine && r < a.R) {
            const float* u = a.u + (size_t)t * a.R + r;
#pragma unroll
            for (int v = 0; v < 8; ++v) {
              hi[v] = (__bf16)u[v];
              const float rest = u[v] - (float)hi[v];
              lo[v] = __builtin_isfinite(rest) ? (__bf16)rest : (__bf16)0.0f;
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int n = min(n0 + wn + 16 * i + r16, N - 1);
            v8bf B = {};
            if (r < a.R) B = *reinterpret_cast<const v8bf*>(a.b + ((size_t)l * N + n) * a.R + r);
            add[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(B, lo, add[i], 0, 0, 0);
            add[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(B, hi, add[i], 0, 0, 0);
          }
        }
        if (mine) {
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[i][j] += add[i];
        }
      }
    }
    if (t < T) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = n0 + wn + 16 * i + 4 * q;
        if (n < N) {  // (N is a multiple of 16)
          const size_t at = (size_t)t * N + n;
          const v4f o = acc[i][j];
          if (a.out_f32)
            *reinterpret_cast<v4f*>(static_cast<float*>(a.out) + at) = o;
          else
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
                uint2{bf16_bits(o[0]) | (bf16_bits(o[1]) << 16), bf16_bits(o[2]) | (bf16_bits(o[3]) << 16)};
        }
      }
    }
  }
}

template <int MODE, int NG>
void launch_few_tokens(const ProjectArgs& a, hipStream_t s) {
  const dim3 grid(a.N / 16), block(512);
  if (a.K <= 2048) hipLaunchKernelGGL((project_few_kernel<MODE, NG, 1>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((project_few_kernel<MODE, NG, 3>), grid, block, 0, s, a);
}

template <int MODE>
hipError_t launch_mode(const ProjectArgs& a, hipStream_t s) {
  const bool few = a.T <= kProjectFew;
  const bool dot = a.L > 0 && a.T <= kProjectDot;
  const int prep = few || MODE == 0 ? a.T : 0;
  const int blocks = prep + (dot ? a.T * (a.R / kShrinkRanks) : 0);
  if (blocks > 0) {
    if (few) hipLaunchKernelGGL((project_prep_kernel<MODE == 0, true>), dim3(blocks), dim3(256), 0, s, a, prep);
    else hipLaunchKernelGGL((project_prep_kernel<MODE == 0, false>), dim3(blocks), dim3(256), 0, s, a, prep);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  if (a.L > 0 && !dot) {
    hipLaunchKernelGGL(project_shrink_kernel, dim3((a.T + 15) / 16), dim3(256), 0, s, a);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  if (few) {
    if (a.T <= 16) launch_few_tokens<MODE, 1>(a, s);
    else if (a.T <= 32) launch_few_tokens<MODE, 2>(a, s);
    else launch_few_tokens<MODE, 4>(a, s);
  } else {
    const int rt = (a.N + kTile - 1) / kTile, tt = (a.T + kTile - 1) / kTile;
    hipLaunchKernelGGL(project_gemm_kernel<MODE>, dim3(rt * tt), dim3(256), 0, s, a, rt);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_project(const ProjectArgs& a, hipStream_t s) {
  return a.g16 ? launch_mode<0>(a, s) : launch_mode<1>(a, s);
}

}  // namespace moefp4
