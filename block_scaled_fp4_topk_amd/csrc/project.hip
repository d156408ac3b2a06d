// A projection over block-scaled FP4 weights with low-rank adapters of many
// requests beside it: y[t] = W x[t] + s_l B_l (A_l x[t]), l = the token's
// adapter (none for ids outside [0, L)).
//
//  1. up to 128 tokens, project_prep: x in the order project_few's lanes read,
//     for group16 weights as fp16 * 2**-p (exact down to 2**-24 of the row's
//     maximum), for group32 as it is, and the low-rank activations u =
//     s_l A_l x (one workgroup per token and 4 ranks).  (More tokens: grouped
//     by adapter as the router groups by expert, and project_shrink computes u
//     with matrix instructions.)
//  2. up to 128 tokens, project_few: the FP4 stream bounds it (an N x K matrix
//     is read once for N K / 2 bytes), and the reading of x by every workgroup.
//     A workgroup owns 16 or 32 output rows, its 8 waves an eighth of K each;
//     the weights come as whole 128-byte lines into registers, the wave's first
//     one to three chunks requested before any is used.
//     more, project_gemm: matrix instructions bound it, and the LDS that feeds
//     them.  256 rows x 256 tokens per workgroup where that fills the chip;
//     the weights are decoded once per workgroup into LDS, beside x's tile,
//     double-buffered.  Both formats multiply in bfloat16 there, x as it is (an
//     E2M1 code times an E4M3 scale has 6 significant bits: exact).
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

// Eight bfloat16 values times eight floats.
__device__ __forceinline__ float dot8(const uint4& v, const v4f& a, const v4f& b) {
  float s = u2f(v.x << 16) * a[0];
  s = __builtin_fmaf(u2f(v.x & 0xFFFF0000u), a[1], s);
  s = __builtin_fmaf(u2f(v.y << 16), a[2], s);
  s = __builtin_fmaf(u2f(v.y & 0xFFFF0000u), a[3], s);
  s = __builtin_fmaf(u2f(v.z << 16), b[0], s);
  s = __builtin_fmaf(u2f(v.z & 0xFFFF0000u), b[1], s);
  s = __builtin_fmaf(u2f(v.w << 16), b[2], s);
  return __builtin_fmaf(u2f(v.w & 0xFFFF0000u), b[3], s);
}

// ---------------------------------------------------------------------------
// 1. preparation

// Element k (a multiple of 8) of token t in the order project_few's lanes
// read: [16-token group][256-element chunk][j][q][token][8] for k % 256 =
// 64 q + 8 j + (0 .. 7).
__device__ __forceinline__ size_t frag_at(int t, int k, int K) {
  const int c = k >> 8, q = (k >> 6) & 3, j = (k >> 3) & 7;
  return ((((size_t)(t >> 4) * (K >> 8) + c) * 8 + j) * 64 + q * 16 + (t & 15)) * 8;
}

// One token's row, in that order, by 256 threads.  F16: as fp16 * 2**-p, with
// xs = 2**p.
template <bool F16>
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
    *reinterpret_cast<uint4*>(a.x16 + frag_at(t, i, K)) = uint4{w[0], w[1], w[2], w[3]};
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
template <bool F16>
__global__ __launch_bounds__(256) void project_prep_kernel(ProjectArgs a, int prep) {
  __shared__ uint32_t s_max[4];
  __shared__ float s_red[4 * kShrinkRanks];
  const int b = blockIdx.x;
  if (b < prep) {
    prep_row<F16>(a, b, s_max);
  } else {
    const int nr = a.R / kShrinkRanks, i = b - prep;
    shrink_dot(a, i / nr, (i % nr) * kShrinkRanks, s_red);
  }
}

// The adapters to group the tokens by: L for tokens without one, which come
// last.
__global__ __launch_bounds__(256) void project_ids_kernel(ProjectArgs a) {
  const int t = blockIdx.x * 256 + threadIdx.x;
  if (t < a.T) a.ids[t] = (unsigned)a.id[t] < (unsigned)a.L ? a.id[t] : a.L;
}

// u of many tokens with matrix instructions: the tokens grouped by adapter (the
// router's stable grouping), a tile of up to 32 tokens of one adapter per
// workgroup, K split over its 8 waves and, where there are few tiles, over
// a.ku workgroups (a CU draws about 30 bytes
// per ns here, so it takes all of them: 512 tokens, K = 6144, rank 64 39 us by
// 24 workgroups, 11 us by 192); NT: tiles of 16 ranks.
template <int NT>
__global__ __launch_bounds__(512, NT >= 8 ? 2 : 4) void project_shrink_kernel(ProjectArgs a) {
  __shared__ v4f s_part[4][NT][2][64];
  if ((int)blockIdx.x >= a.route.ntiles[0]) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, q = lane >> 4, K = a.K, R = a.R;
  const int l = a.route.tiles[2 * blockIdx.x], m0 = a.route.tiles[2 * blockIdx.x + 1];
  if (l >= a.L) return;
  const int ne = a.route.counts[l], oe = a.route.offsets[l];
  int tok[2];
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const int m = m0 + 16 * g + r16;
    tok[g] = a.route.sorted_assign[oe + (m < ne ? m : m0)];  // (rows past the last: not stored)
  }
  const uint16_t* A = a.a + (size_t)l * R * K + 8 * q;
  const uint16_t* xr[2] = {a.x + (size_t)tok[0] * K + 8 * q, a.x + (size_t)tok[1] * K + 8 * q};
  const int per = K / (8 * a.ku), k0 = (blockIdx.y * 8 + wave) * per;  // (whole steps of 32: ku divides K / 256)
  const int n = per >> 5;
  v4f acc[NT][2];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i][0] = acc[i][1] = v4f{0.f, 0.f, 0.f, 0.f};
  const uint16_t* ar[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) ar[i] = A + (size_t)min(16 * i + r16, R - 1) * K;  // (ranks past R: not stored)
  constexpr int PD = NT >= 8 ? 2 : NT >= 4 ? 3 : 4;  // steps in flight
  v8bf bx[PD][2], ba[PD][NT];
  auto load = [&](int s, int slot) __attribute__((always_inline)) {
    const int k = k0 + 32 * min(s, n - 1);
    bx[slot][0] = *reinterpret_cast<const v8bf*>(xr[0] + k);
    bx[slot][1] = *reinterpret_cast<const v8bf*>(xr[1] + k);
#pragma unroll
    for (int i = 0; i < NT; ++i) ba[slot][i] = *reinterpret_cast<const v8bf*>(ar[i] + k);
  };
#pragma unroll
  for (int s = 0; s < PD; ++s) load(s, s);
  for (int s = 0; s < n; s += PD) {
#pragma unroll
    for (int p = 0; p < PD; ++p) {
      if (s + p < n) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          acc[i][0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ba[p][i], bx[p][0], acc[i][0], 0, 0, 0);
          acc[i][1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ba[p][i], bx[p][1], acc[i][1], 0, 0, 0);
        }
      }
      load(s + p + PD, p);
    }
  }
  // the waves' parts: 4 .. 7 hand theirs to 0 .. 3, whose sums meet in LDS
  if (wave >= 4) {
#pragma unroll
    for (int i = 0; i < NT; ++i) s_part[wave - 4][i][0][lane] = acc[i][0], s_part[wave - 4][i][1][lane] = acc[i][1];
  }
  __syncthreads();
  if (wave < 4) {
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int g = 0; g < 2; ++g) s_part[wave][i][g][lane] = acc[i][g] + s_part[wave][i][g][lane];
  }
  __syncthreads();
  // lane: ranks 16 i + 4 q .. + 3, token r16 of group g
  const float sl = a.scale[l];
  for (int j = wave; j < 2 * NT; j += 8) {
    const int i = j >> 1, g = j & 1;
    const v4f v = (s_part[0][i][g][lane] + s_part[1][i][g][lane]) + (s_part[2][i][g][lane] + s_part[3][i][g][lane]);
    const int r = 16 * i + 4 * q;
    if (m0 + 16 * g + r16 < ne && r < R) *reinterpret_cast<v4f*>(a.u + ((size_t)blockIdx.y * a.T + tok[g]) * R + r) = v * sl;
  }
}

// u = the sum of its parts, in order (parts 1 .. ku - 1 added to the first).
__global__ __launch_bounds__(256) void project_u_sum_kernel(ProjectArgs a) {
  const long long n = (long long)a.T * a.R, i = ((long long)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  v4f s = *reinterpret_cast<const v4f*>(a.u + i);
  for (int z = 1; z < a.ku; ++z) s += *reinterpret_cast<const v4f*>(a.u + z * n + i);
  *reinterpret_cast<v4f*>(a.u + i) = s;
}

// ---------------------------------------------------------------------------
// 2a. few tokens

// 16 rows x 256 K of weights: instruction j holds rows 8 j + lane / 8, bytes
// 16 (lane & 7) of the chunk's 128; s: the scales of row r16, K [64 q, + 64).
struct WTile {
  u32x4 c[2];
  uint32_t s;
};

// NG: 16-token groups; NC: chunks of K in flight per wave; NR: 16-row tiles of a
// workgroup.
template <int MODE, int NG, int NC, int NR>
__global__ __launch_bounds__(512, 2) void project_few_kernel(ProjectArgs a) {
  constexpr int GP = NG < 4 ? NG : 4;  // groups summed over the waves at a time
  constexpr int ROWS = 16 * NR, TS = 512 / ROWS;  // rows, and tokens that the threads store at a time
  __shared__ float4 s_red[8][GP][NR][64];
  __shared__ __attribute__((aligned(16))) uint8_t s_turn[8][2048];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, q = lane >> 4, K = a.K;
  const int n0 = blockIdx.x * ROWS, nch = K >> 8;
  const uint32_t rowb = K >> 1, rows = MODE == 0 ? K >> 4 : K >> 5;
  const uint32_t o0 = (lane >> 3) * rowb + 16 * (lane & 7), step8 = 8 * rowb;
  const uint32_t f0 = r16 * rows + (MODE == 0 ? 4 * q : 2 * q);
  // (no load is conditional: chunks past the end repeat the last one, and
  // their products are not added; a tile past the last row repeats the first)
  auto load = [&](int c, WTile (&w)[NR]) __attribute__((always_inline)) {
    c = c < nch ? c : nch - 1;
#pragma unroll
    for (int t = 0; t < NR; ++t) {
      const size_t n = n0 + 16 * t < a.N ? n0 + 16 * t : n0;
      const uint8_t *codes = a.w + n * rowb, *sf = a.w_sf + n * rows;
      w[t].c[0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(codes + o0 + c * 128));
      w[t].c[1] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(codes + o0 + step8 + c * 128));
      if (MODE == 0) w[t].s = *reinterpret_cast<const uint32_t*>(sf + f0 + c * 16);
      else w[t].s = *reinterpret_cast<const uint16_t*>(sf + f0 + c * 8);
    }
  };
  WTile w[NC][NR];
#pragma unroll
  for (int i = 0; i < NC; ++i) load(wave + 8 * i, w[i]);

  // the adapters' part of output (row rn, token rt + TS p): for few groups
  // while the weights come, else behind the products
  const int rn = tid & (ROWS - 1), rt = tid / ROWS;
  constexpr int NP = (16 * NG + TS - 1) / TS;
  auto adapted = [&](int p) __attribute__((always_inline)) {
    float s = 0.0f;
    const int t = rt + TS * p;
    if (a.L > 0 && t < a.T && n0 + rn < a.N) {
      const int l = a.id[t];
      if ((unsigned)l < (unsigned)a.L) {
        const uint16_t* B = a.b + ((size_t)l * a.N + n0 + rn) * a.R;
        const float* u = a.u + (size_t)t * a.R;
        for (int r = 0; r < a.R; r += 8) {
          s += dot8(*reinterpret_cast<const uint4*>(B + r), *reinterpret_cast<const v4f*>(u + r),
                    *reinterpret_cast<const v4f*>(u + r + 4));
        }
      }
    }
    return s;
  };
  float lora[NP];
#pragma unroll
  for (int p = 0; p < NP; ++p) lora[p] = NG <= 4 ? adapted(p) : 0.0f;

  v4f acc[NR][NG];
#pragma unroll
  for (int t = 0; t < NR; ++t)
#pragma unroll
    for (int g = 0; g < NG; ++g) acc[t][g] = v4f{0.f, 0.f, 0.f, 0.f};
  uint8_t* turn = s_turn[wave];
  const int wr = lane >> 3, seg = lane & 7;
  const uint32_t tw0 = wr * 128 + 16 * (seg ^ (wr >> 1)), tw1 = (wr + 8) * 128 + 16 * (seg ^ ((wr + 8) >> 1));
  const uint32_t tr0 = r16 * 128 + 16 * ((2 * q) ^ (r16 >> 1)), tr1 = r16 * 128 + 16 * ((2 * q + 1) ^ (r16 >> 1));
  const u32x4* xf = reinterpret_cast<const u32x4*>(a.x16) + lane;
  u32x4 x_ahead[2][8];
  auto load_x = [&](int g, int c, u32x4 (&b)[8]) __attribute__((always_inline)) {
    const u32x4* xc = xf + ((size_t)g * nch + min(c, nch - 1)) * 512;
#pragma unroll
    for (int j = 0; j < 8; ++j) b[j] = xc[64 * j];
  };
  load_x(0, wave, x_ahead[0]);
  for (int c0 = 0; c0 < nch; c0 += 8 * NC) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = c0 + wave + 8 * i;
      u32x4 A[NR][8];
#pragma unroll
      for (int t = 0; t < NR; ++t) {
        asm volatile("" : "+v"(w[i][t].c[0]), "+v"(w[i][t].c[1]), "+v"(w[i][t].s));
        // the codes turned into operand order through the wave's own LDS
        *reinterpret_cast<u32x4*>(turn + tw0) = w[i][t].c[0];
        *reinterpret_cast<u32x4*>(turn + tw1) = w[i][t].c[1];
        const u32x4 c4[2] = {*reinterpret_cast<const u32x4*>(turn + tr0), *reinterpret_cast<const u32x4*>(turn + tr1)};
        const uint32_t sc = w[i][t].s;
        if constexpr (MODE == 0) {
          const v2h lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(sc, 1.0f, false);
          const v2h hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(sc, 1.0f, true);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const _Float16 s = j < 2 ? lo[0] : j < 4 ? lo[1] : j < 6 ? hi[0] : hi[1];
            A[t][j] = __builtin_bit_cast(u32x4, dq8_f16(c4[j >> 2][j & 3], v2h{s, s}));
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            A[t][j] = __builtin_bit_cast(u32x4, dq8_bf16(c4[j >> 2][j & 3], ue8m0_to_f32((sc >> (8 * (j >> 2))) & 0xFFu)));
        }
      }
      if (c < nch) {
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          u32x4 (&xb)[8] = x_ahead[(i * NG + g) & 1];
          // the next group's (or chunk's) x, while this one multiplies
          if (g + 1 < NG) load_x(g + 1, c, x_ahead[(i * NG + g + 1) & 1]);
          else load_x(0, i + 1 < NC ? c + 8 : c0 + 8 * NC + wave, x_ahead[(i * NG + g + 1) & 1]);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int t = 0; t < NR; ++t) {
              if constexpr (MODE == 0)
                acc[t][g] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, A[t][j]),
                                                                   __builtin_bit_cast(v8h, xb[j]), acc[t][g], 0, 0, 0);
              else
                acc[t][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    __builtin_bit_cast(v8bf, A[t][j]), __builtin_bit_cast(v8bf, xb[j]), acc[t][g], 0, 0, 0);
            }
        }
      }
      if (c0 + 8 * NC < nch) load(c + 8 * NC, w[i]);
    }
    if constexpr ((NC * NG) & 1) {  // the two buffers change places
#pragma unroll
      for (int j = 0; j < 8; ++j) x_ahead[0][j] = x_ahead[1][j];
    }
  }
  const float gs = a.w_gs ? a.w_gs[0] : 1.0f;
#pragma unroll
  for (int g0 = 0; g0 < NG; g0 += GP) {
    if (g0 > 0) __syncthreads();  // (the groups before are summed)
#pragma unroll
    for (int g = 0; g < GP; ++g)
#pragma unroll
      for (int t = 0; t < NR; ++t) {
        const v4f v = acc[t][g0 + g];
        s_red[wave][g][t][lane] = float4{v[0], v[1], v[2], v[3]};
      }
    __syncthreads();
#pragma unroll
    for (int p = 16 * g0 / TS; p < (16 * (g0 + GP) + TS - 1) / TS; ++p) {
      const int t = rt + TS * p;
      if (t >= a.T || n0 + rn >= a.N) continue;
      float s = 0.0f;
#pragma unroll
      for (int v = 0; v < 8; ++v)
        s += reinterpret_cast<const float*>(&s_red[v][(t >> 4) - g0][rn >> 4][(t & 15) + 16 * ((rn & 15) >> 2)])[rn & 3];
      s = __builtin_fmaf(s, gs * (MODE == 0 ? a.xs[t] : 1.0f), NG <= 4 ? lora[p] : adapted(p));
      const size_t at = (size_t)t * a.N + n0 + rn;
      if (a.out_f32) static_cast<float*>(a.out)[at] = s;
      else static_cast<uint16_t*>(a.out)[at] = (uint16_t)bf16_bits(s);
    }
  }
}

// ---------------------------------------------------------------------------
// 2b. many tokens

constexpr int kTile = 128;  // weight rows per workgroup (256 x 256 tiles: 256)
constexpr int kGK = 64;     // K elements per stage

// LDS rows of 128 bytes; 16-byte segment s of row r sits at s ^ ((r >> 1) & 7),
// so that the 16 rows a lane group reads touch all 64 banks.
__device__ __forceinline__ int pswz(int r) { return (r >> 1) & 7; }

// The token at place t of the order that the tiled product takes them in:
// grouped by adapter, where they have been grouped for u, so that a tile's
// tokens share theirs (8192 tokens of 16 adapters of rank 64 in random order,
// N = 4096, K = 6144: 437 us against 716 us).
__device__ __forceinline__ int token_at(const ProjectArgs& a, int t) { return a.order ? a.order[t] : t; }

// The tokens that lane r16 has of each 16 from place t0 on, -1 past the last.
template <int NJ>
__device__ __forceinline__ void tokens_at(const ProjectArgs& a, int t0, int (&tok)[NJ]) {
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int t = t0 + 16 * j + (threadIdx.x & 15);
    tok[j] = t < a.T ? token_at(a, t) : -1;
  }
}

// One wave's 16 NJ tokens x 16 NI rows from n0 on (lane: token r16 of each 16,
// rows 4 q .. + 3 of each 16): the adapters that occur among the tokens added to
// o, one after the other.  u enters as two bfloat16 parts; a token takes its own
// adapter's product and nothing of the others'.  (The high part is the largest
// bfloat16 where rounding would make it infinite: a finite u stays finite, and
// an infinite one is in the low part.)
//
// An infinity of B times u's two parts is NaN where their signs differ or the
// low one is 0, and so is a product past FP32's range.  EXACT: where an
// adapter's sum is NaN it is formed again from parts of one sign (u / 2, the
// high one taken off but for 1/64), which give an infinity's own sign, and NaN
// only where the product is NaN; what is finite counts from the first pass.
template <int NI, int NJ, bool EXACT>
__device__ __forceinline__ void add_adapters(const ProjectArgs& a, v4f (&o)[NI][NJ], const int (&tok)[NJ], int n0) {
  const int lane = threadIdx.x & 63, r16 = lane & 15, q = lane >> 4, N = a.N;
  int id[NJ];
  uint64_t left[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) id[j] = tok[j] >= 0 ? a.id[tok[j]] : -1;
#pragma unroll
  for (int j = 0; j < NJ; ++j) left[j] = __ballot((unsigned)id[j] < (unsigned)a.L && q == 0);
  for (;;) {
    int l = -1;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      if (l < 0 && left[j]) l = __builtin_amdgcn_readlane(id[j], __builtin_ctzll(left[j]));
    if (l < 0) break;
    bool some[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const uint64_t mine = __ballot(id[j] == l);
      some[j] = mine != 0;
      left[j] &= ~mine;
    }
#pragma unroll 1
    for (int pass = 0;; pass = 1) {
      const float whole = pass ? 0.5f : 1.0f, off = pass ? 0x1.F8p-1f : 1.0f;  // (1 - 2^-6)
      v4f add[NI][NJ];
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < NI; ++i) add[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
      for (int r0 = 0; r0 < a.R; r0 += 32) {
        const int r = r0 + 8 * q;
        v8bf B[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int n = min(n0 + 16 * i + r16, N - 1);
          B[i] = v8bf{};
          if (r < a.R) B[i] = *reinterpret_cast<const v8bf*>(a.b + ((size_t)l * N + n) * a.R + r);
        }
        v4f u[NJ][2];
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          u[j][0] = u[j][1] = v4f{0.f, 0.f, 0.f, 0.f};
          if (id[j] == l && r < a.R) {
            const float* p = a.u + (size_t)tok[j] * a.R + r;
            u[j][0] = *reinterpret_cast<const v4f*>(p);
            u[j][1] = *reinterpret_cast<const v4f*>(p + 4);
          }
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          if (!some[j]) continue;
          v8bf hi, lo;
#pragma unroll
          for (int v = 0; v < 8; ++v) {
            const float f = EXACT ? u[j][v >> 2][v & 3] * whole : u[j][v >> 2][v & 3];
            hi[v] = (__bf16)__builtin_amdgcn_fmed3f(f, -kBf16Max, kBf16Max);
            lo[v] = (__bf16)(EXACT ? __builtin_fmaf((float)hi[v], -off, f) : f - (float)hi[v]);
          }
#pragma unroll
          for (int i = 0; i < NI; ++i) {
            add[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(B[i], lo, add[i][j], 0, 0, 0);
            add[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(B[i], hi, add[i][j], 0, 0, 0);
          }
        }
      }
      bool odd = false;
      if constexpr (EXACT) {
        odd = pass != 0;
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int v = 0; v < 4; v += 2) odd |= id[j] == l && __builtin_isunordered(add[i][j][v], add[i][j][v + 1]);
      }
      if (!EXACT || __ballot(odd) == 0) {
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          if (id[j] == l) {
#pragma unroll
            for (int i = 0; i < NI; ++i) o[i][j] += add[i][j];
          }
        break;
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int v = 0; v < 4; ++v)
            // (of the second pass what is not finite, of the first all but NaN)
            if (id[j] == l && __builtin_amdgcn_classf(add[i][j][v], pass ? 0x207 : 0x3FC)) o[i][j][v] += add[i][j][v];
      if (pass) break;
    }
  }
}

// What a wave holds as above, stored.
template <int NI, int NJ>
__device__ __forceinline__ void store_rows(const ProjectArgs& a, const v4f (&o)[NI][NJ], const int (&tok)[NJ], int n0) {
  const int q = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    if (tok[j] < 0) continue;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int n = n0 + 16 * i + 4 * q;
      if (n >= a.N) continue;  // (N is a multiple of 16)
      const size_t at = (size_t)tok[j] * a.N + n;
      const v4f v = o[i][j];
      if (a.out_f32)
        *reinterpret_cast<v4f*>(static_cast<float*>(a.out) + at) = v;
      else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
            uint2{bf16_bits(v[0]) | (bf16_bits(v[1]) << 16), bf16_bits(v[2]) | (bf16_bits(v[3]) << 16)};
    }
  }
}

// Eight E2M1 codes times an E4M3 scale -> bfloat16, exact (6 significant bits):
// multiplied as floats, whose upper halves are the result.
__device__ __forceinline__ u32x4 dq8_scaled_bf16(uint32_t codes, float scale) {
  typedef float v2f __attribute__((ext_vector_type(2)));
  const v2f p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 0),
                    __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 1),
                    __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 2),
                    __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 3)};
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __builtin_amdgcn_perm(f2u(p[i][1] * scale), f2u(p[i][0] * scale), 0x07060302u);
  return v;
}

// 16 bytes per lane from memory to consecutive places in LDS.
__device__ __forceinline__ void direct_load(const uint16_t* src, uint8_t* lds) {
  __builtin_amdgcn_global_load_lds(src, lds, 16, 0, 0);
}

// TT: tokens per workgroup, 256 (x 256 rows, 8 waves of 128 rows x 64 tokens),
// 128 (x 128 rows, 4 waves of 64 x 64) or 64 (x 128, 32 x 64).  The larger a
// wave's tile, the fewer LDS bytes per product: 12 reads of 1 KB for 32 matrix
// instructions at 256, 8 for 16 at 128, where LDS (128 bytes per cycle) and not
// the matrix units would be full.  N = 4096, K = 6144, group32: 8192 tokens 345
// us (1.2 PFLOP/s) at 256, 451 us at 128, 605 us at 64; 2048 tokens, which fill
// half the chip at 256, 173, 118 and 155 us.
// blockIdx.y: the part of K (stages [y * per, + per)); with more than one part
// the products go to a.part as float32, which project_sum adds up.
//
// Two ways to the next stage.  TT = 64, where few workgroups hide each other's
// waits: x, codes and scales through registers, two stages ahead, with a
// barrier that leaves the loads in flight (N = 4096, K = 6144, 256 tokens: 29
// us against 62 us with direct loads).  Else, where the traffic through LDS and
// the number of requests count: x by direct loads to LDS one stage ahead, the
// weights of two stages per load.
template <int MODE, int TT>
__global__ __launch_bounds__(TT == 256 ? 512 : 256, 2) void project_gemm_kernel(ProjectArgs a, int row_tiles, int per) {
  constexpr int RW = TT == 256 ? 256 : kTile;  // weight rows per workgroup
  constexpr int NW = RW / 32;                  // waves
  constexpr int NH = TT == 256 ? 2 : 1;        // a wave's rows: NH times NI 16-row tiles
  constexpr int NI = TT == 64 ? 2 : 4;
  constexpr int NP = TT == 256 ? 2 : 1, NJ = 4 / NP;  // its 64 tokens: NP times NJ 16-token tiles
  constexpr int XD = TT / NW / 8;              // 16-byte pieces of x per thread and stage
  constexpr bool DIRECT = TT != 64;
  // (x's two buffers are objects of their own: reads of one do not wait for
  // direct loads into the other)
  __shared__ __attribute__((aligned(16))) uint8_t s_x0[TT * 128], s_x1[TT * 128], s_w[2][RW * 128];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, q = lane >> 4, K = a.K, N = a.N, T = a.T;
  // TT = 256: tiles in order of tokens, an eighth of them per XCD, so that
  // workgroups that share x share an L2 (8192 tokens 345 us against 354 us; the
  // smaller tiles lose 1 to 4% that way)
  const int nt = gridDim.x, xcd = blockIdx.x & 7;
  const int tile = TT == 256 ? xcd * (nt >> 3) + min(xcd, nt & 7) + (blockIdx.x >> 3) : blockIdx.x;
  const int n0 = (tile % row_tiles) * RW, t0 = (tile / row_tiles) * TT;
  const int wn = TT == 64 ? wave * 32 : (wave & 1) * 64 * NH, wt = TT == 64 ? 0 : (wave >> 1) * 64;
  const int s_begin = blockIdx.y * per, s_end = min(K / kGK, s_begin + per);

  // x: eight whole 128-byte rows per instruction (rows past T repeat the last
  // one: their results are not stored)
  const uint16_t* xr[XD];
  uint32_t xat[XD];
#pragma unroll
  for (int i = 0; i < XD; ++i) {
    const int r = TT / NW * wave + 8 * i + (lane >> 3);
    // (direct loads land in lane order: the swizzle is in what they fetch)
    xr[i] = a.x + (size_t)token_at(a, min(t0 + r, T - 1)) * K + 8 * (DIRECT ? (lane & 7) ^ pswz(r) : lane & 7);
    xat[i] = r * 128 + 16 * ((lane & 7) ^ pswz(r));
  }
  // weights: thread = (row, half of the stage's 32 bytes), with the scales of its 32 K
  const int wrow = tid >> 1, half = tid & 1;
  const int nrow = min(n0 + wrow, N - 1);
  const uint8_t* wsrc = a.w + (size_t)nrow * (K >> 1) + 16 * half;
  const uint8_t* ssrc = a.w_sf + (size_t)nrow * (MODE == 0 ? K >> 4 : K >> 5) + (MODE == 0 ? 2 * half : half);
  struct Raw { u32x4 x[DIRECT ? 1 : XD], c; uint32_t s; };
  auto load = [&](int s, Raw& r) __attribute__((always_inline)) {
    s = min(s, s_end - 1);  // (past the last stage: loaded again, not used)
    if constexpr (!DIRECT) {
#pragma unroll
      for (int i = 0; i < XD; ++i) r.x[i] = *reinterpret_cast<const u32x4*>(xr[i] + s * kGK);
    }
    r.c = *reinterpret_cast<const u32x4*>(wsrc + s * 32);
    if (MODE == 0) r.s = *reinterpret_cast<const uint16_t*>(ssrc + s * 4);
    else r.s = ssrc[s * 2];
  };
  const uint32_t wat = wrow * 128, wsz = pswz(wrow);
  auto store = [&](const Raw& r, int buf) __attribute__((always_inline)) {
    if constexpr (!DIRECT) {
#pragma unroll
      for (int i = 0; i < XD; ++i) *reinterpret_cast<u32x4*>((buf ? s_x1 : s_x0) + xat[i]) = r.x[i];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u32x4 v;
      if constexpr (MODE == 0) v = dq8_scaled_bf16(r.c[j], e4m3_to_f32((r.s >> (8 * (j >> 1))) & 0xFFu));
      else v = __builtin_bit_cast(u32x4, dq8_bf16(r.c[j], ue8m0_to_f32(r.s)));
      *reinterpret_cast<u32x4*>(s_w[buf] + wat + 16 * ((4 * half + j) ^ wsz)) = v;
    }
  };

  v4f acc[NH][NP][NI][NJ];
#pragma unroll
  for (int h = 0; h < NH; ++h)
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[h][j / NJ][i][j % NJ] = v4f{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](int buf) __attribute__((always_inline)) {
    const uint8_t *sx = buf ? s_x1 : s_x0, *sw = s_w[buf];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      u32x4 B[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = wt + 16 * j + r16;
        B[j] = *reinterpret_cast<const u32x4*>(sx + r * 128 + 16 * ((4 * ks + q) ^ pswz(r)));
      }
#pragma unroll
      for (int h = 0; h < NH; ++h)
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int r = wn + 16 * (NI * h + i) + r16;
          const u32x4 A = *reinterpret_cast<const u32x4*>(sw + r * 128 + 16 * ((4 * ks + q) ^ pswz(r)));
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v4f& c = acc[h][j / NJ][i][j % NJ];
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, A), __builtin_bit_cast(v8bf, B[j]), c, 0,
                                                        0, 0);
          }
        }
    }
  };

  auto stage_x = [&](int s, int buf) __attribute__((always_inline)) {
    if (DIRECT && s < s_end) {
#pragma unroll
      for (int i = 0; i < XD; ++i)
        direct_load(xr[i] + s * kGK, (buf ? s_x1 : s_x0) + (TT / NW * wave + 8 * i) * 128);
    }
  };
  // The barrier that hands a stage over: with direct loads every wave first
  // waits for its own.
  auto handover = []() __attribute__((always_inline)) {
    if constexpr (DIRECT) asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    else asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  };
  if constexpr (DIRECT) {
    // Codes and scales of two stages at a time (64 bytes of a row are the least
    // that memory delivers): the thread's 16 bytes of each stage's 32.  K and
    // the parts are whole pairs of stages.
    struct Pair { u32x4 c[2]; uint64_t s; };
    auto load2 = [&](int s, Pair& r) __attribute__((always_inline)) {
      s = min(s, s_end - 2);
      r.c[0] = *reinterpret_cast<const u32x4*>(wsrc + s * 32);
      r.c[1] = *reinterpret_cast<const u32x4*>(wsrc + s * 32 + 32);
      const uint8_t* sp = a.w_sf + (size_t)nrow * (MODE == 0 ? K >> 4 : K >> 5) + s * (MODE == 0 ? 4 : 2);
      if (MODE == 0) r.s = *reinterpret_cast<const uint64_t*>(sp);
      else r.s = *reinterpret_cast<const uint32_t*>(sp);
    };
    auto store2 = [&](const Pair& r, int par, int buf) __attribute__((always_inline)) {
      Raw w;
      w.c = r.c[par];
      w.s = (uint32_t)(r.s >> (MODE == 0 ? 32 * par + 16 * half : 16 * par + 8 * half)) & (MODE == 0 ? 0xFFFFu : 0xFFu);
      store(w, buf);
    };
    Pair cur, nxt;
    stage_x(s_begin, 0);
    load2(s_begin, cur);
    store2(cur, 0, 0);
    for (int s = s_begin; s < s_end; s += 2) {
      handover();  // stage s is in buffer 0, and every wave is past stage s - 1
      stage_x(s + 1, 1);
      load2(s + 2, nxt);
      store2(cur, 1, 1);
      multiply(0);
      handover();  // stage s + 1 is in buffer 1, and every wave is past stage s
      if (s + 2 < s_end) {
        stage_x(s + 2, 0);
        store2(nxt, 0, 0);
      }
      multiply(1);
      cur = nxt;
    }
  } else {
  Raw raw0, raw1;
  load(s_begin, raw0);
  load(s_begin + 1, raw1);
  store(raw0, 0);
  for (int s = s_begin; s < s_end; s += 2) {
    handover();  // stage s is in buffer 0, and every wave is past stage s - 1
    load(s + 2, raw0);
    __builtin_amdgcn_sched_barrier(0);  // (the loads first: what follows waits for older ones)
    multiply(0);
    store(raw1, 1);
    if (s + 1 >= s_end) break;
    handover();  // stage s + 1 is in buffer 1, and every wave is past stage s
    load(s + 3, raw1);
    __builtin_amdgcn_sched_barrier(0);
    multiply(1);
    store(raw0, 0);
  }
  }

  const float gs = a.w_gs ? a.w_gs[0] : 1.0f;
#pragma unroll
  for (int h = 0; h < NH; ++h) {
    const int nh = n0 + wn + 16 * NI * h;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = t0 + wt + 16 * j + r16;
#pragma unroll
      for (int i = 0; i < NI; ++i) acc[h][j / NJ][i][j % NJ] *= gs;
      if (gridDim.y > 1 && t < T) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int n = nh + 16 * i + 4 * q;
          if (n < N) *reinterpret_cast<v4f*>(a.part + ((size_t)blockIdx.y * T + t) * N + n) = acc[h][j / NJ][i][j % NJ];
        }
      }
    }
  }
  if (gridDim.y == 1) {
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      int tok[NJ];
      tokens_at(a, t0 + wt + 16 * NJ * p, tok);
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        if (a.L > 0) add_adapters<NI, NJ, true>(a, acc[h][p], tok, n0 + wn + 16 * NI * h);
        store_rows(a, acc[h][p], tok, n0 + wn + 16 * NI * h);
      }
    }
  }
}

// out = the sum of the parts, in order, and the adapters' part: 16 tokens x 256
// rows per workgroup, 64 rows per wave, as the product's waves hold them.
__global__ __launch_bounds__(256) void project_sum_kernel(ProjectArgs a, int parts) {
  const int lane = threadIdx.x & 63, r16 = lane & 15, q = lane >> 4;
  const int t = blockIdx.x * 16 + r16, n0 = blockIdx.y * 256 + (threadIdx.x >> 6) * 64;
  if (n0 >= a.N) return;
  int tok[1];
  tokens_at(a, blockIdx.x * 16, tok);
  v4f o[4][1];
  auto sum = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i][0] = v4f{0.f, 0.f, 0.f, 0.f};
    const float* p = a.part + (size_t)min(t, a.T - 1) * a.N;
#pragma unroll 2
    for (int z = 0; z < parts; ++z, p += (size_t)a.T * a.N)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i][0] += *reinterpret_cast<const v4f*>(p + min(n0 + 16 * i + 4 * q, a.N - 4));
  };
  sum();
  if (a.L > 0) {
    // (the test for NaN behind all adapters, and then from the start: in the
    // chain of their products it costs 300 tokens 1.5 us of 40)
    add_adapters<4, 1, false>(a, o, tok, n0);
    bool odd = false;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      odd |= __builtin_isunordered(o[i][0][0], o[i][0][1]) || __builtin_isunordered(o[i][0][2], o[i][0][3]);
    if (__ballot(odd) != 0) {
      sum();
      add_adapters<4, 1, true>(a, o, tok, n0);
    }
  }
  store_rows(a, o, tok, n0);
}

template <int MODE, int NG, int NR>
void launch_few_rows(const ProjectArgs& a, hipStream_t s) {
  const dim3 grid((a.N + 16 * NR - 1) / (16 * NR)), block(512);
  if (a.K <= 2048) hipLaunchKernelGGL((project_few_kernel<MODE, NG, 1, NR>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((project_few_kernel<MODE, NG, NR == 1 ? 3 : NG <= 4 ? 2 : 1, NR>), grid, block, 0, s, a);
}

// 32 rows per workgroup where 16 would give a CU more than one workgroup: each
// reads all of x from the L2.  16 / 32 rows, us: N = 6144, K = 6144, group16: 1
// token 14.4/13.3, 37 tokens 24.3/20.7, 128 tokens 41.4/31.1; N = 16384, K =
// 4096: 20.3/16.4, 33.3/24.2, 56.5/39.1; N = 4096, K = 6144: 10.0/12.7,
// 15.9/20.3, 25.5/30.8.
template <int MODE, int NG>
void launch_few_tokens(const ProjectArgs& a, hipStream_t s) {
  if (a.N > 16 * 256) launch_few_rows<MODE, NG, 2>(a, s);
  else launch_few_rows<MODE, NG, 1>(a, s);
}

template <int MODE>
hipError_t launch_mode(const ProjectArgs& a, hipStream_t s) {
  const bool few = a.T <= kProjectFew;
  const bool dot = a.L > 0 && project_dot(a.T, a.K, a.R);
  const int prep = few ? a.T : 0;
  const int blocks = prep + (dot ? a.T * (a.R / kShrinkRanks) : 0);
  if (blocks > 0) {
    hipLaunchKernelGGL(project_prep_kernel<MODE == 0>, dim3(blocks), dim3(256), 0, s, a, prep);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  if (a.L > 0 && !dot) {
    hipLaunchKernelGGL(project_ids_kernel, dim3((a.T + 255) / 256), dim3(256), 0, s, a);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    err = launch_route(a.ids, a.T, a.L + 1, 32, a.route, s);
    if (err != hipSuccess) return err;
    const dim3 grid((a.T + 31) / 32 + a.L + 1, a.ku);
    if (a.R <= 16) hipLaunchKernelGGL(project_shrink_kernel<1>, grid, dim3(512), 0, s, a);
    else if (a.R <= 32) hipLaunchKernelGGL(project_shrink_kernel<2>, grid, dim3(512), 0, s, a);
    else if (a.R <= 64) hipLaunchKernelGGL(project_shrink_kernel<4>, grid, dim3(512), 0, s, a);
    else hipLaunchKernelGGL(project_shrink_kernel<8>, grid, dim3(512), 0, s, a);
    err = hipGetLastError();
    if (err != hipSuccess) return err;
    if (a.ku > 1) {
      const long long n = (long long)a.T * a.R / 4;
      hipLaunchKernelGGL(project_u_sum_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, a);
      err = hipGetLastError();
      if (err != hipSuccess) return err;
    }
  }
  if (few) {
    if (a.T <= 16) launch_few_tokens<MODE, 1>(a, s);
    else if (a.T <= 32) launch_few_tokens<MODE, 2>(a, s);
    else if (a.T <= 64) launch_few_tokens<MODE, 4>(a, s);
    else launch_few_tokens<MODE, 8>(a, s);
  } else {
    const ProjectGemm g = project_gemm_plan(a.T, a.N, a.K);
    const int rows = g.tt == 256 ? 256 : kTile, rt = (a.N + rows - 1) / rows;
    const dim3 grid(rt * ((a.T + g.tt - 1) / g.tt), g.parts);
    if (g.tt == 256) hipLaunchKernelGGL((project_gemm_kernel<MODE, 256>), grid, dim3(512), 0, s, a, rt, g.per);
    else if (g.tt == 128) hipLaunchKernelGGL((project_gemm_kernel<MODE, 128>), grid, dim3(256), 0, s, a, rt, g.per);
    else hipLaunchKernelGGL((project_gemm_kernel<MODE, 64>), grid, dim3(256), 0, s, a, rt, g.per);
    if (g.parts > 1) {
      const hipError_t err = hipGetLastError();
      if (err != hipSuccess) return err;
      hipLaunchKernelGGL(project_sum_kernel, dim3((a.T + 15) / 16, (a.N + 255) / 256), dim3(256), 0, s, a, g.parts);
    }
  }
  return hipGetLastError();
}

}  // namespace

// 64 tokens per workgroup, and K in parts of at least 8 stages, where 128 would
// not fill the chip twice over (two workgroups per CU); beyond, rounds of 512
// tiles at 128 against rounds of 256 four times as large at 256, which take 1.5
// times as long (118 us and 173 us a round at N = 4096, K = 6144).
ProjectGemm project_gemm_plan(long long T, long long N, long long K) {
  ProjectGemm g;
  const long long rt = (N + kTile - 1) / kTile;
  const long long t128 = rt * ((T + 127) / 128), t256 = (N + 255) / 256 * ((T + 255) / 256);
  g.tt = t128 < 512 ? 64 : 3 * ((t256 + 255) / 256) <= 2 * ((t128 + 511) / 512) ? 256 : 128;
  if (g.tt == 256) {
    g.per = (int)(K / kGK);
    g.parts = 1;
    return g;
  }
  const long long tiles = rt * ((T + g.tt - 1) / g.tt), nst = K / kGK;
  long long parts = 512 / tiles;
  parts = parts > nst / 8 ? nst / 8 : parts;
  parts = parts < 1 ? 1 : parts;
  g.per = (int)((nst + parts - 1) / parts);
  g.parts = (int)((nst + g.per - 1) / g.per);
  return g;
}

int project_u_parts(long long T, long long K, long long R) {
  if (project_dot(T, K, R)) return 1;
  int n = 8;
  while (n > 1 && ((T + 31) / 32 * n > 256 || (K / 256) % n)) n >>= 1;
  return n;
}

// (more than one part: at most 256 tiles of 32 tokens, parts times tiles)
long long project_u_rows(long long T, long long K, long long R) {
  if (project_dot(T, K, R)) return T;
  const long long split = 8 * T < 256 * 32 ? 8 * T : 256 * 32;
  return T > split ? T : split;
}

// (more than one part: at most 512 tiles of 64 tokens, parts times tiles; none
// where 129 tokens fill 256 tiles)
long long project_part_rows(long long T, long long N, long long K) {
  const long long rt = (N + kTile - 1) / kTile, most = K / kGK / 8;
  if (T <= kProjectFew || most < 2 || 3 * rt > 256) return 0;
  return most * T < 512 * 64 / rt ? most * T : 512 * 64 / rt;
}

hipError_t launch_project(const ProjectArgs& a, hipStream_t s) {
  return a.g16 ? launch_mode<0>(a, s) : launch_mode<1>(a, s);
}

}  // namespace moefp4
