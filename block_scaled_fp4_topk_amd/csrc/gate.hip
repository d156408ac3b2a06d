// The router: logits = x Wg^T, then per token the top-k experts and their
// weights (gate_core.h).
//
// Logits.  Few tokens: one workgroup per expert row reads it once and dots it
// with up to 8 tokens.  More tokens: a tiled matrix product, 128 experts x
// 128 tokens per workgroup and K split over workgroups until the chip is
// covered (a router is narrow: 256 experts are two tiles); the parts are
// summed by the selection in a fixed order.  FP32 router weights enter the
// matrix instructions as three bfloat16 parts, the value's upper, middle and
// lower 8 significant bits (exact, by truncation), so that products stay as
// precise as in FP32.
#include "gate_core.h"

namespace moefp4 {

namespace {

template <bool WF32, int TB>
__global__ __launch_bounds__(256) void gate_dot_kernel(const void* __restrict__ w, const uint16_t* __restrict__ x,
                                                       int T, int ld, int H, float* __restrict__ logits) {
  __shared__ float s_red[4 * TB];
  const int t0 = blockIdx.y * TB;
  gate_dot_expert<WF32, TB>(w, x, blockIdx.x, t0, min(TB, T - t0), ld, H, logits, s_red);
}

// FP32 [E, H] -> three bfloat16 planes [3][E][H] by truncation.
__global__ __launch_bounds__(256) void gate_split_kernel(const float* __restrict__ w, long long n,
                                                         uint16_t* __restrict__ planes) {
  const long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * 8;
  if (i >= n) return;
  uint32_t q[3][4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float4 v = *reinterpret_cast<const float4*>(w + i + 4 * h);
    const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float r = f[j];
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        const uint32_t b = f2u(r) & 0xFFFF0000u;
        r -= u2f(b);  // exact
        if (j & 1) q[p][2 * h + (j >> 1)] |= b;
        else q[p][2 * h + (j >> 1)] = b >> 16;
      }
    }
  }
#pragma unroll
  for (int p = 0; p < 3; ++p)
    *reinterpret_cast<uint4*>(planes + (size_t)p * n + i) = uint4{q[p][0], q[p][1], q[p][2], q[p][3]};
}

constexpr int kTile = 128;  // experts and tokens per workgroup
constexpr int kGK = 64;     // K elements per stage
constexpr int kGWaves = 8;

// LDS rows of 128 bytes; 16-byte segment s of row r sits at s ^ ((r >> 1) & 7),
// so that the 16 rows a lane group reads touch all 64 banks.
__device__ __forceinline__ int gswz(int r) { return (r >> 1) & 7; }

// Stages rows [0, 128) x K [k0, k0 + 64) of a row-major bf16 matrix; each of
// the 8 waves loads 16 rows, eight whole ones per instruction.  Rows past the
// last one repeat it (their results are not stored); K past H is zero.
__device__ __forceinline__ void gate_stage(const uint16_t* __restrict__ src, int row0, int rows, int H, int k0,
                                           uint8_t* lds, int wave, int lane) {
#pragma unroll
  for (int i = 0; i < 16 / kGWaves; ++i) {
    const int r = kTile / kGWaves * wave + 8 * i + (lane >> 3);
    const int seg = (lane & 7) ^ gswz(r);
    const int k = k0 + 8 * seg;
    const int row = min(row0 + r, rows - 1);
    uint8_t* base = lds + (kTile / kGWaves * wave + 8 * i) * 128;
    if (k < H)
      __builtin_amdgcn_global_load_lds(src + (size_t)row * H + k, base, 16, 0, 0);
    else
      *reinterpret_cast<uint4*>(base + 16 * lane) = uint4{0u, 0u, 0u, 0u};
  }
}

// One 128 x 128 tile over K stages [blockIdx.z * per, + per): part z of the
// logits.  A wave has 32 experts x 64 tokens; WP planes of W.
template <int WP>
__global__ __launch_bounds__(64 * kGWaves) void gate_gemm_kernel(const uint16_t* __restrict__ w,
                                                                 const uint16_t* __restrict__ x, int T, int E, int ld,
                                                                 int H, int per, float* __restrict__ part) {
  __shared__ __attribute__((aligned(16))) uint8_t s[2][(WP + 1) * kTile * 128];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, q = lane >> 4;
  const int t0 = blockIdx.x * kTile, e0 = blockIdx.y * kTile;
  const int nst = (H + kGK - 1) / kGK;
  const int s0 = blockIdx.z * per, s1 = min(nst, s0 + per);
  constexpr int NI = 16 / kGWaves;  // 16-expert tiles of a wave
  const int we = (wave % (kGWaves / 2)) * 16 * NI, wt = wave / (kGWaves / 2) * 64;
  auto stage = [&](int c, uint8_t* b) __attribute__((always_inline)) {
    gate_stage(x, t0, T, H, c * kGK, b, wave, lane);
#pragma unroll
    for (int p = 0; p < WP; ++p)
      gate_stage(w + (size_t)p * E * H, e0, E, H, c * kGK, b + (p + 1) * kTile * 128, wave, lane);
  };
  v4f acc[NI][4];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  if (s0 < s1) stage(s0, s[0]);
  for (int c = s0; c < s1; ++c) {
    // every wave waits for its own direct loads of this stage before the
    // barrier that hands them to the others, and is past the stage before,
    // whose buffer the next one's loads take
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    const uint8_t* b = s[(c - s0) & 1];
    if (c + 1 < s1) stage(c + 1, s[(c + 1 - s0) & 1]);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      v8bf B[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = wt + 16 * j + r16;
        B[j] = *reinterpret_cast<const v8bf*>(b + r * 128 + 16 * ((4 * ks + q) ^ gswz(r)));
      }
#pragma unroll
      for (int p = 0; p < WP; ++p)
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int r = we + 16 * i + r16;
          const v8bf A = *reinterpret_cast<const v8bf*>(b + (p + 1) * kTile * 128 + r * 128 +
                                                        16 * ((4 * ks + q) ^ gswz(r)));
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A, B[j], acc[i][j], 0, 0, 0);
        }
    }
  }
  // lane: experts 4 q .. + 3 of each 16, token r16
  float* out = part + (size_t)blockIdx.z * T * ld;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int t = t0 + wt + 16 * j + r16;
    if (t >= T) continue;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int e = e0 + we + 16 * i + 4 * q;
      if (e < ld) *reinterpret_cast<v4f*>(out + (size_t)t * ld + e) = acc[i][j];
    }
  }
}

// One wavefront per token.  The logits' rows are padded to 64 * NI experts
// (what lies past E is not looked at).
template <int NI>
__global__ __launch_bounds__(256) void gate_select_kernel(const float* __restrict__ part, int nparts, int T,
                                                          GateSel g, int32_t* __restrict__ ids,
                                                          float* __restrict__ wts) {
  const int lane = threadIdx.x & 63, t = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= T) return;
  using vec = typename std::conditional<NI == 1, float, float __attribute__((ext_vector_type(NI)))>::type;
  float bias[NI];
  gate_bias<NI>(g, lane, bias);
  vec sum = 0.0f;
  const float* row = part + (size_t)t * (64 * NI) + lane * NI;
#pragma unroll 8
  for (int s = 0; s < nparts; ++s) sum += *reinterpret_cast<const vec*>(row + (size_t)s * T * (64 * NI));
  float l[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    if constexpr (NI == 1) l[i] = sum;
    else l[i] = sum[i];
  }
  const int kt = g.top_k + g.shared;
  gate_select<NI>(l, bias, g, lane, [&](int j, int id, float w) __attribute__((always_inline)) {
    ids[(size_t)t * kt + j] = id;
    wts[(size_t)t * kt + j] = w;
  });
  for (int j = lane; j < g.shared; j += 64) {
    ids[(size_t)t * kt + g.top_k + j] = g.E + j;
    wts[(size_t)t * kt + g.top_k + j] = 1.0f;
  }
}

template <int NI>
void launch_select(const float* part, int nparts, int T, const GateSel& g, int32_t* ids, float* wts, hipStream_t s) {
  const dim3 grid((T + 3) / 4);
  hipLaunchKernelGGL(gate_select_kernel<NI>, grid, dim3(256), 0, s, part, nparts, T, g, ids, wts);
}

// K stages per workgroup and the number of parts: workgroups for every CU
// once, each with at least 2 stages.  With three planes of W, whose LDS leaves a
// CU one workgroup, no more than that (6000 tokens of 256 experts, H = 6144: 3
// parts for 94 tiles are a second round, 103 us against 83).
void gate_split_k(int T, int E, int H, bool w_f32, int* per, int* parts) {
  const int nst = (H + kGK - 1) / kGK;
  const int tiles = ((T + kTile - 1) / kTile) * ((E + kTile - 1) / kTile);
  int n = w_f32 ? 256 / tiles : (256 + tiles - 1) / tiles;
  n = n > 16 ? 16 : n;
  n = n > nst / 2 ? nst / 2 : n;
  n = n < 1 ? 1 : n;
  *per = (nst + n - 1) / n;
  *parts = (nst + *per - 1) / *per;
}

}  // namespace

GatePlan gate_plan(int T, int E, int H, bool w_f32) {
  GatePlan p;
  p.dot = T <= (w_f32 ? kGateDotMaxF32 : kGateDotMax);
  p.per = 0;
  p.parts = 1;
  if (!p.dot) gate_split_k(T, E, H, w_f32, &p.per, &p.parts);
  p.planes_bytes = !p.dot && w_f32 ? (size_t)3 * E * H * 2 : 0;
  p.ld = E <= 64 ? 64 : E <= 128 ? 128 : E <= 256 ? 256 : 512;
  p.part_bytes = (size_t)p.parts * T * p.ld * 4;
  // Fewer tokens can have more parts.  n parts of t tokens, in ce tiles per 128
  // of them, take less than n t rows: 32768 / ce with FP32 weights, as n times
  // the tiles is at most 256; t + 127 more with bfloat16 ones, where it is below
  // 256 plus the tiles and n > 1 only below 256 tiles.
  size_t rows = T;
  if (!p.dot) {
    const size_t nst = (H + kGK - 1) / kGK, most = nst / 2 < 1 ? 1 : nst / 2 > 16 ? 16 : nst / 2;
    const size_t full = 32768 / ((E + kTile - 1) / kTile);
    const size_t cap = w_f32 ? full : full + (rows < full ? rows : full) + 127;
    const size_t split = most * rows < cap ? most * rows : cap;
    rows = rows > split ? rows : split;
  }
  p.most_bytes = rows * p.ld * 4;
  return p;
}

template <int TB>
static void launch_dot(const void* w, bool w_f32, const uint16_t* x, int T, int E, int ld, int H, float* part,
                       hipStream_t s) {
  const dim3 grid(E, (T + TB - 1) / TB);
  if (w_f32) hipLaunchKernelGGL((gate_dot_kernel<true, TB>), grid, dim3(256), 0, s, w, x, T, ld, H, part);
  else hipLaunchKernelGGL((gate_dot_kernel<false, TB>), grid, dim3(256), 0, s, w, x, T, ld, H, part);
}

hipError_t launch_gate(const GatePlan& p, const GateSel& g, const void* w, bool w_f32, const uint16_t* x, int T, int H,
                       uint16_t* planes, float* part, int32_t* ids, float* wts, hipStream_t s) {
  if (T <= 0) return hipSuccess;
  const int E = g.E;
  if (p.dot) {
    if (T == 1) launch_dot<1>(w, w_f32, x, T, E, p.ld, H, part, s);
    else if (T <= 4) launch_dot<4>(w, w_f32, x, T, E, p.ld, H, part, s);
    else launch_dot<8>(w, w_f32, x, T, E, p.ld, H, part, s);
  } else {
    const dim3 grid((T + kTile - 1) / kTile, (E + kTile - 1) / kTile, p.parts);
    if (w_f32) {
      const long long n = (long long)E * H;
      hipLaunchKernelGGL(gate_split_kernel, dim3((unsigned)((n / 8 + 255) / 256)), dim3(256), 0, s,
                         static_cast<const float*>(w), n, planes);
      const hipError_t err = hipGetLastError();
      if (err != hipSuccess) return err;
      hipLaunchKernelGGL(gate_gemm_kernel<3>, grid, dim3(64 * kGWaves), 0, s, planes, x, T, E, p.ld, H, p.per, part);
    } else {
      hipLaunchKernelGGL(gate_gemm_kernel<1>, grid, dim3(64 * kGWaves), 0, s, static_cast<const uint16_t*>(w), x,
                         T, E, p.ld, H, p.per, part);
    }
  }
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  if (E <= 64) launch_select<1>(part, p.parts, T, g, ids, wts, s);
  else if (E <= 128) launch_select<2>(part, p.parts, T, g, ids, wts, s);
  else if (E <= 256) launch_select<4>(part, p.parts, T, g, ids, wts, s);
  else launch_select<8>(part, p.parts, T, g, ids, wts, s);
  return hipGetLastError();
}

}  // namespace moefp4
