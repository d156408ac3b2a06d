// Norms before and after a block, fused with its gate and residual scale:
//   a  = rms(y) * post_w  (or y),  rms(v) = v / sqrt(mean(v^2) + eps)
//   h' = h_scale h + scale act(gate) a
//   n  = rms(h') * pre_w
// and the gradient.  Memory bounds both: every tensor is read once and written
// once, a row stays in registers between the two norms.  8192 x 6144, bfloat16: 84 us,
// 4.8 TB/s, where a large copy reaches 4.9; the gradient with a float32 stream 206 us
// and 5 us for the sums over rows, 4.4 TB/s.
#include "common.h"
#include "kernels.h"

namespace moefp4 {

namespace {

__device__ __forceinline__ uint32_t bf16_bits(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

// Eight values at element i.
__device__ __forceinline__ void load8(const void* p, bool f32, size_t i, float (&v)[8]) {
  if (f32) {
    const v4f a = *reinterpret_cast<const v4f*>(static_cast<const float*>(p) + i);
    const v4f b = *reinterpret_cast<const v4f*>(static_cast<const float*>(p) + i + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = a[j], v[4 + j] = b[j];
  } else {
    const u32x4 a = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[2 * j] = u2f(a[j] << 16), v[2 * j + 1] = u2f(a[j] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ void store8(void* p, bool f32, size_t i, const float (&v)[8]) {
  if (f32) {
    *reinterpret_cast<v4f*>(static_cast<float*>(p) + i) = v4f{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<v4f*>(static_cast<float*>(p) + i + 4) = v4f{v[4], v[5], v[6], v[7]};
  } else {
    u32x4 a;
#pragma unroll
    for (int j = 0; j < 4; ++j) a[j] = bf16_bits(v[2 * j]) | (bf16_bits(v[2 * j + 1]) << 16);
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + i) = a;
  }
}

__device__ __forceinline__ float load1(const void* p, bool f32, size_t i) {
  return f32 ? static_cast<const float*>(p)[i] : bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
}

// 1 / (1 + e^-g) to a few ulp: 2^t with the rounding of t = -g log2(e) put back,
// and the hardware's reciprocal.  Beyond +-87, where one side is 1 and the other
// leaves FP32's normal range, 1 and 0: a gate that is closed by -infinity or by its
// type's lowest value lets nothing through.  (NaN stays.)  Its slope is e / (1 + e)^2,
// e = e^-g, and 0 beyond +-87: of a large gate s (1 - s) would leave the rounding of s
// (0 from 17 on).
__device__ __forceinline__ float sigmoid(float g, float* slope = nullptr) {
  const float x = g > 87.0f ? -87.0f : g < -87.0f ? 87.0f : -g;
  const float t = x * 0x1.715476p+0f;
  const float lo = __builtin_fmaf(x, 0x1.715476p+0f, -t) + x * 0x1.4AE0C0p-26f;  // log2(e) = the two parts' sum
  const float e0 = __builtin_amdgcn_exp2f(t), e = __builtin_fmaf(e0, lo * 0x1.62E430p-1f, e0);
  const float s = __builtin_amdgcn_rcpf(1.0f + e);
  if (slope) *slope = fabsf(g) > 87.0f ? 0.0f : e * s * s;
  return g < -87.0f ? 0.0f : s;
}

// Eight values as they lie in memory.
template <bool F32>
struct Eight {
  u32x4 v[F32 ? 2 : 1];
  __device__ __forceinline__ void zero() {
    v[0] = u32x4{0, 0, 0, 0};
    if constexpr (F32) v[1] = v[0];
  }
  __device__ __forceinline__ void load(const void* p, size_t i) {
    const u32x4* q = reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(p) + (F32 ? 4 : 2) * i);
    v[0] = q[0];
    if constexpr (F32) v[1] = q[1];
  }
  __device__ __forceinline__ float operator[](int j) const {
    if constexpr (F32) return u2f(v[j >> 2][j & 3]);
    else return u2f(j & 1 ? v[0][j >> 1] & 0xFFFF0000u : v[0][j >> 1] << 16);
  }
};

// A row is one wave's (WAVE: 4 rows per workgroup) or a workgroup's; sums over
// its threads, the same in all of them.  LDS is used in turns, so that one
// barrier per call is enough.
constexpr int kMostWaves = 16, kMostSums = 3;
template <bool WAVE>
struct RowSum {
  float (*s)[kMostSums][kMostWaves];  // [2], zeros for waves that are not there
  int turn = 0;
  __device__ __forceinline__ void init() {
    if constexpr (!WAVE) {
      if (threadIdx.x < 64) {  // (at least a wave)
        for (int i = threadIdx.x; i < 2 * kMostSums * kMostWaves; i += 64) (&s[0][0][0])[i] = 0.0f;
      }
      __syncthreads();
    }
  }
  template <int N>
  __device__ __forceinline__ void operator()(float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) v[i] += __shfl_xor(v[i], d, 64);
    if constexpr (!WAVE) {
      if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) s[turn][i][threadIdx.x >> 6] = v[i];
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const v4f* p = reinterpret_cast<const v4f*>(s[turn][i]);
        const v4f t = (p[0] + p[1]) + (p[2] + p[3]);
        v[i] = (t[0] + t[1]) + (t[2] + t[3]);
      }
      turn ^= 1;
    }
  }
};

constexpr float kDown = 0x1p-80f;

// 1 / sqrt(mean + eps) of a row whose squares add up to ss (already summed).
// Where they left FP32's range, of the row scaled down.
template <bool WAVE, int C, class V>
__device__ __forceinline__ float rms_factor(float ss, const V (&v)[C], float inv, float eps, RowSum<WAVE>& sum) {
  if (ss != __builtin_inff()) return 1.0f / sqrtf(__builtin_fmaf(ss, inv, eps));
  float t[1] = {0.0f};
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = v[c][j] * kDown;
      t[0] = __builtin_fmaf(x, x, t[0]);
    }
  sum(t);
  return kDown / sqrtf(t[0] * inv);
}

struct Floats {
  float f[8];
  __device__ __forceinline__ float operator[](int j) const { return f[j]; }
};

// KIND: -1 without a branch (y), else the gate's kind.
// 8 C elements per thread.
template <bool WAVE, int C, bool F32, int KIND>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void block_norm_kernel(NormArgs a) {
  __shared__ __attribute__((aligned(16))) float s_sum[2][kMostSums][kMostWaves];
  RowSum<WAVE> sum{s_sum};
  sum.init();
  const int tid = WAVE ? threadIdx.x & 63 : threadIdx.x, tpr = WAVE ? 64 : blockDim.x, H = a.H;
  const long long b = (long long)blockIdx.y * gridDim.x + blockIdx.x, t = WAVE ? b * 4 + (threadIdx.x >> 6) : b;
  if (t >= a.T) return;  // (WAVE: whole waves, without barriers)
  const size_t row = (size_t)t * H;
  const float inv = 1.0f / (float)H;
  Eight<F32> hr[C];
  Eight<false> y[C];
  Floats h[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int at = (c * tpr + tid) * 8;
    hr[c].zero();
    y[c].zero();
    if (at < H) {
      hr[c].load(a.h, row + at);
      if (KIND >= 0) y[c].load(a.y, row + at);
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) h[c].f[j] = hr[c][j];
  if constexpr (KIND >= 0) {
    float ry = 1.0f;
    if (a.post_w) {
      float ss[1] = {0.0f};
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss[0] = __builtin_fmaf(y[c][j], y[c][j], ss[0]);
      sum(ss);
      ry = rms_factor(ss[0], y, inv, a.eps, sum);
    }
    float gt = a.scale;
    if (KIND == 2) {
      const float g = load1(a.gate, a.gate_f32, t);
      gt *= a.gate_act ? sigmoid(g) : g;
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int at = (c * tpr + tid) * 8;
      if (at >= H) continue;
      float w[8], g[8], b[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) b[j] = y[c][j];
      if (a.post_w) {
        load8(a.post_w, a.post_f32, at, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] = b[j] * ry * w[j];
      }
      if (KIND == 1 || KIND == 3) {
        load8(a.gate, a.gate_f32, (KIND == 3 ? row : 0) + at, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] *= a.gate_act ? sigmoid(g[j]) : g[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) h[c].f[j] = __builtin_fmaf(gt, b[j], a.h_scale * h[c][j]);
      store8(a.h_out, F32, row + at, h[c].f);
    }
  }
  if (!a.pre_w) return;
  float ss[1] = {0.0f};
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) ss[0] = __builtin_fmaf(h[c][j], h[c][j], ss[0]);
  sum(ss);
  const float r = rms_factor(ss[0], h, inv, a.eps, sum);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int at = (c * tpr + tid) * 8;
    if (at >= H) continue;
    float w[8];
    load8(a.pre_w, a.pre_f32, at, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = h[c][j] * r * w[j];
    store8(a.n, false, row + at, w);
  }
}

// The gradient.  With hh = h r, yy = y ry (the rows over their root mean
// squares), u = dn pre_w, D = dh + r (u - hh mean(u hh)):
//   d_h = h_scale D, da = scale act(gate) D, v = da post_w,
//   dy = ry (v - yy mean(v yy)), d_gate = scale act'(gate) D a,
//   d_pre_w = sum of dn hh, d_post_w = sum of da yy over the rows.
// A workgroup takes every grid-th row and keeps its part of the sums over rows,
// a thread its own columns', in LDS (MOST threads at most); norm_sum_kernel adds
// the parts in order.  Where registers allow it (kAhead) the next row is asked for
// before this one's sums (on one card 8192 x 6144, float32: 245 us without, 235 with;
// bfloat16 193 and 184; x 1024 84 and 41).
template <bool WAVE, bool F32, int KIND, int MOST>
__global__ __launch_bounds__(MOST) void block_norm_grad_kernel(NormArgs a) {
  __shared__ __attribute__((aligned(16))) float s_sum[2][kMostSums][kMostWaves];
  RowSum<WAVE> sum{s_sum};
  sum.init();
  const int tid = WAVE ? threadIdx.x & 63 : threadIdx.x, tpr = WAVE ? 64 : blockDim.x, H = a.H;
  constexpr int C = 1;
  const float inv = 1.0f / (float)H;
  const long long first = WAVE ? (long long)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  const long long step = (long long)gridDim.x * (WAVE ? 4 : 1);
  constexpr int kKinds = KIND < 0 ? 1 : KIND == 1 ? 3 : 2;
  __shared__ v4f s_acc[kKinds * 2 * MOST];
#pragma unroll
  for (int i = 0; i < 2 * kKinds; ++i) s_acc[i * MOST + threadIdx.x] = v4f{0.f, 0.f, 0.f, 0.f};
  // v added to the thread's part of a sum (0: pre_w's, 1: post_w's, 2: the gate's)
  auto add = [&](int kind, const float (&v)[8]) __attribute__((always_inline)) {
    v4f* p = s_acc + 2 * kind * MOST + threadIdx.x;
    p[0] += v4f{v[0], v[1], v[2], v[3]};
    p[MOST] += v4f{v[4], v[5], v[6], v[7]};
  };
  // A row's values; the next row's are asked for before this one's sums.
  struct Row {
    Eight<F32> h[C], d[C];
    Eight<false> y[C], dn[C];
  } ahead;
  auto load = [&](long long t) __attribute__((always_inline)) {
    const size_t row = (size_t)t * H;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int at = (c * tpr + tid) * 8;
      ahead.h[c].zero();
      ahead.d[c].zero();
      ahead.y[c].zero();
      ahead.dn[c].zero();
      if (at < H) {
        if (a.pre_w) {
          ahead.h[c].load(a.h, row + at);
          ahead.dn[c].load(a.dn, row + at);
        }
        if (KIND >= 0) ahead.y[c].load(a.y, row + at);
        if (a.dh) ahead.d[c].load(a.dh, row + at);
      }
    }
  };
  // (512 threads: two workgroups per CU without it take 133 us for 8192 rows of 4096,
  // float32, one with it 157 us; 1024 threads have too few registers)
  constexpr bool kAhead = MOST == 768 || MOST == 256;
  if (kAhead && first < a.T) load(first);
  for (long long t = first; t < a.T; t += step) {
    const size_t row = (size_t)t * H;
    if (!kAhead) load(t);
    const Row now = ahead;
    if (kAhead && t + step < a.T) load(t + step);
    const Eight<F32>(&h)[C] = now.h, (&d)[C] = now.d;
    const Eight<false>(&y)[C] = now.y, (&dn)[C] = now.dn;
    float ss[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int at = (c * tpr + tid) * 8;
      float w[8] = {};
      if (a.pre_w && at < H) load8(a.pre_w, a.pre_f32, at, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ss[0] = __builtin_fmaf(h[c][j], h[c][j], ss[0]);
        ss[1] = __builtin_fmaf(dn[c][j] * w[j], h[c][j], ss[1]);
        ss[2] = __builtin_fmaf(y[c][j], y[c][j], ss[2]);
      }
    }
    sum(ss);
    Floats D[C];
    float r = 0.0f, m = 0.0f;  // m = mean(u hh)
    if (a.pre_w) {
      r = rms_factor(ss[0], h, inv, a.eps, sum);
      m = ss[1] * r * inv;
      if (ss[0] == __builtin_inff()) {
        float u[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const int at = (c * tpr + tid) * 8;
          float w[8] = {};
          if (at < H) load8(a.pre_w, a.pre_f32, at, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) u[0] = __builtin_fmaf(dn[c][j] * w[j], h[c][j] * r, u[0]);
        }
        sum(u);
        m = u[0] * inv;
      }
    }
    const float hs = KIND >= 0 ? a.h_scale : 1.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int at = (c * tpr + tid) * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) D[c].f[j] = d[c][j];
      if (at >= H) continue;
      if (a.pre_w) {
        float w[8], p[8];
        load8(a.pre_w, a.pre_f32, at, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float hh = h[c][j] * r;
          p[j] = dn[c][j] * hh;
          D[c].f[j] = __builtin_fmaf(r, dn[c][j] * w[j] - hh * m, D[c][j]);
        }
        add(0, p);
      }
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = hs * D[c][j];
      store8(a.d_h, F32, row + at, o);
    }
    if (KIND < 0) continue;

    const float ry = a.post_w ? rms_factor(ss[2], y, inv, a.eps, sum) : 1.0f;
    float act_t = 1.0f, slope_t = 1.0f;
    if (KIND == 2) {
      act_t = load1(a.gate, a.gate_f32, t);
      if (a.gate_act) act_t = sigmoid(act_t, &slope_t);
    }
    float vs[2] = {0.0f, 0.0f};  // sums of v yy and of D a
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int at = (c * tpr + tid) * 8;
      if (at >= H) continue;
      float w[8], g[8], o[8], p[8];
      if (a.post_w) load8(a.post_w, a.post_f32, at, w);
      if (KIND == 1 || KIND == 3) load8(a.gate, a.gate_f32, (KIND == 3 ? row : 0) + at, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float yy = y[c][j] * ry, wj = a.post_w ? w[j] : 1.0f;
        const float sd = a.scale * D[c][j], Da = sd * (yy * wj);
        float act = act_t, slope = slope_t;
        if (KIND == 1 || KIND == 3) {
          slope = 1.0f;
          act = a.gate_act ? sigmoid(g[j], &slope) : g[j];
        }
        o[j] = Da * slope;
        const float da = sd * act;
        p[j] = da * yy;
        D[c].f[j] = da * wj;  // v from here on
        vs[0] = __builtin_fmaf(D[c][j], yy, vs[0]);
        vs[1] += Da;
      }
      if (a.post_w) add(1, p);
      if (KIND == 1) add(2, o);
      if (KIND == 3) store8(a.d_gate, a.gate_f32, row + at, o);
    }
    if (a.post_w || KIND == 2) sum(vs);
    if (KIND == 2 && tid == 0) static_cast<float*>(a.d_gate)[t] = vs[1] * slope_t;
    const float mv = a.post_w ? vs[0] * inv : 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int at = (c * tpr + tid) * 8;
      if (at >= H) continue;
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = a.post_w ? ry * (D[c][j] - y[c][j] * ry * mv) : D[c][j];  // (y may be an infinity)
      store8(a.d_y, false, row + at, o);
    }
  }
  // the parts: [kind][workgroup (or wave)][H]
  const int at = tid * 8;
  if (at >= H) return;
#pragma unroll
  for (int kind = 0; kind < kKinds; ++kind) {
    if (kind == 0 ? !a.pre_w : kind == 1 && !a.post_w) continue;
    v4f* p = reinterpret_cast<v4f*>(a.part + ((size_t)kind * step + first) * H + at);
    p[0] = s_acc[2 * kind * MOST + threadIdx.x];
    p[1] = s_acc[(2 * kind + 1) * MOST + threadIdx.x];
  }
}

// The same for rows beyond 8192, which are read three times (a row lies in the
// caches then): the sums of squares; D and what follows from it elementwise; dy.
// The parts of the sums over rows stay in the workspace.
template <bool F32, int KIND>
__global__ __launch_bounds__(1024) void block_norm_grad_wide_kernel(NormArgs a) {
  __shared__ __attribute__((aligned(16))) float s_sum[2][kMostSums][kMostWaves];
  RowSum<false> sum{s_sum};
  sum.init();
  const int H = a.H, step8 = blockDim.x * 8;
  const float inv = 1.0f / (float)H;
  for (long long t = blockIdx.x; t < a.T; t += gridDim.x) {
    const size_t row = (size_t)t * H;
    const bool fresh = t == blockIdx.x;
    auto add = [&](int kind, int at, const float (&v)[8]) __attribute__((always_inline)) {
      float* p = a.part + ((size_t)kind * gridDim.x + blockIdx.x) * H;
      float o[8] = {};
      if (!fresh) load8(p, true, at, o);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] += v[j];
      store8(p, true, at, o);
    };
    // the sums, of the rows scaled by a power of two
    float ss[3], down = 1.0f;
    auto squares = [&]() __attribute__((always_inline)) {
      ss[0] = ss[1] = ss[2] = 0.0f;
#pragma unroll 1
      for (int at = threadIdx.x * 8; at < H; at += step8) {
        if (a.pre_w) {
          Eight<F32> h;
          Eight<false> dn;
          float w[8];
          h.load(a.h, row + at);
          dn.load(a.dn, row + at);
          load8(a.pre_w, a.pre_f32, at, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float x = h[j] * down;
            ss[0] = __builtin_fmaf(x, x, ss[0]);
            ss[1] = __builtin_fmaf(dn[j] * w[j], x, ss[1]);
          }
        }
        if (KIND >= 0 && a.post_w) {
          Eight<false> y;
          y.load(a.y, row + at);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float x = y[j] * down;
            ss[2] = __builtin_fmaf(x, x, ss[2]);
          }
        }
      }
      sum(ss);
    };
    squares();
    float r = 1.0f / sqrtf(__builtin_fmaf(ss[0], inv, a.eps)), m = ss[1] * r * inv;
    float ry = KIND >= 0 && a.post_w ? 1.0f / sqrtf(__builtin_fmaf(ss[2], inv, a.eps)) : 1.0f;
    if (ss[0] == __builtin_inff() || ss[2] == __builtin_inff()) {
      const bool h_big = ss[0] == __builtin_inff(), y_big = ss[2] == __builtin_inff();
      down = kDown;
      squares();
      if (h_big) {
        const float rs = 1.0f / sqrtf(ss[0] * inv);
        r = rs * kDown;
        m = ss[1] * rs * inv;
      }
      if (y_big) ry = kDown / sqrtf(ss[2] * inv);
    }
    float act_t = 1.0f, slope_t = 1.0f;
    if (KIND == 2) {
      act_t = load1(a.gate, a.gate_f32, t);
      if (a.gate_act) act_t = sigmoid(act_t, &slope_t);
    }
    // d = D of the eight at `at`
    auto total = [&](int at, bool first, float (&d)[8]) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = 0.0f;
      if (a.dh) load8(a.dh, F32, row + at, d);
      if (a.pre_w) {
        Eight<F32> h;
        Eight<false> dn;
        float w[8], p[8];
        h.load(a.h, row + at);
        dn.load(a.dn, row + at);
        load8(a.pre_w, a.pre_f32, at, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float hh = h[j] * r;
          p[j] = dn[j] * hh;
          d[j] = __builtin_fmaf(r, dn[j] * w[j] - hh * m, d[j]);
        }
        if (first) add(0, at, p);
      }
    };
    // v of the eight, yy; with them the gate's gradient and the sums
    float vs[2] = {0.0f, 0.0f};
    auto branch = [&](int at, bool first, const float (&d)[8], float (&v)[8], float (&yy)[8]) __attribute__((always_inline)) {
      Eight<false> y;
      float w[8], g[8], o[8], p[8];
      y.load(a.y, row + at);
      if (a.post_w) load8(a.post_w, a.post_f32, at, w);
      if (KIND == 1 || KIND == 3) load8(a.gate, a.gate_f32, (KIND == 3 ? row : 0) + at, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        yy[j] = y[j] * ry;
        const float wj = a.post_w ? w[j] : 1.0f, sd = a.scale * d[j], Da = sd * (yy[j] * wj);
        float act = act_t, slope = slope_t;
        if (KIND == 1 || KIND == 3) {
          slope = 1.0f;
          act = a.gate_act ? sigmoid(g[j], &slope) : g[j];
        }
        o[j] = Da * slope;
        p[j] = sd * act * yy[j];
        v[j] = sd * act * wj;
        if (first) {
          vs[0] = __builtin_fmaf(v[j], yy[j], vs[0]);
          vs[1] += Da;
        }
      }
      if (!first) return;
      if (a.post_w) add(1, at, p);
      if (KIND == 1) add(2, at, o);
      if (KIND == 3) store8(a.d_gate, a.gate_f32, row + at, o);
    };
    const float hs = KIND >= 0 ? a.h_scale : 1.0f;
    // (d_h may lie where dh does: it is written when dh is no longer read)
#pragma unroll 1
    for (int at = threadIdx.x * 8; at < H; at += step8) {
      float d[8];
      total(at, true, d);
      if (KIND >= 0) {
        float v[8], yy[8];
        branch(at, true, d, v, yy);
      } else {
        store8(a.d_h, F32, row + at, d);
      }
    }
    if (KIND < 0) continue;
    if (a.post_w || KIND == 2) sum(vs);
    if (KIND == 2 && threadIdx.x == 0) static_cast<float*>(a.d_gate)[t] = vs[1] * slope_t;
    const float mv = a.post_w ? vs[0] * inv : 0.0f;
#pragma unroll 1
    for (int at = threadIdx.x * 8; at < H; at += step8) {
      float d[8], v[8], yy[8];
      total(at, false, d);
      branch(at, false, d, v, yy);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        d[j] *= hs;
        if (a.post_w) v[j] = ry * (v[j] - yy[j] * mv);  // (else v: y may be an infinity)
      }
      store8(a.d_h, F32, row + at, d);
      store8(a.d_y, false, row + at, v);
    }
  }
}

// The sums over the parts, in order: 64 columns per workgroup, the parts split
// over its 16 waves.
__global__ __launch_bounds__(1024) void norm_sum_kernel(NormArgs a, int parts) {
  __shared__ float s[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, kind = blockIdx.y;
  float* out = kind == 0 ? a.d_pre_w : kind == 1 ? a.d_post_w : a.gate_kind == 1 ? static_cast<float*>(a.d_gate) : nullptr;
  if (!out) return;
  const int c = blockIdx.x * 64 + lane, per = (parts + 15) / 16;
  float v = 0.0f;
  if (c < a.H) {
    const float* p = a.part + (size_t)kind * parts * a.H + c;
#pragma unroll 16
    for (int i = wave * per; i < min(parts, (wave + 1) * per); ++i) v += p[(size_t)i * a.H];
  }
  s[wave][lane] = v;
  __syncthreads();
  if (wave == 0 && c < a.H) {
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w) v += s[w][lane];
    out[c] = v;
  }
}

// Rows of up to 512 elements: a wave each.  Beyond, a workgroup of as many waves
// as the row has pieces of 512 elements (1024 beyond 8192).
constexpr long long kGridX = 1 << 20;  // (a dimension of a grid has less than 2^32 threads)
int threads_of(int H, int C) { return (H + 512 * C - 1) / (512 * C) * 64; }

template <bool WAVE, int C, bool F32, int KIND>
void launch_one(const NormArgs& a, int parts, hipStream_t s) {
  const dim3 block(WAVE ? 256 : threads_of(a.H, C));
  if (parts > 0) {
    const dim3 grid(WAVE ? parts / 4 : parts);
    if constexpr (C > 1) hipLaunchKernelGGL((block_norm_grad_wide_kernel<F32, KIND>), grid, block, 0, s, a);
    else if constexpr (WAVE) hipLaunchKernelGGL((block_norm_grad_kernel<true, F32, KIND, 256>), grid, block, 0, s, a);
    else if (block.x <= 256) hipLaunchKernelGGL((block_norm_grad_kernel<false, F32, KIND, 256>), grid, block, 0, s, a);
    else if (block.x <= 512) hipLaunchKernelGGL((block_norm_grad_kernel<false, F32, KIND, 512>), grid, block, 0, s, a);
    else if (block.x <= 768) hipLaunchKernelGGL((block_norm_grad_kernel<false, F32, KIND, 768>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((block_norm_grad_kernel<false, F32, KIND, 1024>), grid, block, 0, s, a);
  } else {
    const long long n = WAVE ? (a.T + 3) / 4 : a.T, x = n < kGridX ? n : kGridX;
    const dim3 grid((unsigned)x, (unsigned)((n + x - 1) / x));
    hipLaunchKernelGGL((block_norm_kernel<WAVE, C, F32, KIND>), grid, block, 0, s, a);
  }
}

template <bool WAVE, int C, bool F32>
void launch_kind(const NormArgs& a, int parts, hipStream_t s) {
  if (!a.y) launch_one<WAVE, C, F32, -1>(a, parts, s);
  else if (a.gate_kind == 0) launch_one<WAVE, C, F32, 0>(a, parts, s);
  else if (a.gate_kind == 1) launch_one<WAVE, C, F32, 1>(a, parts, s);
  else if (a.gate_kind == 2) launch_one<WAVE, C, F32, 2>(a, parts, s);
  else launch_one<WAVE, C, F32, 3>(a, parts, s);
}

template <bool WAVE, int C>
void launch_type(const NormArgs& a, int parts, hipStream_t s) {
  if (a.h_f32) launch_kind<WAVE, C, true>(a, parts, s);
  else launch_kind<WAVE, C, false>(a, parts, s);
}

// parts: the gradient's, or 0 for the norms themselves
hipError_t launch(const NormArgs& a, int parts, hipStream_t s) {
  if (a.H <= 512) launch_type<true, 1>(a, parts, s);
  else if (a.H <= 8192) launch_type<false, 1>(a, parts, s);
  else launch_type<false, 2>(a, parts, s);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_block_norm(const NormArgs& a, hipStream_t s) { return launch(a, 0, s); }

// As many workgroups as the chip holds at a time, so that the parts of the sums
// over rows are few (8192 x 6144, float32: 256 of them 235 us, 512 242 us).
int norm_grad_parts(long long T, int H) {
  if (H <= 512) return (int)(T < 4096 ? (T + 3) / 4 * 4 : 4096);
  const int waves = threads_of(H, H <= 8192 ? 1 : 2) / 64;
  const long long most = 256 * (waves > 8 ? 1 : waves > 4 ? 2 : 12 / waves);
  return (int)(T < most ? T : most);
}

hipError_t launch_block_norm_grad(const NormArgs& a, hipStream_t s) {
  const int parts = norm_grad_parts(a.T, a.H);
  if (parts > 0) {
    const hipError_t err = launch(a, parts, s);
    if (err != hipSuccess) return err;
  }
  if (a.pre_w || a.post_w || a.gate_kind == 1)
    hipLaunchKernelGGL(norm_sum_kernel, dim3((a.H + 63) / 64, 3), dim3(1024), 0, s, a, parts);
  return hipGetLastError();
}

}  // namespace moefp4
