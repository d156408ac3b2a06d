// The router's selection of one token by one wavefront, shared by the router
// and the few-token layer.
#pragma once

#include "common.h"
#include "kernels.h"

#include <type_traits>

namespace moefp4 {

// Maximum over the wavefront, in every lane: four shifts inside a row of 16
// lanes, two broadcasts across the rows (data-parallel-primitive moves, no
// LDS), the last lane's value read back.  v is never NaN.
template <int CTRL>
__device__ __forceinline__ float dpp_move(float v) {
  const int i = __builtin_bit_cast(int, v);
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(i, i, CTRL, 0xf, 0xf, false));
}
template <int CTRL>
__device__ __forceinline__ double dpp_move(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const int lo = (int)(uint32_t)u, hi = (int)(uint32_t)(u >> 32);
  const uint32_t l = (uint32_t)__builtin_amdgcn_update_dpp(lo, lo, CTRL, 0xf, 0xf, false);
  const uint32_t h = (uint32_t)__builtin_amdgcn_update_dpp(hi, hi, CTRL, 0xf, 0xf, false);
  return __builtin_bit_cast(double, (uint64_t)l | ((uint64_t)h << 32));
}
__device__ __forceinline__ float max_of(float a, float b) { return __builtin_fmaxf(a, b); }
__device__ __forceinline__ double max_of(double a, double b) { return __builtin_fmax(a, b); }
__device__ __forceinline__ float last_lane(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}
__device__ __forceinline__ double last_lane(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t l = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, 63);
  const uint32_t h = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), 63);
  return __builtin_bit_cast(double, (uint64_t)l | ((uint64_t)h << 32));
}
template <class S>
__device__ __forceinline__ S wave_max(S v) {
  v = max_of(v, dpp_move<0x111>(v));  // row_shr 1, 2, 4, 8
  v = max_of(v, dpp_move<0x112>(v));
  v = max_of(v, dpp_move<0x114>(v));
  v = max_of(v, dpp_move<0x118>(v));
  v = max_of(v, dpp_move<0x142>(v));  // row_bcast 15, 31
  v = max_of(v, dpp_move<0x143>(v));
  return last_lane(v);
}
template <class S>
__device__ __forceinline__ S wave_sum(S v) {
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// Selects the experts of one token.  Lane l holds the logits of experts
// l * NI + i, so that among equal scores the lowest lane, and in it the
// lowest i, is the lowest expert index.  score = softmax over the finite
// logits, or sigmoid; selection by score + bias (BIAS) or by score alone,
// for which the logits themselves are compared (both scores grow with the
// logit).  Experts whose logit is not finite, or whose score + bias is NaN or
// -inf, are never selected; when none is left the remaining places get id -1
// and weight 0.
//
// With a bias the scores are formed and compared in 64 bits: score + bias is
// a rounded number, two of them can be closer than the FP32 rounding of exp,
// and the experts a token takes should not depend on that rounding.  (E / 64
// 64-bit exponentials per lane: not visible beside the logits.)
//
// emit(j, id, weight) is called by lane j % 64 with place j's expert and its
// weight: the score, divided by the selected scores' sum if renorm, times
// scale.
template <int NI, bool BIAS, class F>
__device__ __forceinline__ void gate_select(const float (&l)[NI], const GateSel& g, int lane, F&& emit) {
  using S = typename std::conditional<BIAS, double, float>::type;
  const S kNone = (S)-__builtin_inff();
  S p[NI], sel[NI];
  bool fin[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) fin[i] = lane * NI + i < g.E && __builtin_isfinite(l[i]);
  float m = -__builtin_inff();
  S inv = 1;
  const bool softmax = g.scoring == MOEFP4_SCORE_SOFTMAX;
  if (softmax) {
#pragma unroll
    for (int i = 0; i < NI; ++i) m = fin[i] ? max_of(m, l[i]) : m;
    m = wave_max(m);
    S sum = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if constexpr (BIAS) p[i] = fin[i] ? exp((double)l[i] - (double)m) : 0.0;
      else p[i] = fin[i] ? expf(l[i] - m) : 0.0f;
      sum += p[i];
    }
    inv = (S)1 / wave_sum(sum);
  }
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    if constexpr (BIAS) {
      p[i] = softmax ? p[i] * inv : 1.0 / (1.0 + exp(-(double)l[i]));
      const int e = lane * NI + i;
      const double s = p[i] + (double)(fin[i] ? g.bias[e] : 0.0f);
      sel[i] = fin[i] && s > kNone ? s : kNone;  // (false for NaN)
    } else {
      sel[i] = fin[i] ? (S)l[i] : kNone;
    }
  }
  S mine = 0;   // the score of the place this lane holds
  int my = -1;  // and its expert
  for (int j = 0; j < g.top_k; ++j) {
    S best = sel[0];
    int bi = 0;
#pragma unroll
    for (int i = 1; i < NI; ++i)
      if (sel[i] > best) best = sel[i], bi = i;
    const S top = wave_max(best);
    if (!(top > kNone)) break;
    const int who = __builtin_ctzll(ballot(best == top));
    const int wi = __builtin_amdgcn_readlane(bi, who);
    S ps = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if (i == wi) {
        if constexpr (BIAS) ps = p[i];
        else ps = softmax ? p[i] : sel[i];
        if (lane == who) sel[i] = kNone;
      }
    }
    ps = __shfl(ps, who, 64);
    if (lane == (j & 63)) mine = ps, my = who * NI + wi;
  }
  if constexpr (!BIAS) {
    if (my >= 0) mine = softmax ? mine * inv : 1.0f / (1.0f + expf(-mine));
    else mine = 0;
  }
  S f = (S)g.scale;
  if (g.renorm) {
    const S sum = wave_sum(lane < g.top_k ? mine : (S)0);
    f = sum > 0 ? f / sum : (S)0;
  }
  if (lane < g.top_k) emit(lane, my, (float)(mine * f));
}

// One W row (bf16 or fp32) against up to TB rows of x by one workgroup of
// 256 threads: acc[t] = sum over this thread's K elements (8 at a time, every
// 2048), reduced by the caller.
template <bool WF32, int TB>
__device__ __forceinline__ void gate_dot(const void* __restrict__ w_row, const uint16_t* __restrict__ x, int nt,
                                         int H, int tid, float (&acc)[TB]) {
#pragma unroll
  for (int t = 0; t < TB; ++t) acc[t] = 0.0f;
  for (int k = tid * 8; k < H; k += 2048) {
    float w[8];
    if constexpr (WF32) {
      const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(w_row) + k);
      const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(w_row) + k + 4);
      w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    } else {
      const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w_row) + k);
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) w[2 * i] = u2f(u[i] << 16), w[2 * i + 1] = u2f(u[i] & 0xFFFF0000u);
    }
    uint4 xv[TB];
#pragma unroll
    for (int t = 0; t < TB; ++t)
      xv[t] = *reinterpret_cast<const uint4*>(x + (size_t)(t < nt ? t : 0) * H + k);
#pragma unroll
    for (int t = 0; t < TB; ++t) {
      const uint32_t u[4] = {xv[t].x, xv[t].y, xv[t].z, xv[t].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[t] = __builtin_fmaf(u2f(u[i] << 16), w[2 * i], acc[t]);
        acc[t] = __builtin_fmaf(u2f(u[i] & 0xFFFF0000u), w[2 * i + 1], acc[t]);
      }
    }
  }
}

// Expert e's logits of tokens [t0, t0 + nt) by one workgroup of 256 threads;
// s_red: 4 * TB floats of LDS.
template <bool WF32, int TB>
__device__ __forceinline__ void gate_dot_expert(const void* __restrict__ w, const uint16_t* __restrict__ x, int e,
                                                int t0, int nt, int E, int H, float* __restrict__ logits,
                                                float* s_red) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  float acc[TB];
  gate_dot<WF32, TB>(static_cast<const uint8_t*>(w) + (size_t)e * H * (WF32 ? 4 : 2), x + (size_t)t0 * H, nt, H, tid,
                     acc);
#pragma unroll
  for (int t = 0; t < TB; ++t) {
    const float s = wave_sum(acc[t]);
    if (lane == 0) s_red[wave * TB + t] = s;
  }
  __syncthreads();
  if (tid < nt)
    logits[(size_t)(t0 + tid) * E + e] = (s_red[tid] + s_red[TB + tid]) + (s_red[2 * TB + tid] + s_red[3 * TB + tid]);
}

}  // namespace moefp4
