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

// The top_k + extra experts by sel, in descending order: take(j, who, wi, top)
// for place j, held by lane `who` as its element wi.  extra: one more place is
// found than is needed (its value only bounds the last gap).  Stops early
// where nothing above -inf is left.
template <int NI, class S, class F>
__device__ __forceinline__ void take_top(S (&sel)[NI], int n, int lane, F&& take) {
  const S kNone = (S)-__builtin_inff();
  for (int j = 0; j < n; ++j) {
    S best = sel[0];
    int bi = 0;
#pragma unroll
    for (int i = 1; i < NI; ++i)
      if (sel[i] > best) best = sel[i], bi = i;
    const S top = wave_max(best);
    if (!(top > kNone)) break;
    const int who = __builtin_ctzll(ballot(best == top));
    const int wi = __builtin_amdgcn_readlane(bi, who);
    take(j, who, wi, top);
    if (lane == who) {
#pragma unroll
      for (int i = 0; i < NI; ++i)
        if (i == wi) sel[i] = kNone;
    }
  }
}

// The 64-bit selection of gate_select's biased form: the expert and score of
// place j to lane j.  (No loop over the lane's experts that is not unrolled: the
// arrays would be indexed in memory, for which every launch of the few-token
// layer, with or without such a token, pays 6 to 11 us at its start.)
template <int NI>
__device__ __forceinline__ void gate_select64(const float (&l)[NI], const float (&bias)[NI], const GateSel& g, int lane,
                                              int* expert, float* score) {
  const double kNone = -__builtin_inf();
  const bool softmax = g.scoring == MOEFP4_SCORE_SOFTMAX;
  double m = kNone, sum = 0, p[NI], sel[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i)
    if (lane * NI + i < g.E && __builtin_isfinite(l[i])) m = max_of(m, (double)l[i]);
  if (softmax) m = wave_max(m);
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const bool fin = lane * NI + i < g.E && __builtin_isfinite(l[i]);
    const double x = exp(softmax ? (double)l[i] - m : -(double)l[i]);
    p[i] = !fin ? 0.0 : softmax ? x : 1.0 / (1.0 + x);
    sum += p[i];
  }
  const double inv = softmax ? 1.0 / wave_sum(sum) : 1.0;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    p[i] *= inv;
    const double s = p[i] + (double)bias[i];
    sel[i] = lane * NI + i < g.E && __builtin_isfinite(l[i]) && s > kNone ? s : kNone;
  }
  int my = -1;
  float mine = 0.0f;
  take_top<NI>(sel, g.top_k, lane, [&](int j, int who, int wi, double) __attribute__((always_inline)) {
    float ps = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (i == wi) ps = (float)p[i];
    const float at = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, ps), who));
    if (lane == j) mine = at, my = who * NI + wi;
  });
  *expert = my;
  *score = mine;
}

// The lane's biases, for gate_select: requested before the logits, so that one
// wait serves both.
template <int NI>
__device__ __forceinline__ void gate_bias(const GateSel& g, int lane, float (&bias)[NI]) {
#pragma unroll
  for (int i = 0; i < NI; ++i) bias[i] = 0.0f;
  if (g.bias) {
#pragma unroll
    for (int i = 0; i < NI; ++i) bias[i] = g.bias[min(lane * NI + i, g.E - 1)];
  }
}

// Selects the experts of one token.  Lane l holds the logits of experts
// l * NI + i, so that among equal scores the lowest lane, and in it the
// lowest i, is the lowest expert index.  score = softmax over the finite
// logits, or sigmoid; selection by score + bias, or without a bias by score alone,
// for which the logits themselves are compared (both scores grow with the
// logit).  Experts whose logit is not finite, or whose score + bias is NaN or
// -inf, are never selected; when none is left the remaining places get id -1
// and weight 0.
//
// With a bias two scores can be closer than the FP32 rounding of the
// exponential, and the experts a token takes should not depend on that
// rounding: FP32 decides where every gap between the places in turn (and
// behind the last one) is wider than 2^-20 of the larger of 1 and the score,
// several times what expf, the division and the addition can be off together;
// a token with a narrower gap (about 1 in 300 of 256 sigmoid scores) is
// selected again in 64 bits.  (All in 64 bits: 26 us against 17 us for 8192
// tokens of 256 experts.)
//
// l: the lane's logits; bias: gate_bias.
// emit(j, id, weight) is called by lane j with place j's expert and its
// weight: the score, divided by the selected scores' sum if renorm, times
// scale.
//
// The quotient of two scores can be an ordinary number where the scores
// themselves are below FP32's range (sigmoids of logits below -87, softmax
// scores beside masked experts that hold all of the mass).  Below a sum of
// 2^-100 the weights are formed from the logits, relative to the largest
// selected one: a softmax's scores are e^l times the same factor, and so are
// sigmoids down there (1 + e^l is 1 to 2^-100).
template <int NI, class F>
__device__ __forceinline__ void gate_select(const float (&l)[NI], const float (&bias)[NI], const GateSel& g, int lane,
                                            F&& emit) {
  const float kNone = -__builtin_inff();
  const bool softmax = g.scoring == MOEFP4_SCORE_SOFTMAX, biased = g.bias != nullptr;
  float p[NI], sel[NI];
  bool fin[NI];
  float m = kNone, inv = 1.0f;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int e = lane * NI + i;
    fin[i] = e < g.E && __builtin_isfinite(l[i]);
    if (fin[i]) m = max_of(m, l[i]);
  }
  if (softmax) m = wave_max(m);
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    // e^(l - m) of the softmax, or e^-l of the sigmoid
    // (for every expert, with no branch)
    const float x = expf(softmax ? l[i] - m : -l[i]), y = 1.0f / (1.0f + x);
    p[i] = fin[i] ? softmax ? x : y : 0.0f;
    sum += p[i];
  }
  if (softmax) inv = 1.0f / wave_sum(sum);
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    p[i] *= inv;
    const float s = biased ? p[i] + bias[i] : l[i];
    sel[i] = fin[i] && s > kNone ? s : kNone;  // (false for NaN)
  }
  float mine = 0.0f;  // the score of the place this lane holds
  int my = -1;        // and its expert
  float prev = 0.0f;
  bool narrow = false;
  // (biased: one place more than needed, for the gap behind the last one)
  take_top<NI>(sel, biased ? g.top_k + 1 : g.top_k, lane, [&](int j, int who, int wi, float top)
                                                             __attribute__((always_inline)) {
    if (biased && j > 0 && !(prev - top > 0x1p-20f * max_of(1.0f, __builtin_fabsf(prev)))) narrow = true;
    prev = top;
    float ps = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (i == wi) ps = p[i];
    ps = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, ps), who));
    if (lane == j && j < g.top_k) mine = ps, my = who * NI + wi;
  });
  if (narrow) gate_select64<NI>(l, bias, g, lane, &my, &mine);
  float f = g.scale;
  if (g.renorm) {
    float total = wave_sum(mine);  // (lanes without a place hold 0)
    if (total < 0x1p-100f) {
      float z = kNone;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const float v = __shfl(l[i], my < 0 ? 0 : my / NI, 64);
        if (my >= 0 && my % NI == i) z = v;
      }
      const float most = wave_max(z);
      mine = my >= 0 ? expf(z - most) : 0.0f;
      total = wave_sum(mine);
    }
    f = total > 0.0f ? f / total : 0.0f;
    if (!__builtin_isfinite(f)) mine /= total, f = g.scale;  // (the weights are at most the scale)
  }
  if (lane < g.top_k) emit(lane, my, mine * f);
}

// One expert's logits of tokens [t0, t0 + nt), nt <= TB, by one workgroup of
// 256 threads: logits[t][e] = sum over K, 8 elements of a strip of 2048 per
// thread, the strips' loads issued together (latency is all there is to hide
// where few tokens are routed).  s_red: 4 * TB floats of LDS.
template <bool WF32, int TB>
__device__ __forceinline__ void gate_dot_expert(const void* __restrict__ w, const uint16_t* __restrict__ x, int e,
                                                int t0, int nt, int ld, int H, float* __restrict__ logits,
                                                float* s_red) {
  constexpr int NS = TB >= 8 ? 1 : TB >= 4 ? 2 : 4;  // strips in flight
  constexpr int WV = WF32 ? 2 : 1;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const uint8_t* wr = static_cast<const uint8_t*>(w) + (size_t)e * H * (WF32 ? 4 : 2);
  x += (size_t)t0 * H;
  float acc[TB];
#pragma unroll
  for (int t = 0; t < TB; ++t) acc[t] = 0.0f;
  for (int k0 = tid * 8; k0 < H; k0 += 2048 * NS) {
    uint4 wv[NS][WV], xv[NS][TB];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int k = k0 + 2048 * s;
#pragma unroll
      for (int i = 0; i < WV; ++i) wv[s][i] = uint4{0u, 0u, 0u, 0u};
#pragma unroll
      for (int t = 0; t < TB; ++t) xv[s][t] = uint4{0u, 0u, 0u, 0u};
      if (s == 0 || k < H) {
#pragma unroll
        for (int i = 0; i < WV; ++i) wv[s][i] = *reinterpret_cast<const uint4*>(wr + (size_t)k * (WF32 ? 4 : 2) + 16 * i);
#pragma unroll
        for (int t = 0; t < TB; ++t)
          if (t < nt) xv[s][t] = *reinterpret_cast<const uint4*>(x + (size_t)t * H + k);
      }
    }
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      float wf[8];
      if constexpr (WF32) {
        const uint32_t u[8] = {wv[s][0].x, wv[s][0].y, wv[s][0].z, wv[s][0].w,
                               wv[s][1].x, wv[s][1].y, wv[s][1].z, wv[s][1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) wf[i] = u2f(u[i]);
      } else {
        const uint32_t u[4] = {wv[s][0].x, wv[s][0].y, wv[s][0].z, wv[s][0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) wf[2 * i] = u2f(u[i] << 16), wf[2 * i + 1] = u2f(u[i] & 0xFFFF0000u);
      }
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        const uint32_t u[4] = {xv[s][t].x, xv[s][t].y, xv[s][t].z, xv[s][t].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[t] = __builtin_fmaf(u2f(u[i] << 16), wf[2 * i], acc[t]);
          acc[t] = __builtin_fmaf(u2f(u[i] & 0xFFFF0000u), wf[2 * i + 1], acc[t]);
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < TB; ++t) {
    const float s = wave_sum(acc[t]);
    if (lane == 0) s_red[wave * TB + t] = s;
  }
  __syncthreads();
  if (tid < nt)
    logits[(size_t)(t0 + tid) * ld + e] = (s_red[tid] + s_red[TB + tid]) + (s_red[2 * TB + tid] + s_red[3 * TB + tid]);
}

}  // namespace moefp4
