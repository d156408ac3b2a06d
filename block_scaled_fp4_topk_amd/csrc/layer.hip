// A whole mixture-of-experts layer for at most 16 tokens, in two launches:
// router logits, then one persistent kernel that selects the experts, runs
// FC1 + SwiGLU and FC2 over their FP4 weights and writes the weighted sum.
//
// With so few tokens the layer is a stream of weights (an expert's FP4 codes
// and scales, read once) and what costs beside it are the dependences: token
// -> experts -> h -> output.  Decisions that follow from that:
//
// * Every activation a wavefront needs for FC1 stays in its registers.  A
//   wave owns a fixed slice of H (1/8 of it: at most 3 chunks of 256), whose
//   MFMA operands for all 16 token columns are loaded once (32 registers per
//   chunk) and serve every expert; the weights come straight from HBM into
//   registers, are decoded there and multiplied.  No operand passes through
//   LDS; it only sums the 8 waves' partial tiles.  Columns of tokens that did
//   not choose the expert are computed and dropped (the matrix instruction
//   has 16 columns anyway).
// * Each chunk's registers are refilled with the same chunk of the next item
//   as soon as it is consumed, so that 8 waves keep a whole item (up to 110 KB
//   per CU) in flight.
// * FC1 items (an expert's 16 gate rows and the 16 matching up rows) are
//   claimed from one counter; no workgroup waits before every item has been
//   claimed by a workgroup that is running and finishes it without waiting:
//   however few workgroups are resident, every wait ends.  (The wait is
//   bounded all the same, as the single-launch forward's.)
// * FC2's work is split evenly by workgroup number: row blocks of 32 outputs
//   x steps of 8 (expert, chunk) units, one per wave, laid end to end and cut
//   into equal runs.  A workgroup's first weights are requested before it
//   waits for FC1.  Router weights are applied per unit, so that a row block's
//   accumulators hold the output itself; where a run's border cuts a row
//   block, its parts are summed in run order by whichever workgroup ends last
//   (no atomics on values: the result does not depend on timing).
// * What passes between workgroups of one launch (h, parts, counters) goes
//   through agent-scope accesses, which do not stay in an XCD's L2.
//
// h keeps more than bfloat16: group16 weights multiply in fp16, h as fp16 with
// one power of two per 16 values (11 significant bits); group32 weights
// multiply in bfloat16, h as a high and a low part (16 bits), two
// instructions per product.  The output's own rounding (8 bits) dominates.
#include "gate_core.h"

namespace moefp4 {

namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;

// Longest wait for FC1, in ticks of the 100 MHz real-time counter (50 ms).
constexpr uint64_t kFewMaxWait = 5000000;

// bf16 row -> fp16 * 2**-p (exact down to 2**-24 of the row's maximum, which
// lands in [2**14, 2**15)) by 256 threads.
__device__ void few_row_to_f16(const uint16_t* __restrict__ row, int H, uint16_t* __restrict__ out, float* scale) {
  __shared__ uint32_t s_max[4];
  const int tid = threadIdx.x;
  uint32_t m = 0;
  for (int i = tid * 8; i < H; i += 2048) {
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
  const float inv = __builtin_ldexpf(1.0f, -p);
  for (int i = tid * 8; i < H; i += 2048) {
    const uint4 v = *reinterpret_cast<const uint4*>(row + i);
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const _Float16 lo = (_Float16)(bf16_to_f32(w[j] & 0xFFFFu) * inv);
      const _Float16 hi = (_Float16)(bf16_to_f32(w[j] >> 16) * inv);
      w[j] = (uint32_t)__builtin_bit_cast(uint16_t, lo) | ((uint32_t)__builtin_bit_cast(uint16_t, hi) << 16);
    }
    *reinterpret_cast<uint4*>(out + i) = uint4{w[0], w[1], w[2], w[3]};
  }
  if (tid == 0) *scale = __builtin_ldexpf(1.0f, p);
}

// Launch 1: router logits (one workgroup per expert and TB tokens), the fp16
// rows (one workgroup per token), and the counters of launch 2 cleared.
template <bool WF32, int TB>
__global__ __launch_bounds__(256) void few_gate_kernel(FewArgs a) {
  __shared__ float s_red[4 * TB];
  const int nt = (a.T + TB - 1) / TB, nd = a.g.E * nt;
  const int b = blockIdx.x;
  if (b < nd) {
    const int t0 = (b % nt) * TB;
    gate_dot_expert<WF32, TB>(a.gate_w, a.x, b / nt, t0, min(TB, a.T - t0), a.ld, a.H, a.logits, s_red);
  } else if (b == nd) {
    for (int i = threadIdx.x; i < 2 + a.H / 32; i += 256) a.sync[i] = 0;
    if (threadIdx.x < 2) a.flags[threadIdx.x] = 0;
  } else {
    const int t = b - nd - 1;
    few_row_to_f16(a.x + (size_t)t * a.H, a.H, a.x16 + (size_t)t * a.H, a.xs + t);
  }
}

// Agent-scope accesses of launch 2's own exchanges.
__device__ __forceinline__ uint64_t ld_agent(const void* p) {
  return __hip_atomic_load(static_cast<const uint64_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void st_agent(void* p, uint64_t v) {
  __hip_atomic_store(static_cast<uint64_t*>(p), v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// float -> bf16 bits, round to nearest even, NaN kept.
__device__ __forceinline__ uint32_t bf16_bits(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

// LDS-only barrier: the waves' loads from memory stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}
__device__ __forceinline__ void drain_memory() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// A wave-uniform pointer in scalar registers, for loads with a 32-bit
// per-lane offset.
__device__ __forceinline__ const uint8_t* uniform_ptr(const uint8_t* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32));
  return reinterpret_cast<const uint8_t*>((uint64_t)lo | ((uint64_t)hi << 32));
}

// Two 16-row weight tiles x 256 K in registers: lane (r16, q) holds K [64 q,
// 64 q + 64) of row r16 of each (32 bytes of codes; 4 group16 or 2 group32
// scale bytes).
struct WPair {
  uint4 c[4];
  uint32_t s[2];
};

template <int MODE>
__device__ __forceinline__ void load_pair(WPair& w, const uint8_t* codes, uint32_t o0, uint32_t o1, const uint8_t* sf,
                                          uint32_t f0, uint32_t f1) {
  w.c[0] = ld_nt(codes + o0);
  w.c[1] = ld_nt(codes + o0 + 16);
  w.c[2] = ld_nt(codes + o1);
  w.c[3] = ld_nt(codes + o1 + 16);
  if (MODE == 0) {
    w.s[0] = *reinterpret_cast<const uint32_t*>(sf + f0);
    w.s[1] = *reinterpret_cast<const uint32_t*>(sf + f1);
  } else {
    w.s[0] = *reinterpret_cast<const uint16_t*>(sf + f0);
    w.s[1] = *reinterpret_cast<const uint16_t*>(sf + f1);
  }
}

__device__ __forceinline__ uint32_t dword(const uint4& v, int r) {
  return r == 0 ? v.x : r == 1 ? v.y : r == 2 ? v.z : v.w;
}

// acc[i] += tile i x B over the chunk; B(j): the operand of K [64 q + 8 j, + 8),
// NB of them per j (NB = 2: a high and a low part).
template <int MODE, int NB, class BF>
__device__ __forceinline__ void mfma_pair(const WPair& w, v4f (&acc)[2], BF&& B) {
  if constexpr (MODE == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const v2h lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w.s[i], 1.0f, false);
      const v2h hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w.s[i], 1.0f, true);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const _Float16 s = j < 2 ? lo[0] : j < 4 ? lo[1] : j < 6 ? hi[0] : hi[1];
        const v8h A = dq8_f16(dword(w.c[2 * i + (j >> 2)], j & 3), v2h{s, s});
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(A, __builtin_bit_cast(v8h, B(j, 0)), acc[i], 0, 0, 0);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float lo = ue8m0_to_f32(w.s[i] & 0xFFu), hi = ue8m0_to_f32(w.s[i] >> 8);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const v8bf A = dq8_bf16(dword(w.c[2 * i + (j >> 2)], j & 3), j < 4 ? lo : hi);
#pragma unroll
        for (int n = 0; n < NB; ++n)
          acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A, __builtin_bit_cast(v8bf, B(j, n)), acc[i], 0, 0, 0);
      }
    }
  }
}

// Launch 2.  MODE 0: group16 (fp16 products), 1: group32 (bf16); NC: chunks of
// H per wave.
template <int MODE, int NC>
__global__ __launch_bounds__(kThreads, 2) void few_layer_kernel(FewArgs a) {
  __shared__ float4 s_red[2][kWaves][2][64];
  __shared__ int s_ids[kFewTokens * kFewMaxK];
  __shared__ float s_tw[kFewTokens * kFewMaxK];
  __shared__ short s_rank[kMaxExperts], s_act[kMaxExperts];
  __shared__ uint8_t s_col[kMaxExperts * kFewTokens];  // [active][token]: place of the expert in the token's list
  __shared__ int s_cnt[kWaves], s_claim[2];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, q = lane >> 4;
  const int T = a.T, H = a.H, I = a.I, kt = a.g.top_k + a.g.shared;
  int32_t* const queue = a.sync;
  int32_t* const done = a.sync + 1;

  // the first claim does not need the selection
  if (tid == 0) s_claim[0] = __hip_atomic_fetch_add(queue, 2, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);

  // ---- selection, by every workgroup for itself
  for (int i = tid; i < kMaxExperts; i += kThreads) s_rank[i] = 0;
  for (int i = tid; i < kMaxExperts * kFewTokens / 4; i += kThreads) reinterpret_cast<uint32_t*>(s_col)[i] = ~0u;
  for (int t = wave; t < T; t += kWaves) {
    const float* row = a.logits + (size_t)t * a.ld;
    auto emit = [&](int j, int id, float w) __attribute__((always_inline)) {
      s_ids[t * kt + j] = id;
      s_tw[t * kt + j] = w;
    };
    if (a.ld <= 256) {
      float l[4];
      // (rows are padded to ld: lanes past it hold nothing)
      const float4 v = 4 * lane < a.ld ? *reinterpret_cast<const float4*>(row + 4 * lane) : float4{0.f, 0.f, 0.f, 0.f};
      l[0] = v.x, l[1] = v.y, l[2] = v.z, l[3] = v.w;
      if (a.g.bias) gate_select<4, true>(l, a.g, lane, emit);
      else gate_select<4, false>(l, a.g, lane, emit);
    } else {
      float l[8];
      const float4 u = *reinterpret_cast<const float4*>(row + 8 * lane);
      const float4 v = *reinterpret_cast<const float4*>(row + 8 * lane + 4);
      l[0] = u.x, l[1] = u.y, l[2] = u.z, l[3] = u.w, l[4] = v.x, l[5] = v.y, l[6] = v.z, l[7] = v.w;
      if (a.g.bias) gate_select<8, true>(l, a.g, lane, emit);
      else gate_select<8, false>(l, a.g, lane, emit);
    }
    for (int j = lane; j < a.g.shared; j += 64) {
      s_ids[t * kt + a.g.top_k + j] = a.g.E + j;
      s_tw[t * kt + a.g.top_k + j] = 1.0f;
    }
  }
  // this wave's activations (behind the selection: its registers are free now)
  const int nch = H >> 8;
  uint4 xb[NC][8];
  {
    const uint16_t* src = (MODE == 0 ? a.x16 : a.x) + (size_t)(r16 < T ? r16 : 0) * H + 64 * q;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int ck = wave * NC + i;
#pragma unroll
      for (int j = 0; j < 8; ++j) xb[i][j] = uint4{0u, 0u, 0u, 0u};
      if (ck < nch && r16 < T) {
#pragma unroll
        for (int j = 0; j < 8; ++j) xb[i][j] = *reinterpret_cast<const uint4*>(src + ck * 256 + 8 * j);
      }
    }
  }
  __syncthreads();
  int item = __builtin_amdgcn_readfirstlane(s_claim[0]), next = item + 1;
  for (int i = tid; i < T * kt; i += kThreads)
    if (s_ids[i] >= 0) s_rank[s_ids[i]] = 1;
  __syncthreads();
  // the active experts in ascending order (512 threads, an expert each)
  const uint64_t on = ballot(s_rank[tid] != 0);
  if (lane == 0) s_cnt[wave] = __popcll(on);
  __syncthreads();
  int nact = 0, before = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    before += w < wave ? s_cnt[w] : 0;
    nact += s_cnt[w];
  }
  nact = __builtin_amdgcn_readfirstlane(nact);
  if ((on >> lane) & 1) {
    const int rank = before + __popcll(on & ((1ull << lane) - 1ull));
    s_act[rank] = (short)tid;
    s_rank[tid] = (short)rank;
  }
  __syncthreads();
  int none = 0;
  for (int i = tid; i < T * kt; i += kThreads) {
    const int id = s_ids[i], t = i / kt;
    if (id >= 0) s_col[s_rank[id] * kFewTokens + t] = (uint8_t)(i - t * kt);
    if (blockIdx.x == 0) {
      none += id < 0;
      if (a.ids) a.ids[i] = id;
      if (a.wts) a.wts[i] = s_tw[i];
    }
  }
  if (none) atomicAdd(a.flags, none);
  __syncthreads();

  // ---- FC1 + SwiGLU: h
  const int npt = I >> 4;
  const int n1 = nact * npt;
  const uint32_t rowb = (uint32_t)(H >> 1), rows = (uint32_t)(MODE == 0 ? H >> 4 : H >> 5);
  const size_t A = (size_t)T * kt;
  WPair w1[NC];
  auto expert = [&](int act) __attribute__((always_inline)) { return __builtin_amdgcn_readfirstlane((int)s_act[act]); };
  auto load1 = [&](int item, int i, WPair& w) __attribute__((always_inline)) {
    const int ck = wave * NC + i;
    if (item < n1 && ck < nch) {
      const int act = item / npt, pt = item - act * npt, e = expert(act);
      const uint8_t* codes = uniform_ptr(a.w13 + (size_t)e * 2 * I * rowb);
      const uint8_t* sf = uniform_ptr(a.w13_sf + (size_t)e * 2 * I * rows);
      const uint32_t g0 = (uint32_t)(pt * 16 + r16) + (a.w13_order ? (uint32_t)I : 0u);
      const uint32_t u0 = (uint32_t)(pt * 16 + r16) + (a.w13_order ? 0u : (uint32_t)I);
      const uint32_t co = (uint32_t)(ck * 128 + 32 * q), so = MODE == 0 ? ck * 16 + 4 * q : ck * 8 + 2 * q;
      load_pair<MODE>(w, codes, g0 * rowb + co, u0 * rowb + co, sf, g0 * rows + so, u0 * rows + so);
    }
  };
  int buf = 0, mine = 0;
#pragma unroll
  for (int i = 0; i < NC; ++i) load1(item, i, w1[i]);
  while (item < n1) {
    int claim = 0;
    if (wave == 0) claim = __hip_atomic_fetch_add(queue, lane == 0 ? 1 : 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    v4f acc[2] = {v4f{0.f, 0.f, 0.f, 0.f}, v4f{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (wave * NC + i < nch)
        mfma_pair<MODE, 1>(w1[i], acc, [&](int j, int) __attribute__((always_inline)) { return xb[i][j]; });
      load1(next, i, w1[i]);
    }
    s_red[buf][wave][0][lane] = float4{acc[0][0], acc[0][1], acc[0][2], acc[0][3]};
    s_red[buf][wave][1][lane] = float4{acc[1][0], acc[1][1], acc[1][2], acc[1][3]};
    if (wave == 0) s_claim[buf] = __builtin_amdgcn_readfirstlane(claim);
    lds_barrier();
    const int after = __builtin_amdgcn_readfirstlane(s_claim[buf]);
    if (wave == (mine & (kWaves - 1))) {
      // the waves take turns: sum, SwiGLU, store.  Lane: rows 4 q .. + 3, token r16.
      float g[4] = {0.f, 0.f, 0.f, 0.f}, u[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float4 gv = s_red[buf][w][0][lane], uv = s_red[buf][w][1][lane];
        g[0] += gv.x, g[1] += gv.y, g[2] += gv.z, g[3] += gv.w;
        u[0] += uv.x, u[1] += uv.y, u[2] += uv.z, u[3] += uv.w;
      }
      const int act = item / npt, pt = item - act * npt, e = expert(act);
      const float cs = (a.w13_gs ? a.w13_gs[e] : 1.0f) * (MODE == 0 && r16 < T ? a.xs[r16] : 1.0f);
      const int col = s_col[act * kFewTokens + r16];
      float h[4];
      float amax = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[i] = swiglu(g[i] * cs, u[i] * cs);
        amax = fmaxf(amax, fabsf(h[i]));
      }
      // K [16 pt + 4 q, + 4) in the order FC2's lanes read a chunk: [j][q'][8]
      // for K = 64 q' + 8 j + (0 .. 7)
      const int kk = (pt & 15) * 16 + 4 * q;
      const size_t slot = (size_t)r16 * kt + col;
      const size_t at = slot * I + (size_t)(pt >> 4) * 256 + ((kk >> 3) & 7) * 32 + (kk >> 6) * 8 + (kk & 4);
      if constexpr (MODE == 0) {
        amax = fmaxf(amax, __shfl_xor(amax, 16, 64));
        amax = fmaxf(amax, __shfl_xor(amax, 32, 64));
        int p = (int)(f2u(amax) >> 23) - 127 - 14;
        p = p < -128 ? -128 : p;
        uint64_t v = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v |= (uint64_t)__builtin_bit_cast(uint16_t, (_Float16)__builtin_ldexpf(h[i], -p)) << (16 * i);
        if (r16 < T && col != 255) {
          st_agent(a.h + at, v);
          if (q == 0)
            __hip_atomic_store(a.hexp + slot * (I >> 4) + pt, (int8_t)p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
      } else {
        uint64_t hi = 0, lo = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t b = bf16_bits(h[i]);
          hi |= (uint64_t)b << (16 * i);
          if (__builtin_isfinite(h[i])) lo |= (uint64_t)bf16_bits(h[i] - bf16_to_f32(b)) << (16 * i);
        }
        if (r16 < T && col != 255) {
          st_agent(a.h + at, hi);
          st_agent(a.h + A * I + at, lo);
        }
      }
    }
    ++mine;
    buf ^= 1;
    item = next;
    next = after;
  }

  // ---- FC2: this workgroup's run of steps
  const int nch2 = I >> 8, units = nact * nch2;
  const int ns = units > kWaves ? (units + kWaves - 1) / kWaves : 1;
  const int nrb = H >> 5;
  const long long total = (long long)nrb * ns;
  const int G = a.nwg < total ? a.nwg : (int)total;
  const int wg = blockIdx.x;
  drain_memory();  // this wave's stores of h are complete
  const bool works = wg < G;
  const long long begin = works ? wg * total / G : 0, end = works ? (wg + 1) * total / G : 0;
  const uint32_t rowb2 = (uint32_t)(I >> 1), rows2 = (uint32_t)(MODE == 0 ? I >> 4 : I >> 5);
  constexpr int NB = MODE == 0 ? 1 : 2;
  constexpr int NS = MODE == 0 ? 3 : 2;  // steps in flight (what the registers hold)
  WPair w2[NS];
  uint2 hb[NS][8 * NB][2];
  uint32_t hx[NS];
  // the (row block, step) walked by the loads, and by the products
  struct Pos { int rb, st; };
  auto advance = [&](Pos& p) __attribute__((always_inline)) {
    if (++p.st == ns) p.st = 0, ++p.rb;
  };
  Pos lw = {(int)(begin / ns), (int)(begin % ns)}, lh = lw, pc = lw;
  auto load_w2 = [&](const Pos& p, WPair& w) __attribute__((always_inline)) {
    const int f = p.st * kWaves + wave;
    if (f < units) {
      const int act = f / nch2, c = f - act * nch2, e = expert(act);
      const uint8_t* codes = uniform_ptr(a.w2 + (size_t)e * H * rowb2);
      const uint8_t* sf = uniform_ptr(a.w2_sf + (size_t)e * H * rows2);
      const uint32_t r0 = (uint32_t)(p.rb * 32 + r16), r1 = r0 + 16;
      const uint32_t co = (uint32_t)(c * 128 + 32 * q), so = MODE == 0 ? c * 16 + 4 * q : c * 8 + 2 * q;
      load_pair<MODE>(w, codes, r0 * rowb2 + co, r1 * rowb2 + co, sf, r0 * rows2 + so, r1 * rows2 + so);
    }
  };
  auto load_h = [&](const Pos& p, uint2 (&b)[8 * NB][2], uint32_t& x) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 8 * NB; ++j) b[j][0] = b[j][1] = uint2{0u, 0u};
    x = 0x80808080u;
    const int f = p.st * kWaves + wave;
    if (f < units) {
      const int act = f / nch2, c = f - act * nch2;
      const int col = s_col[act * kFewTokens + r16];
      if (col != 255) {
        const size_t slot = (size_t)r16 * kt + col;
        const uint16_t* src = a.h + slot * I + c * 256 + 8 * q;
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            b[8 * n + j][0] = __builtin_bit_cast(uint2, ld_agent(src + n * A * I + 32 * j));
            b[8 * n + j][1] = __builtin_bit_cast(uint2, ld_agent(src + n * A * I + 32 * j + 4));
          }
        if (MODE == 0)
          x = __hip_atomic_load(reinterpret_cast<const uint32_t*>(a.hexp + slot * (I >> 4) + c * 16 + 4 * q),
                                __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
  };
  long long ahead = begin;
#pragma unroll
  for (int s = 0; s < NS; ++s)
    if (begin + s < end) {
      load_w2(lw, w2[s]);
      advance(lw);
      ++ahead;
    }
  lds_barrier();  // (every wave's stores are complete)
  if (wave == 0 && (works || mine)) {
    if (mine) __hip_atomic_fetch_add(done, lane == 0 ? mine : 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const uint64_t t0 = __builtin_amdgcn_s_memrealtime();
    while (works) {
      const int d =
          __builtin_amdgcn_readfirstlane(__hip_atomic_load(done, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
      if (d >= n1) break;
      if (__builtin_amdgcn_s_memrealtime() - t0 > kFewMaxWait) {
        __hip_atomic_fetch_add(a.flags + 1, lane == 0 ? 1 : 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        break;
      }
      __builtin_amdgcn_s_sleep(1);
    }
  }
  lds_barrier();
#pragma unroll
  for (int s = 0; s < NS; ++s)
    if (begin + s < end) {
      load_h(lh, hb[s], hx[s]);
      advance(lh);
    }

  float oacc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  int first = 1;  // still in the run's first row block
  int turn = 0;
  // the row block's sum over the waves, and on to the output: directly where
  // the run holds the whole block, else through the parts
  auto flush = [&](int rb) __attribute__((always_inline)) {
    s_red[buf][wave][0][lane] = float4{oacc[0], oacc[1], oacc[2], oacc[3]};
    s_red[buf][wave][1][lane] = float4{oacc[4], oacc[5], oacc[6], oacc[7]};
#pragma unroll
    for (int i = 0; i < 8; ++i) oacc[i] = 0.0f;
    lds_barrier();
    if (wave == (turn & (kWaves - 1))) {
      float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float4 u = s_red[buf][w][0][lane], v = s_red[buf][w][1][lane];
        o[0] += u.x, o[1] += u.y, o[2] += u.z, o[3] += u.w;
        o[4] += v.x, o[5] += v.y, o[6] += v.z, o[7] += v.w;
      }
      const long long s0 = (long long)rb * ns, s1 = s0 + ns;
      bool write = true;
      if (begin > s0 || end < s1) {
        float* mypart = a.part + ((size_t)wg * 2 + (first ? 0 : 1)) * 512 + lane * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) st_agent(mypart + 2 * i, (uint64_t)f2u(o[2 * i]) | ((uint64_t)f2u(o[2 * i + 1]) << 32));
        drain_memory();
        // owners of the block's first and last step (the last w with w total / G <= step)
        const int o0 = (int)(((s0 + 1) * G - 1) / total), o1 = (int)((s1 * G - 1) / total);
        const int arrived = __builtin_amdgcn_readfirstlane(
            __hip_atomic_fetch_add(a.sync + 2 + rb, lane == 0 ? 1 : 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
        write = arrived == o1 - o0;
        if (write) {
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = 0.0f;
          for (int w = o0; w <= o1; ++w) {
            const bool head = (w * total / G) / ns == rb;  // the block is run w's first
            const float* p = a.part + ((size_t)w * 2 + (head ? 0 : 1)) * 512 + lane * 8;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint64_t v = ld_agent(p + 2 * i);
              o[2 * i] += u2f((uint32_t)v);
              o[2 * i + 1] += u2f((uint32_t)(v >> 32));
            }
          }
        }
      }
      if (write && r16 < T) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const size_t at = (size_t)r16 * H + rb * 32 + 16 * i + 4 * q;
          if (a.out_f32)
            *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) =
                float4{o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]};
          else
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
                uint2{bf16_bits(o[4 * i]) | (bf16_bits(o[4 * i + 1]) << 16),
                      bf16_bits(o[4 * i + 2]) | (bf16_bits(o[4 * i + 3]) << 16)};
        }
      }
    }
    ++turn;
    buf ^= 1;
    first = 0;
  };
  for (long long s = begin; s < end; s += NS) {
#pragma unroll
    for (int k = 0; k < NS; ++k) {
      if (s + k < end) {
        const int f = pc.st * kWaves + wave;
        if (f < units) {
          const int act = f / nch2, e = expert(act);
          const int col = s_col[act * kFewTokens + r16];
          float cs = a.w2_gs ? a.w2_gs[e] : 1.0f;
          v4f acc[2] = {v4f{0.f, 0.f, 0.f, 0.f}, v4f{0.f, 0.f, 0.f, 0.f}};
          if constexpr (MODE == 0) {
            // the chunk's largest exponent P; each 16-block's values times 2**(p - P)
            const int p0 = (int)(int8_t)(hx[k] & 0xFFu), p1 = (int)(int8_t)((hx[k] >> 8) & 0xFFu);
            const int p2 = (int)(int8_t)((hx[k] >> 16) & 0xFFu), p3 = (int)(int8_t)(hx[k] >> 24);
            int P = max(max(p0, p1), max(p2, p3));
            P = max(P, __shfl_xor(P, 16, 64));
            P = max(P, __shfl_xor(P, 32, 64));
            cs = __builtin_ldexpf(cs, P);
            const _Float16 fb[4] = {(_Float16)__builtin_ldexpf(1.0f, p0 - P), (_Float16)__builtin_ldexpf(1.0f, p1 - P),
                                    (_Float16)__builtin_ldexpf(1.0f, p2 - P), (_Float16)__builtin_ldexpf(1.0f, p3 - P)};
            mfma_pair<MODE, 1>(w2[k], acc, [&](int j, int) __attribute__((always_inline)) {
              const uint4 v = {hb[k][j][0].x, hb[k][j][0].y, hb[k][j][1].x, hb[k][j][1].y};
              return __builtin_bit_cast(v8h, v) * fb[j >> 1];
            });
          } else {
            mfma_pair<MODE, 2>(w2[k], acc, [&](int j, int n) __attribute__((always_inline)) {
              return uint4{hb[k][8 * n + j][0].x, hb[k][8 * n + j][0].y, hb[k][8 * n + j][1].x, hb[k][8 * n + j][1].y};
            });
          }
          if (col != 255) {
            cs *= s_tw[r16 * kt + col];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              oacc[i] = __builtin_fmaf(acc[0][i], cs, oacc[i]);
              oacc[4 + i] = __builtin_fmaf(acc[1][i], cs, oacc[4 + i]);
            }
          }
        }
        if (ahead < end) {
          load_w2(lw, w2[k]);
          load_h(lw, hb[k], hx[k]);
          advance(lw);
          ++ahead;
        }
        const int rb = pc.rb;
        advance(pc);
        if (pc.st == 0 || s + k + 1 == end) flush(rb);
      }
    }
  }
}

template <int MODE>
void launch_layer(const FewArgs& a, hipStream_t s) {
  const int nc = (a.H / 256 + kWaves - 1) / kWaves;
  const dim3 grid(a.nwg), block(kThreads);
  if (nc <= 1) hipLaunchKernelGGL((few_layer_kernel<MODE, 1>), grid, block, 0, s, a);
  else if (nc == 2) hipLaunchKernelGGL((few_layer_kernel<MODE, 2>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((few_layer_kernel<MODE, 3>), grid, block, 0, s, a);
}

template <bool WF32>
void launch_gate_part(const FewArgs& a, hipStream_t s) {
  const int tb = a.T == 1 ? 1 : a.T <= 4 ? 4 : 8;
  const int nt = (a.T + tb - 1) / tb;
  const dim3 grid(a.g.E * nt + 1 + (a.g16 ? a.T : 0));
  if (tb == 1) hipLaunchKernelGGL((few_gate_kernel<WF32, 1>), grid, dim3(256), 0, s, a);
  else if (tb == 4) hipLaunchKernelGGL((few_gate_kernel<WF32, 4>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((few_gate_kernel<WF32, 8>), grid, dim3(256), 0, s, a);
}

}  // namespace

int cu_count() {
  int dev = 0, cus = 0;
  if (hipGetDevice(&dev) != hipSuccess ||
      hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus < 1)
    return 256;
  return cus;
}

hipError_t launch_few(const FewArgs& a, hipStream_t s) {
  if (a.w_f32) launch_gate_part<true>(a, s);
  else launch_gate_part<false>(a, s);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  if (a.g16) launch_layer<0>(a, s);
  else launch_layer<1>(a, s);
  return hipGetLastError();
}

}  // namespace moefp4
