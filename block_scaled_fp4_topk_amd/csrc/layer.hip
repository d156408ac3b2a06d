// A whole mixture-of-experts layer for at most 8 tokens (2 with group32
// weights), in two launches: router logits, then one persistent kernel that
// selects the experts, runs FC1 + SwiGLU and FC2 over their FP4 weights and
// writes the weighted sum.
//
// With so few tokens the layer is a stream of weights (an expert's FP4 codes
// and scales, read once) and what costs beside it are the dependences: token
// -> experts -> h -> output.  Decisions that follow from that:
//
// * Every activation a wavefront needs for FC1 stays in its registers.  A
//   wave owns a fixed slice of H (1/8 of it: at most 3 chunks of 256), whose
//   MFMA operands for all token columns are loaded once (32 registers per
//   chunk) and serve every expert.  The weights come from HBM into registers
//   as whole 128-byte lines, are turned into operand order through the wave's
//   own 4 KB of LDS (no barrier) and decoded on the way into the matrix
//   instruction.  Columns of tokens that did not choose the expert are computed
//   and dropped (the matrix instruction has 16 columns anyway).  The 8 waves'
//   partial tiles meet in LDS.
// * Each chunk's registers are refilled with the same chunk of the next item
//   as soon as it is consumed, so that 8 waves keep a whole item (up to 110 KB
//   per CU) in flight.
// * FC1 items (an expert's 16 gate rows and the 16 matching up rows) lie in
//   one queue per XCD; a workgroup claims from its own XCD's and, when that is
//   empty, from one that is not.  Whoever claims an item is running and
//   finishes it without waiting, and a claim that succeeds is followed by
//   another look at all queues: after the last one that succeeds there is
//   nothing left.  So every item is finished however few workgroups are
//   resident, and the wait for them ends.  (It is bounded all the same, as the
//   single-launch forward's; a workgroup that gives it up adds NaN.)
// * FC2's work is split evenly by workgroup number: row blocks of 32 outputs
//   x steps of 8 (expert, chunk) units, one per wave, laid end to end and cut
//   into equal runs.  A workgroup's first weights are requested before it
//   waits for FC1.  Router weights are applied per unit, so that a row block's
//   accumulators hold the output itself; where a run's border cuts a row
//   block, its parts are summed in run order by whichever workgroup ends last
//   (no atomics on values: the result does not depend on timing).
// * h, parts and counters are written past the caches of an XCD (agent-scope
//   stores, complete before the counter that reports them is raised).  Parts
//   and counters are read so too; h, which every workgroup reads, comes through
//   the caches, behind one acquire per workgroup: it drops what the CU's L1
//   and the XCD's L2 held of h before, and the barrier behind it holds the
//   other waves' reads back.
//
// h keeps more than bfloat16: group16 weights multiply in fp16, h as fp16 with
// one power of two per 16 values (11 significant bits, less below 2**-28 of the
// largest of 256 values); group32 weights multiply in bfloat16, h as a high and
// a low part (16 bits), two instructions per product.  The output's own
// rounding (8 bits) dominates.
#include "gate_core.h"

namespace moefp4 {

namespace {

constexpr int kWaves = 8;
constexpr int kQueues = kFewQueues, kLine = kFewLine;
constexpr int kCols = 16;                       // columns of a matrix instruction: tokens' places
constexpr int kActive = kFewTokens * kFewMaxK;  // most experts that have a token
constexpr int kThreads = 64 * kWaves;

// Stride in LDS of a token's h (256 values, 16 bytes of padding against bank
// conflicts).
constexpr int kHRow = 512 + 16;

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
    for (int i = threadIdx.x; i < 2 * kQueues * kLine + a.H / 32; i += 256) a.sync[i] = 0;
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

// The XCD (accelerator complex die) this wave runs on.
__device__ __forceinline__ int xcc_id() {
  unsigned v;
  asm volatile("s_getreg_b32 %0, hwreg(HW_REG_XCC_ID)" : "=s"(v));
  return (int)(v & 0xFu);
}

// n items of a queue, by one lane.  (The offset the compiler cannot see keeps
// it from merging the wave's lanes into one atomic, which waits for the result
// on the spot, and with it for every load before it.)
__device__ __forceinline__ int claim_from(int32_t* queue, int n) {
  int zero = 0;
  asm volatile("" : "+v"(zero));
  return __hip_atomic_fetch_add(queue + zero, n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// LDS-only barrier: the waves' loads from memory stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}
__device__ __forceinline__ void drain_memory() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// A wave-uniform pointer to memory in scalar registers, for loads with a
// 32-bit per-lane offset.  (The address space is kept in the type: a generic
// pointer's loads also count as LDS accesses, and the waits for LDS would then
// wait for every weight in flight: 62 us instead of 60 us for one token of the
// 256-expert layer.)
typedef const __attribute__((address_space(1))) uint8_t* GPtr;
__device__ __forceinline__ GPtr uniform_ptr(const uint8_t* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32));
  return (GPtr)((uint64_t)lo | ((uint64_t)hi << 32));
}
template <class V>
__device__ __forceinline__ V gload(GPtr p, uint32_t off) {
  return *(const __attribute__((address_space(1))) V*)(p + off);
}
__device__ __forceinline__ u32x4 gload_nt(GPtr p, uint32_t off) {
  return __builtin_nontemporal_load((const __attribute__((address_space(1))) u32x4*)(p + off));
}

// Two 16-row weight tiles x 256 K on their way: instruction j holds rows
// 8 (j & 1) + lane / 8 of tile j / 2, 16 bytes at 16 (lane & 7): eight whole
// 128-byte lines per instruction, marked non-temporal (measured on this
// stream, 104 experts: 7.0 TB/s; loads in the MFMA operand's own layout ask
// for half lines and reach 6.2 TB/s, 5.2 if non-temporal).  s: the scales of
// the lane's operand rows (r16 of each tile, K [64 q, 64 q + 64): 4 group16 or
// 2 group32 bytes).
struct WPair {
  u32x4 c[4];
  uint32_t s[2];
};

// Where a pair's rows lie: wave-uniform addresses of the two tiles' first rows
// (codes and scales).  The lane's place in a tile is the same for every tile:
// LaneOff.  Chunk c is c * 128 code and c * 16 (group16) or c * 8 scale bytes on.
struct WSrc {
  GPtr c0, c1, f0, f1;
};
struct LaneOff {
  uint32_t lo, hi, sf;  // rows lane / 8 and 8 + lane / 8, 16 bytes; scales of row r16
};
__device__ __forceinline__ LaneOff lane_offsets(int lane, uint32_t row_bytes, uint32_t sf_bytes, int mode) {
  const uint32_t lo = (lane >> 3) * row_bytes + 16 * (lane & 7);
  return LaneOff{lo, lo + 8 * row_bytes, (lane & 15) * sf_bytes + (lane >> 4) * (mode == 0 ? 4u : 2u)};
}

template <int MODE>
__device__ __forceinline__ void load_pair(WPair& w, const WSrc& s, const LaneOff& o, uint32_t c) {
  w.c[0] = gload_nt(s.c0 + c * 128, o.lo);
  w.c[1] = gload_nt(s.c0 + c * 128, o.hi);
  w.c[2] = gload_nt(s.c1 + c * 128, o.lo);
  w.c[3] = gload_nt(s.c1 + c * 128, o.hi);
  if (MODE == 0) {
    w.s[0] = gload<uint32_t>(s.f0 + c * 16, o.sf);
    w.s[1] = gload<uint32_t>(s.f1 + c * 16, o.sf);
  } else {
    w.s[0] = gload<uint16_t>(s.f0 + c * 8, o.sf);
    w.s[1] = gload<uint16_t>(s.f1 + c * 8, o.sf);
  }
}

// The codes turned into operand order through the wave's own 4 KB of LDS (no
// barrier: a wave's LDS accesses stay in order): row r's 16-byte segment s
// sits at s ^ ((r >> 1) & 7), which spreads the 16 rows of a read over all
// banks.  at: the lane's write offsets of instructions 0 and 1 and read offsets
// of its two segments.
struct Turn {
  uint32_t w0, w1, r0, r1;
};
__device__ __forceinline__ Turn turn_offsets(int lane) {
  const int r16 = lane & 15, q = lane >> 4, wr = lane >> 3, seg = lane & 7;
  Turn t;
  t.w0 = wr * 128 + 16 * (seg ^ (wr >> 1));
  t.w1 = (wr + 8) * 128 + 16 * (seg ^ ((wr + 8) >> 1));
  t.r0 = r16 * 128 + 16 * ((2 * q) ^ (r16 >> 1));
  t.r1 = r16 * 128 + 16 * ((2 * q + 1) ^ (r16 >> 1));
  return t;
}
__device__ __forceinline__ void turn_pair(WPair& w, uint8_t* lds, const Turn& t) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    *reinterpret_cast<u32x4*>(lds + 2048 * i + t.w0) = w.c[2 * i];
    *reinterpret_cast<u32x4*>(lds + 2048 * i + t.w1) = w.c[2 * i + 1];
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w.c[2 * i] = *reinterpret_cast<const u32x4*>(lds + 2048 * i + t.r0);
    w.c[2 * i + 1] = *reinterpret_cast<const u32x4*>(lds + 2048 * i + t.r1);
  }
}

// The pair is used from here on: its decoding does not move up in front of
// other pairs' products, where it would wait for its loads too early.
__device__ __forceinline__ void use_from_here(WPair& w) {
  asm volatile("" : "+v"(w.c[0]), "+v"(w.c[1]), "+v"(w.c[2]), "+v"(w.c[3]), "+v"(w.s[0]), "+v"(w.s[1]));
}

// acc[i] += tile i x B over the chunk; B(j): the operand of K [64 q + 8 j, + 8),
// NB of them per j (NB = 2: a high and a low part).
template <int MODE, int NB, class BF>
__device__ __forceinline__ void mfma_pair(const WPair& w, v4f (&acc)[2], BF&& B) {
  if constexpr (MODE == 0) {
    v2h sc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      sc[i][0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w.s[i], 1.0f, false);
      sc[i][1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w.s[i], 1.0f, true);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const v8h b = __builtin_bit_cast(v8h, B(j, 0));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const _Float16 s = sc[i][j >> 2][(j >> 1) & 1];
        const v8h A = dq8_f16(w.c[2 * i + (j >> 2)][j & 3], v2h{s, s});
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(A, b, acc[i], 0, 0, 0);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v8bf b[NB];
#pragma unroll
      for (int n = 0; n < NB; ++n) b[n] = __builtin_bit_cast(v8bf, B(j, n));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const v8bf A = dq8_bf16(w.c[2 * i + (j >> 2)][j & 3], ue8m0_to_f32((w.s[i] >> (8 * (j >> 2))) & 0xFFu));
#pragma unroll
        for (int n = 0; n < NB; ++n) acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A, b[n], acc[i], 0, 0, 0);
      }
    }
  }
}

// Launch 2.  MODE 0: group16 (fp16 products), 1: group32 (bf16); NC: chunks of
// H per wave; NI: router logits per lane.
template <int MODE, int NC, int NI>
__global__ __launch_bounds__(kThreads, 2) void few_layer_kernel(FewArgs a) {
  __shared__ float4 s_red[2][kWaves][2][64];
  __shared__ __attribute__((aligned(16))) uint8_t s_turn[kWaves][4096];
  __shared__ __attribute__((aligned(16))) uint8_t s_h[kWaves][4 * kHRow];
  __shared__ int s_ids[kActive];
  __shared__ float s_tw[kActive];
  // per active expert: its id and tokens, and per token
  __shared__ short s_rank[kMaxExperts];
  __shared__ uint8_t s_col[kActive * kCols];  // [active][token]: place of the expert in the token's list
  __shared__ uint8_t s_idx[kActive * kCols];  // [active][token]: the token's number among the expert's
  __shared__ __attribute__((aligned(16))) uint16_t s_slot[kActive * kCols];  // [active][number]: its h row
  __shared__ float s_wt[kActive * kCols];     // [active][token]: router weight times w2's global scale, 0: none
  __shared__ int s_en[kActive];                    // expert | tokens << 16
  __shared__ float s_gs13[kActive], s_xs[kCols];
  __shared__ int s_cnt[kWaves], s_claim[2], s_late;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, q = lane >> 4;
  const int T = a.T, H = a.H, I = a.I, kt = a.g.top_k + a.g.shared;
  // A queue of items and a counter of finished ones per XCD, a line each:
  // item i belongs to queue i % 8.  (256 workgroups on one counter: 50 ns per
  // claim, 13 us until the last one has its first item.)
  const int xcd = xcc_id() & (kQueues - 1);
  int32_t* const queues = a.sync;
  int32_t* const dones = a.sync + kQueues * kLine;

  // the first claim does not need the selection
  int q_of = xcd;  // the queue this workgroup claims from
  int claimed = 0;
  if (tid == 0) claimed = claim_from(queues + q_of * kLine, 2);

  // ---- selection, by every workgroup for itself
  for (int i = tid; i < kMaxExperts; i += kThreads) s_rank[i] = 0;
  for (int i = tid; i < kActive * kCols / 4; i += kThreads) reinterpret_cast<uint32_t*>(s_col)[i] = ~0u;
  static_assert(kFewTokens <= kWaves, "a wave per token");
  if (wave < T) {
    const int t = wave;
    const float* row = a.logits + (size_t)t * a.ld;
    float bias[NI];
    gate_bias<NI>(a.g, lane, bias);
    auto emit = [&](int j, int id, float w) __attribute__((always_inline)) {
      s_ids[t * kt + j] = id;
      s_tw[t * kt + j] = w;
    };
    // (rows are padded to 64 * NI)
    float l[NI];
#pragma unroll
    for (int i = 0; i < NI; i += 4) {
      const float4 v = *reinterpret_cast<const float4*>(row + lane * NI + i);
      l[i] = v.x, l[i + 1] = v.y, l[i + 2] = v.z, l[i + 3] = v.w;
    }
    gate_select<NI>(l, bias, a.g, lane, emit);
    for (int j = lane; j < a.g.shared; j += 64) {
      s_ids[t * kt + a.g.top_k + j] = a.g.E + j;
      s_tw[t * kt + a.g.top_k + j] = 1.0f;
    }
  }
  // this wave's activations (behind the selection: its registers are free now)
  const int nch = H >> 8;
  u32x4 xb[NC][8];
  {
    const uint16_t* src = (MODE == 0 ? a.x16 : a.x) + (size_t)(r16 < T ? r16 : 0) * H + 64 * q;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int ck = wave + kWaves * i;
#pragma unroll
      for (int j = 0; j < 8; ++j) xb[i][j] = u32x4{0u, 0u, 0u, 0u};
      if (ck < nch && r16 < T) {
#pragma unroll
        for (int j = 0; j < 8; ++j) xb[i][j] = *reinterpret_cast<const u32x4*>(src + ck * 256 + 8 * j);
      }
    }
  }
  if (tid == 0) s_claim[0] = claimed;
  __syncthreads();
  int item = __builtin_amdgcn_readfirstlane(s_claim[0]) * kQueues + q_of, next = item + kQueues;
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
    s_en[rank] = tid;
    s_rank[tid] = (short)rank;
    s_gs13[rank] = a.w13_gs ? a.w13_gs[tid] : 1.0f;
  }
  if (tid < kCols) s_xs[tid] = MODE == 0 && tid < T ? a.xs[tid] : 1.0f;
  __syncthreads();
  int none = 0;
  for (int i = tid; i < T * kt; i += kThreads) {
    const int id = s_ids[i], t = i / kt;
    if (id >= 0) s_col[s_rank[id] * kCols + t] = (uint8_t)(i - t * kt);
    if (blockIdx.x == 0) {
      none += id < 0;
      if (a.ids) a.ids[i] = id;
      if (a.wts) a.wts[i] = s_tw[i];
    }
  }
  if (none) atomicAdd(a.flags, none);
  if (nact == 0) {  // no token has an expert (every workgroup finds the same)
    for (size_t i = (size_t)blockIdx.x * kThreads + tid; i < (size_t)T * H; i += (size_t)gridDim.x * kThreads) {
      if (a.out_f32) static_cast<float*>(a.out)[i] = 0.0f;
      else static_cast<uint16_t*>(a.out)[i] = 0;
    }
    return;
  }
  __syncthreads();
  // 16 lanes per active expert, a token each
  for (int i = tid; i < nact * kCols; i += kThreads) {
    const int act = i >> 4, t = i & 15, col = s_col[i];
    const uint32_t has = (uint32_t)(ballot(col != 255) >> (lane & 48)) & 0xFFFFu;
    const int n = __popc(has & ((1u << t) - 1u)), ne = __popc(has), first = __builtin_ctz(has);
    const int e = s_en[act] & 0xFFFF;  // (lane t = 0 writes the count beside it)
    s_idx[i] = (uint8_t)n;
    s_wt[i] = col != 255 ? s_tw[t * kt + col] * (a.w2_gs ? a.w2_gs[e] : 1.0f) : 0.0f;
    // h rows in token order; past the last, the first again
    if (col != 255) s_slot[act * kCols + n] = (uint16_t)(t * kt + col);
    const int c0 = s_col[act * kCols + first];
    if (t >= ne) s_slot[act * kCols + t] = (uint16_t)(first * kt + c0);
    if (t == 0) s_en[act] = e | (ne << 16);
  }
  __syncthreads();

  // ---- FC1 + SwiGLU: h
  const int npt = I >> 4;
  const int n1 = nact * npt;
  const uint32_t rowb = (uint32_t)(H >> 1), rows = (uint32_t)(MODE == 0 ? H >> 4 : H >> 5);
  const size_t A = (size_t)T * kt;
  WPair w1[NC];
  auto expert = [&](int act) __attribute__((always_inline)) { return __builtin_amdgcn_readfirstlane(s_en[act]) & 0xFFFF; };
  // (past the last item: the first one's rows, for loads that are issued all
  // the same and whose data is not used)
  const LaneOff off1 = lane_offsets(lane, rowb, rows, MODE);
  auto src1 = [&](int it) __attribute__((always_inline)) -> WSrc {
    const int i0 = it < n1 ? it : 0;
    const int act = i0 / npt, pt = i0 - act * npt;
    const size_t r = (size_t)expert(act) * 2 * I + pt * 16;
    const size_t g = r + (a.w13_order ? I : 0), u = r + (a.w13_order ? 0 : I);
    return WSrc{uniform_ptr(a.w13 + g * rowb), uniform_ptr(a.w13 + u * rowb), uniform_ptr(a.w13_sf + g * rows),
                uniform_ptr(a.w13_sf + u * rows)};
  };
  const Turn turn = turn_offsets(lane);
  uint8_t* const my_turn = s_turn[wave];
  int buf = 0, mine = 0;
  // chunk i of this wave, one that exists where H has fewer (its activations
  // are zero).  No load of the loop is conditional: the compiler counts the
  // loads in flight over every path, and waits for more than it has to where
  // one of them has fewer.
  uint32_t ck1[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) ck1[i] = (uint32_t)(wave + kWaves * i < nch ? wave + kWaves * i : nch - 1);
  while (item < n1) {
    const WSrc src = src1(item);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      load_pair<MODE>(w1[i], src, off1, ck1[i]);
      __builtin_amdgcn_sched_barrier(0);
    }
    // (the activations, requested earlier, have arrived: without this they
    // would count as in flight throughout the loop)
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) asm volatile("" : "+v"(xb[i][j]));
  do {
    int claim = 0;
    if (tid == 0) claim = claim_from(queues + q_of * kLine, 1);
    v4f acc[2] = {v4f{0.f, 0.f, 0.f, 0.f}, v4f{0.f, 0.f, 0.f, 0.f}};
    const WSrc src = src1(next);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      use_from_here(w1[i]);
      turn_pair(w1[i], my_turn, turn);
      mfma_pair<MODE, 1>(w1[i], acc, [&](int j, int) __attribute__((always_inline)) { return xb[i][j]; });
      load_pair<MODE>(w1[i], src, off1, ck1[i]);
      __builtin_amdgcn_sched_barrier(0);
    }
    s_red[buf][wave][0][lane] = float4{acc[0][0], acc[0][1], acc[0][2], acc[0][3]};
    s_red[buf][wave][1][lane] = float4{acc[1][0], acc[1][1], acc[1][2], acc[1][3]};
    if (tid == 0) s_claim[buf] = claim;
    lds_barrier();
    const int after = __builtin_amdgcn_readfirstlane(s_claim[buf]) * kQueues + q_of;
    if (wave == (mine & (kWaves - 1))) {
      // the waves take turns: sum, SwiGLU, store.  Lane: rows 4 q .. + 3, token r16.
      float g[4] = {0.f, 0.f, 0.f, 0.f}, u[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float4 gv = s_red[buf][w][0][lane], uv = s_red[buf][w][1][lane];
        g[0] += gv.x, g[1] += gv.y, g[2] += gv.z, g[3] += gv.w;
        u[0] += uv.x, u[1] += uv.y, u[2] += uv.z, u[3] += uv.w;
      }
      const int act = item / npt, pt = item - act * npt;
      const float cs = s_gs13[act] * s_xs[r16];
      const int col = s_col[act * kCols + r16];
      float h[4];
      float amax = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[i] = swiglu(g[i] * cs, u[i] * cs);
        amax = fmaxf(amax, fabsf(h[i]));
      }
      const size_t slot = (size_t)r16 * kt + col, at = slot * I + pt * 16 + 4 * q;
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
#pragma clang fp contract(off)  // (the low part is of h as rounded, not of its factors)
          // (the high part stays finite where rounding would not; an infinite h
          // is in the low one)
          const uint32_t b = bf16_bits(__builtin_amdgcn_fmed3f(h[i], -kBf16Max, kBf16Max));
          hi |= (uint64_t)b << (16 * i);
          lo |= (uint64_t)bf16_bits(h[i] - bf16_to_f32(b)) << (16 * i);
        }
        if (r16 < T && col != 255) {
          st_agent(a.h + at, hi);
          st_agent(a.h + A * I + at, lo);
        }
      }
    }
    ++mine;
    buf ^= 1;
    // (a queue's claims only grow: with this item past the end, so is the next)
    item = next;
    next = after;
  } while (item < n1);
    // this queue is empty: on to one that is not, if there is one (the XCD's
    // workgroups may not all be running)
    if (wave == 0) {
      const int taken = __hip_atomic_load(queues + (lane & (kQueues - 1)) * kLine, __ATOMIC_RELAXED,
                                          __HIP_MEMORY_SCOPE_AGENT);
      const uint64_t left = ballot(lane < kQueues && taken * kQueues + lane < n1);
      if (lane == 0) s_claim[buf] = left ? (int)__builtin_ctzll(left) : -1;
    }
    lds_barrier();
    const int other = __builtin_amdgcn_readfirstlane(s_claim[buf]);
    buf ^= 1;
    if (other < 0) break;
    q_of = other;
    if (tid == 0) s_claim[buf] = claim_from(queues + q_of * kLine, 2);
    lds_barrier();
    item = __builtin_amdgcn_readfirstlane(s_claim[buf]) * kQueues + q_of;
    buf ^= 1;
    next = item + kQueues;
  }

  // ---- FC2: this workgroup's run of steps
  const int nch2 = I >> 8, units = nact * nch2;
  const int ns = (units + kWaves - 1) / kWaves;
  const int nrb = H >> 5;
  const uint32_t total = (uint32_t)(nrb * ns);  // total * nwg < 2^31 (checked by the launch)
  const uint32_t G = min((uint32_t)a.nwg, total);
  const uint32_t wg = blockIdx.x;
  // This workgroup's stores of h are complete, and said to be before its first
  // weights of FC2 are requested: those fill the CU's queues, and the last
  // workgroup's word would come 3 us later.
  drain_memory();
  lds_barrier();
  if (tid == 0 && mine) __hip_atomic_fetch_add(dones + xcd * kLine, mine, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const bool works = wg < G;
  const int begin = works ? (int)(wg * total / G) : 0, end = works ? (int)((wg + 1) * total / G) : 0;
  const uint32_t rowb2 = (uint32_t)(I >> 1), rows2 = (uint32_t)(MODE == 0 ? I >> 4 : I >> 5);
  constexpr int NB = MODE == 0 ? 1 : 2;  // parts of h
  // tokens of an expert taken at a time (group32: all of them)
  constexpr int kHalf = MODE == 0 ? 4 : kFewTokensG32;
  static_assert(kHalf <= 4 && kFewTokens <= 2 * 4, "h rows are looked up four at a time, at most twice");
  constexpr int NS = 3;                  // steps in flight
  WPair w2[NS];
  uint64_t hb[NS][NB][kHalf];
  uint32_t hx[NS];
  // The run is walked in groups of up to NS steps of one row block.
  struct Group { int rb, st, n; };
  auto group = [&](int s) __attribute__((always_inline)) -> Group {
    const int rb = s / ns, st = s - rb * ns;
    return Group{rb, st, min(NS, min(ns - st, end - s))};
  };
  // The unit (expert, chunk) that this wave takes of a step: units are counted
  // on from step to step, 8 at a time (no divisions).  Where the last step of a
  // block has fewer than 8, the last unit stands in; its product is not added.
  const int d_act = kWaves / nch2, d_c = kWaves - d_act * nch2;
  struct Unit { int act, c; };
  auto unit = [&](int st) __attribute__((always_inline)) -> Unit {
    const int f = st * kWaves + wave, act = f / nch2;
    return Unit{act, f - act * nch2};
  };
  auto next_unit = [&](Unit u) __attribute__((always_inline)) -> Unit {
    u.act += d_act;
    u.c += d_c;
    return u.c >= nch2 ? Unit{u.act + 1, u.c - nch2} : u;
  };
  auto there = [&](Unit u) __attribute__((always_inline)) -> Unit { return u.act < nact ? u : Unit{nact - 1, nch2 - 1}; };
  // Loads of steps that a group does not have are issued too, from the group's
  // last unit again.
  const LaneOff off2 = lane_offsets(lane, rowb2, rows2, MODE);
  auto load_w2 = [&](int rb, Unit u, WPair& w) __attribute__((always_inline)) {
    u = there(u);
    const size_t r = (size_t)expert(u.act) * H + rb * 32;
    const uint8_t *c = a.w2 + r * rowb2, *f = a.w2_sf + r * rows2;
    load_pair<MODE>(w, WSrc{uniform_ptr(c), uniform_ptr(c + 16 * rowb2), uniform_ptr(f), uniform_ptr(f + 16 * rows2)}, off2,
                    u.c);
  };
  // h of the expert's tokens n0 .. n0 + kHalf - 1, a token's 512 bytes per
  // load (and per part); loads for tokens it does not have collapse to one
  // line.  (Offsets in 32 bits: h is below 2 GB.)
  auto h_rows = [&](int act, int c, int n0, uint64_t (&b)[NB][kHalf]) __attribute__((always_inline)) {
    const uint2 four = *reinterpret_cast<const uint2*>(s_slot + act * kCols + n0);
    const int ne = __builtin_amdgcn_readfirstlane(s_en[act]) >> 16;
    const uint32_t pair[2] = {(uint32_t)__builtin_amdgcn_readfirstlane((int)four.x),
                              (uint32_t)__builtin_amdgcn_readfirstlane((int)four.y)};
#pragma unroll
    for (int n = 0; n < kHalf; ++n) {
      const uint32_t slot = (pair[n >> 1] >> (16 * (n & 1))) & 0xFFFFu;
      const uint32_t o = 2 * (slot * (uint32_t)I + c * 256) + (n0 + n < ne ? 8 * lane : 0);
#pragma unroll
      for (int p = 0; p < NB; ++p) b[p][n] = gload<uint64_t>((GPtr)(a.h + p * A * I), o);
    }
  };
  auto load_h = [&](Unit u, uint64_t (&b)[NB][kHalf], uint32_t& x) __attribute__((always_inline)) {
    u = there(u);
    h_rows(u.act, u.c, 0, b);
    if (MODE == 0) {
      const int col = s_col[u.act * kCols + r16];
      const uint32_t slot = col != 255 ? (uint32_t)(r16 * kt + col) : s_slot[u.act * kCols];
      const uint32_t o = slot * (uint32_t)(I >> 4) + u.c * 16 + 4 * q;
      x = gload<uint32_t>((GPtr)a.hexp, o);
    }
  };
  Group cur = group(begin);
  const Unit first_unit = unit(cur.st);
  {
    Unit u = first_unit;
#pragma unroll
    for (int k = 0; k < NS; ++k) {
      load_w2(cur.rb, u, w2[k]);
      __builtin_amdgcn_sched_barrier(0);
      if (k + 1 < cur.n) u = next_unit(u);
    }
  }
  if (wave == 0) {
    int late = 0;
    for (int looks = 0; works; ++looks) {
      if (looks == a.looks) {
        late = 1;
        if (lane == 0) __hip_atomic_fetch_add(a.flags + 1, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        break;
      }
      int d = __hip_atomic_load(dones + (lane & (kQueues - 1)) * kLine, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      d += __shfl_xor(d, 1, 64);
      d += __shfl_xor(d, 2, 64);
      d += __shfl_xor(d, 4, 64);
      if (__builtin_amdgcn_readfirstlane(d) >= n1) break;
      __builtin_amdgcn_s_sleep(4);
    }
    if (lane == 0) s_late = late;
    // (what this CU and XCD cached of h before is dropped: h is read through
    // the caches from here on)
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  }
  lds_barrier();
  {
    Unit u = first_unit;
#pragma unroll
    for (int k = 0; k < NS; ++k) {
      load_h(u, hb[k], hx[k]);
      __builtin_amdgcn_sched_barrier(0);
      if (k + 1 < cur.n) u = next_unit(u);
    }
  }

  // (NaN where the wait was given up: nothing that this workgroup adds to is a
  // number then, whoever looks or does not look at the flags)
  const float from = __builtin_amdgcn_readfirstlane(s_late) ? __builtin_nanf("") : 0.0f;
  float oacc[8] = {from, from, from, from, from, from, from, from};
  int first = 1;  // still in the run's first row block
  int flushes = 0;
  // the row block's sum over the waves, and on to the output: directly where
  // the run holds the whole block, else through the parts
  auto flush = [&](int rb) __attribute__((always_inline)) {
    s_red[buf][wave][0][lane] = float4{oacc[0], oacc[1], oacc[2], oacc[3]};
    s_red[buf][wave][1][lane] = float4{oacc[4], oacc[5], oacc[6], oacc[7]};
#pragma unroll
    for (int i = 0; i < 8; ++i) oacc[i] = from;
    lds_barrier();
    if (wave == (flushes & (kWaves - 1))) {
      float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float4 u = s_red[buf][w][0][lane], v = s_red[buf][w][1][lane];
        o[0] += u.x, o[1] += u.y, o[2] += u.z, o[3] += u.w;
        o[4] += v.x, o[5] += v.y, o[6] += v.z, o[7] += v.w;
      }
      const int s0 = rb * ns, s1 = s0 + ns;
      bool write = true;
      if (begin > s0 || end < s1) {
        float* mypart = a.part + ((size_t)wg * 2 + (first ? 0 : 1)) * 512 + lane * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) st_agent(mypart + 2 * i, (uint64_t)f2u(o[2 * i]) | ((uint64_t)f2u(o[2 * i + 1]) << 32));
        drain_memory();
        // owners of the block's first and last step (the last w with w total / G <= step)
        const uint32_t o0 = ((s0 + 1) * G - 1) / total, o1 = (s1 * G - 1) / total;
        const int came = __builtin_amdgcn_readfirstlane(
            __hip_atomic_fetch_add(a.sync + 2 * kQueues * kLine + rb, lane == 0 ? 1 : 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
        write = came == (int)(o1 - o0);
        if (write) {
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = 0.0f;
          for (uint32_t w = o0; w <= o1; ++w) {
            const bool head = (int)(w * total / G) >= s0;  // the block is run w's first
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
    ++flushes;
    buf ^= 1;
    first = 0;
  };
  uint8_t* const my_h = s_h[wave];
  // (waits for loads of h here, so that code behind a branch does not)
  auto arrived = [](uint64_t (&b)[NB][kHalf]) __attribute__((always_inline)) {
#pragma unroll
    for (int p = 0; p < NB; ++p)
#pragma unroll
      for (int n = 0; n < kHalf; ++n) asm volatile("" : "+v"(b[p][n]));
  };
#pragma unroll
  for (int k = 0; k < NS; ++k) {
    arrived(hb[k]);
    if (MODE == 0) asm volatile("" : "+v"(hx[k]));
  }
  Unit cu = first_unit;
  for (int s = begin; s < end;) {
    const int after = s + cur.n;
    // (past the end: this group's rows again)
    Group nxt = cur;
    Unit nu = cu;
    if (after < end) {
      nxt = group(after);
      nu = unit(nxt.st);
    }
#pragma unroll
    for (int k = 0; k < NS; ++k) {
      use_from_here(w2[k]);
      if (k < cur.n) {
        const Unit u = there(cu);
        const int act = u.act, c = u.c;
        const bool counts = cu.act < nact;
        if (k + 1 < cur.n) cu = next_unit(cu);
        const int ne = __builtin_amdgcn_readfirstlane(s_en[act]) >> 16;
        const int idx = s_idx[act * kCols + r16];
        // (0: not this token's expert, or a unit that only stands in)
        float cs = counts ? s_wt[act * kCols + r16] : 0.0f;
        const bool chosen = counts && s_col[act * kCols + r16] != 255;
        turn_pair(w2[k], my_turn, turn);
        _Float16 f4[4];
        if constexpr (MODE == 0) {
          // the chunk's largest exponent P; each 16-block's values times 2**(p - P)
          int p[4], P = -128;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            p[i] = (int)(int8_t)(hx[k] >> (8 * i));
            P = max(P, p[i]);
          }
          P = max(P, __shfl_xor(P, 16, 64));
          P = max(P, __shfl_xor(P, 32, 64));
          cs = __builtin_ldexpf(cs, P);
#pragma unroll
          for (int i = 0; i < 4; ++i) f4[i] = (_Float16)__builtin_ldexpf(1.0f, p[i] - P);
        }
        // kHalf tokens at a time (more of one expert: once again, their h
        // fetched on the spot)
#pragma unroll 1
        for (int n0 = 0;;) {
#pragma unroll
          for (int p = 0; p < NB; ++p)
#pragma unroll
            for (int n = 0; n < kHalf; ++n)
              *reinterpret_cast<uint64_t*>(my_h + (p * kHalf + n) * kHRow + 8 * lane) = hb[k][p][n];
          // (columns of other tokens read some row and are not used)
          const int r = idx - n0;
          const uint8_t* row = my_h + (r >= 0 && r < kHalf ? r : 0) * kHRow + 128 * q;
          v4f acc[2] = {v4f{0.f, 0.f, 0.f, 0.f}, v4f{0.f, 0.f, 0.f, 0.f}};
          mfma_pair<MODE, NB>(w2[k], acc, [&](int j, int p) __attribute__((always_inline)) {
            const u32x4 v = *reinterpret_cast<const u32x4*>(row + p * kHalf * kHRow + 16 * j);
            if constexpr (MODE == 0) return __builtin_bit_cast(v8h, v) * f4[j >> 1];
            else return v;
          });
          if (chosen && r >= 0 && r < kHalf) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              oacc[i] = __builtin_fmaf(acc[0][i], cs, oacc[i]);
              oacc[4 + i] = __builtin_fmaf(acc[1][i], cs, oacc[4 + i]);
            }
          }
          n0 += kHalf;
          if (MODE == 1 || n0 >= ne) break;
          h_rows(act, c, n0, hb[k]);
          arrived(hb[k]);
        }
      }
      load_w2(nxt.rb, nu, w2[k]);
      load_h(nu, hb[k], hx[k]);
      if (k + 1 < nxt.n) nu = next_unit(nu);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (cur.st + cur.n == ns || after >= end) flush(cur.rb);
    s = after;
    cur = nxt;
    cu = unit(cur.st);
  }
}

template <int MODE, int NI>
void launch_layer(const FewArgs& a, hipStream_t s) {
  const int nc = (a.H / 256 + kWaves - 1) / kWaves;
  const dim3 grid(a.nwg), block(kThreads);
  if (nc <= 1) hipLaunchKernelGGL((few_layer_kernel<MODE, 1, NI>), grid, block, 0, s, a);
  else if (nc == 2) hipLaunchKernelGGL((few_layer_kernel<MODE, 2, NI>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((few_layer_kernel<MODE, 3, NI>), grid, block, 0, s, a);
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
  if (a.g16 && a.ld == 256) launch_layer<0, 4>(a, s);
  else if (a.g16) launch_layer<0, 8>(a, s);
  else if (a.ld == 256) launch_layer<1, 4>(a, s);
  else launch_layer<1, 8>(a, s);
  return hipGetLastError();
}

}  // namespace moefp4
