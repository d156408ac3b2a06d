// Matrix products grouped by expert with ragged sizes: the rows of an operand
// lie in expert order, expert e's in [offsets[e], offsets[e + 1]).
//   product:            y[r]  = W_e x[r]              (NT: both operands along the sum)
//   towards the rows:   dx[r] = W_e^T dy[r]           (NN: the weights across it)
//   towards the weights: dW_e = sum_r dy[r] x[r]^T    (TN: both across it)
// W_e [N, K] bfloat16, or E2M1 codes with group16 or group32 scales (decoded to
// bfloat16, which holds a code times an E4M3 or UE8M0 scale exactly).
#include "common.h"
#include "kernels.h"

#include <type_traits>

namespace moefp4 {

namespace {

enum Form { NT, NN, TN };

constexpr int kS = 64;  // elements of the sum per stage

typedef short v4s __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint32_t bf16_bits(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

// 16 bytes per lane from base + off to consecutive places in LDS.  As an
// instruction of its own (it writes no register): the compiler takes a builtin
// direct load to alias every transposing LDS read, and waits for it there.
// What ends it is wait_all.
__device__ __forceinline__ void direct_load(const uint8_t* base, uint32_t off, const uint8_t* lds) {
  typedef const __attribute__((address_space(3))) uint8_t* lds1;
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"((uint32_t)(uintptr_t)(lds1)lds), "v"(off), "s"(base)
               : "memory");
}

// ---------------------------------------------------------------------------
// tiles

// The place of workgroup b among the tiles: groups of 32 consecutive tiles per
// XCD in turn (an XCD's 32 CUs share an L2).
__device__ __forceinline__ int tile_of(int b) {
  const int i = b >> 3;
  return (((i >> 5) * 8 + (b & 7)) << 5) + (i & 31);
}

// Tile i of the np x nq tiles of one expert, four of np at a time, so that
// neighbours share both operands.
__device__ __forceinline__ void tile_at(int i, int np, int nq, int* p, int* q) {
  const int g = i / (4 * nq), left = i - g * 4 * nq, size = min(4, np - 4 * g);
  *q = left / size;
  *p = 4 * g + left - *q * size;
}

struct Rows { int e, r0, n, i, np; };  // expert, its first row, its rows, the tile among the expert's, row tiles

// The expert that tile `tile` belongs to, where every row tile of `size` rows
// has nq tiles; e = -1 behind the last tile.  Every wave finds it by itself: a
// lane counts the tiles of E / 64 experts.
__device__ __forceinline__ Rows rows_of(const int32_t* offsets, int E, int M, int size, int nq, int tile) {
  const int lane = threadIdx.x & 63, per = (E + 63) >> 6, e0 = min(lane * per, E), e1 = min(e0 + per, E);
  int cnt = 0, a = min(max(offsets[e0], 0), M);
  for (int e = e0; e < e1; ++e) {
    const int b = min(max(offsets[e + 1], 0), M);
    cnt += (max(b - a, 0) + size - 1) / size;
    a = b;
  }
  int incl = cnt;
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(incl, d, 64);
    if (lane >= d) incl += v;
  }
  const int want = tile / nq;
  const uint64_t in = __ballot(want < incl);
  Rows r{-1, 0, 0, 0, 0};
  if (in == 0) return r;
  const int src = __builtin_ctzll(in);
  int before = __builtin_amdgcn_readlane(incl - cnt, src);
  for (int e = src * per; e < E; ++e) {
    const int s = min(max(offsets[e], 0), M), b = min(max(offsets[e + 1], 0), M);
    const int n = max(b - s, 0), t = (n + size - 1) / size;
    if (want < before + t) return Rows{e, s, n, tile - before * nq, t};
    before += t;
  }
  return r;
}

// ---------------------------------------------------------------------------
// operands of a tile

// 16-byte segment s of LDS row r (128 bytes) sits at s ^ pswz(r).
__device__ __forceinline__ int pswz(int r) { return (r >> 1) & 7; }
// 32-byte chunk c of LDS row r (an element of the sum) sits at c ^ tswz(r): the
// 8 rows that 32 lanes of a transposing read take lie in different banks.
__device__ __forceinline__ int tswz(int r) { return (r & 3) | ((r >> 1) & 4); }

// One operand's stage: SIZE rows of kS elements along the sum (TR = false), or
// kS rows of SIZE elements (TR: across it; read by the transposing LDS reads).
// NTH threads load it, 16 bytes per lane straight to LDS.
template <bool TR, int SIZE, int NTH>
struct Operand {
  static constexpr int kPieces = SIZE * 8 / NTH;
  static constexpr int kBytes = SIZE * kS * 2;
  const uint8_t* base;  // uniform
  uint32_t ld;          // bytes per row
  uint32_t off[kPieces];

  // valid: rows (TR: elements across) that exist
  __device__ __forceinline__ void init(const void* p, uint32_t ld_bytes, int valid) {
    base = static_cast<const uint8_t*>(p);
    ld = ld_bytes;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      if constexpr (TR) {
        constexpr int per = SIZE / 8;  // pieces per row
        const int r = (wave * kPieces + i) * (64 / per) + lane / per, piece = lane % per;
        const int c = (((piece >> 1) ^ tswz(r)) << 4) + ((piece & 1) << 3);
        off[i] = 2 * min(c, valid - 8);
      } else {
        const int r = (wave * kPieces + i) * 8 + (lane >> 3);
        off[i] = min(r, valid - 1) * ld;
      }
    }
  }

  // stage s of a sum of n elements (past the last one: the last one again)
  __device__ __forceinline__ void load(int s, int n, uint8_t* lds) const {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint8_t* at = TR ? base + (size_t)s * kS * ld : base;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      uint32_t o;
      if constexpr (TR) {
        constexpr int per = SIZE / 8;
        const int r = (wave * kPieces + i) * (64 / per) + lane / per;
        o = off[i] + (uint32_t)min(r, n - 1 - s * kS) * ld;
      } else {
        const int r = (wave * kPieces + i) * 8 + (lane >> 3);
        o = off[i] + min(s * kS * 2 + (((lane & 7) ^ pswz(r)) << 4), 2 * (n - 8));
      }
      direct_load(at, o, lds + (wave * kPieces + i) * 1024);
    }
  }

  // zeros behind the sum's last element in its last stage, of which `left` exist
  __device__ __forceinline__ static void clear(int left, uint8_t* lds) {
    for (int v = threadIdx.x; v < kBytes / 16; v += NTH) {
      const bool out = TR ? v / (SIZE / 8) >= left : 8 * ((v & 7) ^ pswz(v >> 3)) >= left;
      if (out) *reinterpret_cast<uint4*>(lds + 16 * v) = uint4{0, 0, 0, 0};
    }
  }

  // Where the calling lane reads a matrix operand of the rows from w0 on, whole
  // but for the bits of its tile (frag).
  __device__ __forceinline__ static uint32_t lane_at(int w0) {
    const int lane = threadIdx.x & 63, r16 = lane & 15, q = lane >> 4;
    if constexpr (TR) {
      const int r = 8 * q + (r16 >> 2);
      return r * (SIZE * 2) + ((tswz(r) ^ (w0 >> 4)) << 5) + ((r16 & 3) << 3);
    } else {
      return (w0 + r16) * 128 + ((q ^ pswz(r16)) << 4);
    }
  }

  // The 16 rows from w0 + 16 t on, elements 32 ks .. + 31 of the stage, as a
  // matrix operand (lane: row lane % 16, elements 8 (lane / 16) .. + 7).
  __device__ __forceinline__ static u32x4 frag(const uint8_t* lds, uint32_t lane_at, int t, int ks) {
    if constexpr (TR) {
      const uint8_t* p = lds + (lane_at ^ (t << 5)) + ks * 32 * (SIZE * 2);
      typedef __attribute__((address_space(3))) v4s* lds4;
      const v4s a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)p);
      const v4s b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(p + 4 * SIZE * 2));
      typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
      const u32x2 x = __builtin_bit_cast(u32x2, a), y = __builtin_bit_cast(u32x2, b);
      return u32x4{x[0], x[1], y[0], y[1]};
    } else {
      return *reinterpret_cast<const u32x4*>(lds + (lane_at ^ (ks << 6)) + t * 2048);
    }
  }
};

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

// FP4 weights as such an operand: a thread takes the 16 bytes of 32 codes of a
// row through registers, and decodes them to where the direct loads would have
// put them, a stage after they were asked for.
template <bool TR, int SIZE, int NTH, int GRAN>
struct Fp4Operand : Operand<TR, SIZE, NTH> {
  static_assert(SIZE * kS == 32 * NTH, "32 codes per thread and stage");
  static constexpr int kPer = TR ? SIZE / 32 : 2;  // pieces of a row
  const uint8_t *codes, *sf;  // uniform
  int K;
  uint32_t row_c, row_s;  // the thread's row (TR: column), in bytes
  u32x4 c;
  uint32_t s;

  // w, w_sf: the tile's first row (TR: of the whole sum) and column; valid rows (TR: columns)
  __device__ __forceinline__ void init(const uint8_t* w, const uint8_t* w_sf, int k, int valid) {
    codes = w;
    sf = w_sf;
    K = k;
    const uint32_t r = TR ? min(32 * ((int)threadIdx.x % kPer), valid - 32) : min((int)threadIdx.x / kPer, valid - 1);
    row_c = TR ? r / 2 : r * (K / 2);
    row_s = TR ? r / GRAN : r * (K / GRAN);
  }

  __device__ __forceinline__ void fetch(int st, int n) {
    const uint8_t *pc = codes, *ps = sf;
    uint32_t oc, os;
    if (TR) {
      pc += (size_t)st * kS * (K / 2);
      ps += (size_t)st * kS * (K / GRAN);
      const uint32_t r = min((int)threadIdx.x / kPer, n - 1 - st * kS);
      oc = row_c + r * (K / 2);
      os = row_s + r * (K / GRAN);
    } else {
      const uint32_t at = min(st * kS + 32 * ((int)threadIdx.x % kPer), n - 32);
      oc = row_c + at / 2;
      os = row_s + at / GRAN;
    }
    c = *reinterpret_cast<const u32x4*>(pc + oc);
    if (GRAN == 16) s = *reinterpret_cast<const uint16_t*>(ps + os);
    else s = ps[os];
  }

  // what was fetched into stage buffer lds, and the next stage asked for
  __device__ __forceinline__ void load(int st, int n, uint8_t* lds) {
    const int row = threadIdx.x / kPer, piece = threadIdx.x % kPer;
    uint32_t at = TR ? row * (SIZE * 2) + ((2 * piece ^ tswz(row)) << 5) : row * 128 + ((4 * piece ^ pswz(row)) << 4);
    asm volatile("" : "+v"(at));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u32x4 v;
      if (GRAN == 16) v = dq8_scaled_bf16(c[j], e4m3_to_f32((s >> (8 * (j >> 1))) & 0xFFu));
      else v = __builtin_bit_cast(u32x4, dq8_bf16(c[j], ue8m0_to_f32(s)));
      *reinterpret_cast<u32x4*>(lds + (TR ? (at ^ ((j >> 1) << 5)) + 16 * (j & 1) : at ^ (j << 4))) = v;
      __builtin_amdgcn_sched_barrier(0);  // (one after the other: registers are short)
    }
    fetch(min(st + 1, (n - 1) / kS), n);  // (behind the last stage: the last one again)
  }
};

template <bool TR, int SIZE, int NTH, int GRAN>
struct WeightOperand { typedef Fp4Operand<TR, SIZE, NTH, GRAN> type; };
template <bool TR, int SIZE, int NTH>
struct WeightOperand<TR, SIZE, NTH, 0> { typedef Operand<TR, SIZE, NTH> type; };

// Every wave's loads and LDS accesses done, and a barrier.
__device__ __forceinline__ void wait_all() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// ---------------------------------------------------------------------------
// the tiled product

// P x Q outputs per workgroup: P along the rows (TN: along N), Q along the
// output's contiguous side; WP x WQ waves.  GRAN: 0, or FP4 weights' group.
template <int FORM, int GRAN, int P, int Q, int WP, int WQ>
__global__ __launch_bounds__(WP * WQ * 64, 2) void grouped_tile_kernel(GroupedArgs a) {
  constexpr int NTH = WP * WQ * 64;
  constexpr int NP = P / WP / 16, NQ = Q / WQ / 16;  // a wave's 16-row tiles
  typedef Operand<FORM == TN, P, NTH> OpP;
  typedef typename WeightOperand<FORM != NT, Q, NTH, GRAN>::type OpQ;
  __shared__ __attribute__((aligned(16))) uint8_t s_p0[OpP::kBytes], s_p1[OpP::kBytes], s_q0[OpQ::kBytes], s_q1[OpQ::kBytes];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, q4 = lane >> 4;
  const int outs = FORM == NT ? a.N : a.K;  // the output's contiguous side
  const int nq = (outs + Q - 1) / Q;
  const int tile = tile_of(blockIdx.x);
  Rows r;
  if constexpr (FORM == TN) {
    const int np = (a.N + P - 1) / P, e = tile / (np * nq);
    if (e >= a.E) return;
    const int s = min(max(a.offsets[e], 0), a.M);
    r = Rows{e, s, max(min(max(a.offsets[e + 1], 0), a.M) - s, 0), tile - e * np * nq, np};
  } else {
    r = rows_of(a.offsets, a.E, a.M, P, nq, tile);
    if (r.e < 0) return;
  }
  r.e = __builtin_amdgcn_readfirstlane(r.e);
  r.r0 = __builtin_amdgcn_readfirstlane(r.r0);
  r.n = __builtin_amdgcn_readfirstlane(r.n);
  int tp, tq;
  tile_at(__builtin_amdgcn_readfirstlane(r.i), __builtin_amdgcn_readfirstlane(r.np), nq, &tp, &tq);
  const int p0 = tp * P, q0 = tq * Q;
  const int pn = (FORM == TN ? a.N : r.n) - p0, qn = outs - q0;  // what exists of the tile
  const int sum = FORM == NT ? a.K : FORM == NN ? a.N : r.n;
  const int nst = (sum + kS - 1) / kS, tail = sum & (kS - 1);
  const int wp = (wave / WQ) * (P / WP), wq = (wave % WQ) * (Q / WQ);

  OpP op;
  OpQ oq;
  if constexpr (FORM == TN) {
    op.init(a.p + (size_t)r.r0 * a.N + p0, 2 * a.N, pn);
    oq.init(a.q + (size_t)r.r0 * a.K + q0, 2 * a.K, qn);
  } else {
    op.init(a.p + (size_t)(r.r0 + p0) * sum, 2 * sum, pn);
    // the weights' first row and column of the tile
    const size_t row = (size_t)r.e * a.N + (FORM == NT ? q0 : 0);
    const int col = FORM == NT ? 0 : q0;
    if constexpr (GRAN != 0) {
      oq.init(a.w + row * (a.K / 2) + col / 2, a.w_sf + row * (a.K / GRAN) + col / GRAN, a.K, qn);
      oq.fetch(0, sum);
    } else {
      oq.init(a.q + row * a.K + col, 2 * a.K, qn);
    }
  }

  v4f acc[NQ][NP];
#pragma unroll
  for (int i = 0; i < NQ; ++i)
#pragma unroll
    for (int j = 0; j < NP; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  // Half of the row tiles at a time (a phase): 16 products per wave at 128 x 64.
  constexpr int NH = NP / 2;
  u32x4 fq[2][NQ], fp[2][NH];
  uint32_t at_q = OpQ::lane_at(wq), at_p = OpP::lane_at(wp);
  auto read_q = [&](int buf, int ks) __attribute__((always_inline)) {
    asm volatile("" : "+v"(at_q));  // (the tiles' addresses are formed anew: registers are short)
#pragma unroll
    for (int i = 0; i < NQ; ++i) fq[ks][i] = OpQ::frag(buf ? s_q1 : s_q0, at_q, i, ks);
  };
  auto read_p = [&](int buf, int ks, int h) __attribute__((always_inline)) {
    asm volatile("" : "+v"(at_p));
#pragma unroll
    for (int j = 0; j < NH; ++j) fp[h][j] = OpP::frag(buf ? s_p1 : s_p0, at_p, NH * h + j, ks);
  };
  auto multiply = [&](int ks, int h) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < NH; ++j)
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        v4f& c = acc[i][NH * h + j];
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, fq[ks][i]), __builtin_bit_cast(v8bf, fp[h][j]),
                                                    c, 0, 0, 0);
      }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto load = [&](int s, int buf) __attribute__((always_inline)) {
    op.load(s, sum, buf ? s_p1 : s_p0);
    oq.load(s, sum, buf ? s_q1 : s_q0);
  };
  // A stage's loads have landed, and every wave has read the one before.
  auto handover = [&](bool last, int buf) __attribute__((always_inline)) {
    __builtin_amdgcn_sched_barrier(0);
    wait_all();
    if (last && tail) {
      OpP::clear(tail, buf ? s_p1 : s_p0);
      OpQ::clear(tail, buf ? s_q1 : s_q0);
      wait_all();
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  // Stage s in buffer buf, in four phases: the operands of a phase come while the
  // one before multiplies.  The one barrier lies before the last phase, whose
  // operands are in registers: behind it the next stage's first operands are read.
  // NEXT: stages behind this one (2: or more).
  auto stage = [&](auto NEXT, int s, int buf) __attribute__((always_inline)) {
    read_p(buf, 0, 1);
    __builtin_amdgcn_sched_barrier(0);
    multiply(0, 0);
    read_q(buf, 1);
    read_p(buf, 1, 0);
    __builtin_amdgcn_sched_barrier(0);
    multiply(0, 1);
    read_p(buf, 1, 1);
    __builtin_amdgcn_sched_barrier(0);
    multiply(1, 0);
    if constexpr (NEXT.value > 0) {
      handover(NEXT.value == 1, buf ^ 1);
      if constexpr (NEXT.value > 1) load(s + 2, buf);
      read_q(buf ^ 1, 0);
      read_p(buf ^ 1, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
    multiply(1, 1);
  };
  typedef std::integral_constant<int, 0> Last;
  typedef std::integral_constant<int, 1> One;
  typedef std::integral_constant<int, 2> More;
  // (the last stage is always in buffer 1: no branch inside the loop)
  if (FORM != TN || nst > 0) {
    const int first = nst & 1;
    load(0, first);
    handover(nst == 1, first);
    read_q(first, 0);
    read_p(first, 0, 0);
    if (nst > 1) {
      load(1, first ^ 1);
      if (first) stage(More{}, 0, 1);
      int s = first;
      for (; s < nst - 2; s += 2) {
        stage(More{}, s, 0);
        stage(More{}, s + 1, 1);
      }
      stage(One{}, s, 0);
    }
    stage(Last{}, nst - 1, 1);
  }

  if (GRAN == 16 || GRAN == 32) {
    const float gs = a.w_gs ? a.w_gs[r.e] : 1.0f;
#pragma unroll
    for (int i = 0; i < NQ; ++i)
#pragma unroll
      for (int j = 0; j < NP; ++j) acc[i][j] *= gs;
  }
  const size_t row0 = FORM == TN ? (size_t)r.e * a.N + p0 : (size_t)(r.r0 + p0);
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    const int p = wp + 16 * j + r16;
    if (p >= pn) continue;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int q = wq + 16 * i + 4 * q4;
      if (q >= qn) continue;  // (a multiple of 8 exist)
      const size_t at = (row0 + p) * outs + q0 + q;
      v4f v = acc[i][j];
      if (a.out_f32) {
        v4f* o = reinterpret_cast<v4f*>(static_cast<float*>(a.out) + at);
        if (FORM == TN && a.accumulate) v += *o;
        *o = v;
      } else {
        uint2* o = reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at);
        if (FORM == TN && a.accumulate) {
          const uint2 b = *o;
          v += v4f{u2f(b.x << 16), u2f(b.x & 0xFFFF0000u), u2f(b.y << 16), u2f(b.y & 0xFFFF0000u)};
        }
        *o = uint2{bf16_bits(v[0]) | (bf16_bits(v[1]) << 16), bf16_bits(v[2]) | (bf16_bits(v[3]) << 16)};
      }
    }
  }
}

template <int FORM, int GRAN, int P, int Q, int WP, int WQ>
hipError_t launch_tile(const GroupedArgs& a, hipStream_t s) {
  const long long nq = ((FORM == NT ? a.N : a.K) + Q - 1) / Q;
  const long long most = a.E < a.M ? a.E : a.M;  // experts with rows
  const long long tiles = FORM == TN ? (long long)a.E * ((a.N + P - 1) / P) * nq : (a.M / P + most) * nq;
  // whole rounds of 8 XCDs of 32 tiles (tile_of)
  const long long grid = (tiles + 255) / 256 * 256;
  hipLaunchKernelGGL((grouped_tile_kernel<FORM, GRAN, P, Q, WP, WQ>), dim3((unsigned)grid), dim3(WP * WQ * 64), 0, s, a);
  return hipGetLastError();
}

template <int FORM, int GRAN>
hipError_t launch_form(const GroupedArgs& a, hipStream_t s) {
  return launch_tile<FORM, GRAN, 256, 256, 2, 4>(a, s);
}

}  // namespace

hipError_t launch_grouped(const GroupedArgs& a, int form, hipStream_t s) {
  if (form == TN) return launch_form<TN, 0>(a, s);
  if (a.gran == 16) return form == NT ? launch_form<NT, 16>(a, s) : launch_form<NN, 16>(a, s);
  if (a.gran == 32) return form == NT ? launch_form<NT, 32>(a, s) : launch_form<NN, 32>(a, s);
  return form == NT ? launch_form<NT, 0>(a, s) : launch_form<NN, 0>(a, s);
}

}  // namespace moefp4
