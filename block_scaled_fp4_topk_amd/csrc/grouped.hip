// Matrix products grouped by expert with ragged sizes: the rows of an operand
// lie in expert order, expert e's in [offsets[e], offsets[e + 1]).
//   product:            y[r]  = W_e x[r]              (NT: both operands along the sum)
//   towards the rows:   dx[r] = W_e^T dy[r]           (NN: the weights across it)
//   towards the weights: dW_e = sum_r dy[r] x[r]^T    (TN: both across it)
// W_e [N, K] bfloat16, or E2M1 codes with group16 or group32 scales, decoded to
// bfloat16.  That holds a code times its scale exactly, at the lower end as a
// subnormal, which the matrix instructions take, wherever it is below 2^128: with every
// E4M3 scale and with UE8M0 bytes up to 252 (beyond, 4 times 2^126 is an infinity).
//
// All three run on the 16 x 16 x 32 bfloat16 matrix instructions with float32 sums;
// an output is rounded once, to nearest.  Three things bound them: with few rows per
// expert the weights' bytes from HBM, each read once (the stream of the weights below);
// with many the matrix instructions, whose operands pass through LDS (the tiles); with
// a short sum (a low-rank factor) the output's bytes and a tile's fixed time.
#include "common.h"
#include "kernels.h"

#include <type_traits>

namespace moefp4 {

namespace {

enum Form { NT, NN, TN };

constexpr int kS = 64;  // elements of the sum per stage

typedef short v4s __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint32_t bf16_bits(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

// 16 bytes per lane from `off` of a buffer to consecutive places in LDS; zeros
// for what lies behind the buffer's end.  As an instruction of its own (it writes
// no register): the compiler takes a builtin direct load to alias every
// transposing LDS read, and waits for it there.  What ends it is wait_all.
__device__ __forceinline__ void direct_load(const v4i& buffer, uint32_t off, uint32_t uniform_off, const uint8_t* lds) {
  typedef const __attribute__((address_space(3))) uint8_t* lds1;
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"((uint32_t)(uintptr_t)(lds1)lds), "v"(off), "s"(buffer), "s"(uniform_off)
               : "memory");
}

// 2 (else 1) bytes per lane, to a word each.
template <bool TWO>
__device__ __forceinline__ void direct_load_small(const v4i& buffer, uint32_t off, uint32_t uniform_off, const uint8_t* lds) {
  typedef const __attribute__((address_space(3))) uint8_t* lds1;
  const uint32_t to = (uint32_t)(uintptr_t)(lds1)lds;
  if (TWO) asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_ushort %1, %2, %3 offen lds" : : "s"(to), "v"(off), "s"(buffer), "s"(uniform_off) : "memory");
  else asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_ubyte %1, %2, %3 offen lds" : : "s"(to), "v"(off), "s"(buffer), "s"(uniform_off) : "memory");
}

// A buffer descriptor: `bytes` from p on.
__device__ __forceinline__ v4i buffer_of(const uint8_t* p, uint32_t bytes) {
  const uint64_t at = reinterpret_cast<uintptr_t>(p);
  return v4i{(int)at, (int)(at >> 32) & 0xFFFF, (int)bytes, 0x00020000};
}

// ---------------------------------------------------------------------------
// tiles

// The place of workgroup b among the tiles: groups of consecutive tiles per XCD in
// turn (an XCD's 32 CUs share an L2).
__device__ __forceinline__ int tile_of(int b, int group) {
  const int i = b >> 3, g = i / group;
  return (g * 8 + (b & 7)) * group + i - g * group;
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
// has nq tiles; e = -1 behind the last tile.  Every wave finds it by itself, a
// lane counting the tiles of E / 64 experts, whose offsets it loads all at once.
__device__ __forceinline__ Rows rows_of(const int32_t* offsets, int E, int M, int size, int nq, int tile) {
  constexpr int kPer = kMaxExperts / 64;
  const int lane = threadIdx.x & 63, per = (E + 63) >> 6, e0 = lane * per;
  int at[kPer + 1], cnt = 0;
#pragma unroll
  for (int i = 0; i <= kPer; ++i) at[i] = i <= per ? offsets[min(e0 + i, E)] : 0;
#pragma unroll
  for (int i = 0; i <= kPer; ++i) at[i] = min(max(at[i], 0), M);
#pragma unroll
  for (int i = 0; i < kPer; ++i) cnt += i < per ? (max(at[i + 1] - at[i], 0) + size - 1) / size : 0;
  int incl = cnt;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(incl, d, 64);
    if (lane >= d) incl += v;
  }
  const int want = tile / nq;
  const uint64_t in = __ballot(want < incl);
  if (in == 0) return Rows{-1, 0, 0, 0, 0};
  // (every lane among its own; what counts is the lane that holds the tile)
  Rows r{0, 0, 0, 0, 0};
  int before = incl - cnt;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int n = max(at[i + 1] - at[i], 0), t = i < per ? (n + size - 1) / size : 0;
    if (want >= before && want < before + t) r = Rows{e0 + i, at[i], n, tile - before * nq, t};
    before += t;
  }
  const int src = __builtin_ctzll(in);
  return Rows{__builtin_amdgcn_readlane(r.e, src), __builtin_amdgcn_readlane(r.r0, src), __builtin_amdgcn_readlane(r.n, src),
              __builtin_amdgcn_readlane(r.i, src), __builtin_amdgcn_readlane(r.np, src)};
}

// ---------------------------------------------------------------------------
// operands of a tile

// 16-byte segment s of LDS row r (128 bytes) sits at s ^ pswz(r).
__device__ __forceinline__ int pswz(int r) { return (r >> 1) & 7; }
// 32-byte chunk c of LDS row r (an element of the sum; BYTES long) sits at c ^
// tswz(r): the 8 rows that 32 lanes of a transposing read take lie in different
// banks.
template <int BYTES>
__device__ __forceinline__ int tswz(int r) {
  static_assert(BYTES >= 128, "four chunks at least");
  return BYTES >= 256 ? (r & 3) | ((r >> 1) & 4) : ((r >> 1) & 1) | ((r >> 2) & 2);
}

// One operand's stage: SIZE rows of kS elements along the sum (TR = false), or
// kS rows of SIZE elements (TR: across it; read by the transposing LDS reads).
// NTH threads load it, 16 bytes per lane straight to LDS.
template <bool TR, int SIZE, int NTH>
struct Operand {
  static constexpr int kPieces = SIZE * 8 / NTH;
  static constexpr int kBytes = SIZE * kS * 2;
  const uint8_t* base;  // uniform
  uint32_t ld;          // bytes per row
  int valid;            // rows (TR: elements across) that exist
  uint32_t off[kPieces];

  // Where load i's lane is in a stage: row, and element of the row, as their LDS
  // places (lane order) say.
  __device__ __forceinline__ static int row(int i) {
    constexpr int per = TR ? SIZE / 8 : 8;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    return (wave * kPieces + i) * (64 / per) + lane / per;
  }
  __device__ __forceinline__ static int col(int i) {
    const int lane = threadIdx.x & 63, r = row(i);
    if constexpr (TR) return (((lane % (SIZE / 8) >> 1) ^ tswz<SIZE * 2>(r)) << 4) + ((lane & 1) << 3);
    else return ((lane & 7) ^ pswz(r)) << 3;
  }

  // (what lies outside the tile is fetched from the last row or column inside)
  __device__ __forceinline__ void init(const void* p, uint32_t ld_bytes, int exist) {
    base = static_cast<const uint8_t*>(p);
    ld = ld_bytes;
    valid = exist;
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      off[i] = TR ? __umul24(row(i), ld) + 2 * min(col(i), valid - 8) : __umul24(min(row(i), valid - 1), ld) + 2 * col(i);
  }

  // Stage s of a sum of n elements, by kPieces loads.  (Behind the sum's end: the
  // next row's elements, or zeros behind the last row; a stage behind the last one
  // is zeros, without any access to memory.)
  struct Stage { v4i buffer; uint32_t at; };
  __device__ __forceinline__ Stage stage(int s, int n) const {
    if constexpr (TR) {
      const int rows = min(n - s * kS, kS);
      return {buffer_of(base + (size_t)s * kS * ld, rows > 0 ? (rows - 1) * ld + 2 * min(valid, SIZE) : 0), 0u};
    } else {
      return {buffer_of(base, s * kS < n ? (min(valid, SIZE) - 1) * ld + 2 * n : 0), (uint32_t)s * kS * 2};
    }
  }
  __device__ __forceinline__ void piece(const Stage& s, int i, uint8_t* lds) const {
    direct_load(s.buffer, off[i], s.at, lds + (__builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * kPieces + i) * 1024);
  }
  __device__ __forceinline__ void load(int s, int n, uint8_t* lds) const {
    const Stage st = stage(s, n);
#pragma unroll
    for (int i = 0; i < kPieces; ++i) piece(st, i, lds);
  }

  // Zeros behind the sum's last element in its last stage, of which `left` exist.
  // (Across the sum what lies behind it lies behind the buffer's end, and is zeros
  // already.)
  static constexpr bool kClear = !TR;
  __device__ __forceinline__ static void clear(int left, uint8_t* lds) {
    for (int v = threadIdx.x; v < kBytes / 16; v += NTH) {
      if (8 * ((v & 7) ^ pswz(v >> 3)) >= left) *reinterpret_cast<uint4*>(lds + 16 * v) = uint4{0, 0, 0, 0};
    }
  }

  // Where the calling lane reads a matrix operand of the rows from w0 on, whole
  // but for the bits of its tile (frag).
  __device__ __forceinline__ static uint32_t lane_at(int w0) {
    const int lane = threadIdx.x & 63, r16 = lane & 15, q = lane >> 4;
    if constexpr (TR) {
      const int r = 8 * q + (r16 >> 2);
      return r * (SIZE * 2) + ((tswz<SIZE * 2>(r) ^ (w0 >> 4)) << 5) + ((r16 & 3) << 3);
    } else {
      return (w0 + r16) * 128 + ((q ^ pswz(r16)) << 4);
    }
  }

  // The 16 rows from w0 + 16 t on, elements 32 ks .. + 31 of the stage, as a
  // matrix operand (lane: row lane % 16, elements 8 (lane / 16) .. + 7).  at:
  // lane_at + the stage's place in LDS, which is a multiple of 4096.
  __device__ __forceinline__ static u32x4 frag(uint32_t at, int t, int ks) {
    if constexpr (TR) {
      typedef __attribute__((address_space(3))) v4s* lds4;
      const uint32_t p = at ^ (t << 5);
      const v4s a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(uintptr_t)p + ks * 4 * SIZE * 2);
      const v4s b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(uintptr_t)p + ks * 4 * SIZE * 2 + SIZE);
      typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
      const u32x2 x = __builtin_bit_cast(u32x2, a), y = __builtin_bit_cast(u32x2, b);
      return u32x4{x[0], x[1], y[0], y[1]};
    } else {
      typedef const __attribute__((address_space(3))) u32x4* lds16;
      return ((lds16)(uintptr_t)(at ^ (ks << 6)))[t * 128];
    }
  }
};

// LDS as the instructions address it.
__device__ __forceinline__ uint32_t lds_address(const uint8_t* p) {
  typedef const __attribute__((address_space(3))) uint8_t* lds1;
  return (uint32_t)(uintptr_t)(lds1)p;
}

// Eight E2M1 codes times an E4M3 scale -> bfloat16, exact (6 significant bits):
// multiplied as floats, whose upper halves are the result.  (The conversion's own
// scale is a power of two, and takes no E4M3 one.)
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
// put them, a stage after they were asked for.  FAR: with their scales through a
// place of its own in LDS, two stages after: where few workgroups of small tiles wait
// for HBM (32 group16 experts, N = 4096, K = 6144, tiles of 64 rows, 700 rows: 259 us
// without, 190 with; of 128, 1000 rows: 229 and 221).  In tiles of 256 rows, whose
// bound is LDS, its accesses cost more than it brings (8192 rows: 530 us without, 557
// with), and so in the product towards the rows with tiles of 64 where there are many
// (2000 rows: 256 and 276).
template <bool TR, int SIZE, int NTH, int GRAN, bool FAR>
struct Fp4Operand : Operand<TR, SIZE, NTH> {
  static_assert(SIZE * kS == 32 * NTH, "32 codes per thread and stage");
  static constexpr bool kClear = true;
  __device__ __forceinline__ static void clear(int left, uint8_t* lds) {
    for (int v = threadIdx.x; v < SIZE * kS / 8; v += NTH) {
      const bool out = TR ? v / (SIZE / 8) >= left : 8 * ((v & 7) ^ pswz(v >> 3)) >= left;
      if (out) *reinterpret_cast<uint4*>(lds + 16 * v) = uint4{0, 0, 0, 0};
    }
  }
  static constexpr int kPer = TR ? SIZE / 32 : 2;  // pieces of a row
  const uint8_t *codes, *sf;  // uniform
  int K, rows;  // (rows: of the tile, !TR)
  uint32_t row_c, row_s;  // the thread's row (TR: column), in bytes
  // FAR: two stages' codes and scales (a word each), in the order of the threads
  static constexpr int kRing = FAR ? 2 * NTH * 20 : 16;
  static constexpr int kAhead = FAR ? 2 : 1;
  uint8_t* ring;
  u32x4 c;
  uint32_t s;

  // w, w_sf: the tile's first row (TR: of the whole sum) and column; valid rows (TR: columns)
  __device__ __forceinline__ void init(const uint8_t* w, const uint8_t* w_sf, int k, int valid, uint8_t* place) {
    ring = place;
    codes = w;
    sf = w_sf;
    K = k;
    rows = min(valid, SIZE);
    const uint32_t r = TR ? min(32 * ((int)threadIdx.x % kPer), valid - 32) : min((int)threadIdx.x / kPer, valid - 1);
    row_c = TR ? r / 2 : r * (K / 2);
    row_s = TR ? r / GRAN : r * (K / GRAN);
  }

  __device__ __forceinline__ uint8_t* slot(int st) const { return ring + (st & 1) * (kRing / 2); }

  // Stage st of a sum of n elements asked for (behind the last stage: the last one
  // again).  FAR: by two direct loads.
  __device__ __forceinline__ void fetch(int st, int n) {
    const int at = min(st, (n - 1) / kS) * kS;
    const uint8_t *pc = codes, *ps = sf;
    uint32_t oc = row_c, os = row_s;
    int left = rows;
    if (TR) {
      pc += (size_t)at * (K / 2);
      ps += (size_t)at * (K / GRAN);
      left = min(n - at, kS);
      const uint32_t r = min((int)threadIdx.x / kPer, left - 1);
      oc += r * (K / 2);
      os += r * (K / GRAN);
    } else {
      const uint32_t k = min(at + 32 * ((int)threadIdx.x % kPer), n - 32);
      oc += k / 2;
      os += k / GRAN;
    }
    if constexpr (FAR) {
      const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
      direct_load(buffer_of(pc, left * (K / 2)), oc, 0, slot(st) + wave * 1024);
      direct_load_small<GRAN == 16>(buffer_of(ps, left * (K / GRAN)), os, 0, slot(st) + NTH * 16 + wave * 256);
    } else {
      c = *reinterpret_cast<const u32x4*>(pc + oc);
      if (GRAN == 16) s = *reinterpret_cast<const uint16_t*>(ps + os);
      else s = ps[os];
    }
  }

  // What was fetched into stage buffer lds, eight codes at a time, and then a later
  // stage asked for.
  static constexpr int kPieces = 5;
  struct Stage { int st, n; };
  __device__ __forceinline__ Stage stage(int st, int n) const { return {st, n}; }
  __device__ __forceinline__ void piece(const Stage& of, int j, uint8_t* lds) {
    if (j == 4) {
      fetch(of.st + kAhead, of.n);
      return;
    }
    if (FAR && j == 0) {
      c = *reinterpret_cast<const u32x4*>(slot(of.st) + threadIdx.x * 16);
      s = *reinterpret_cast<const uint32_t*>(slot(of.st) + NTH * 16 + threadIdx.x * 4);
    }
    const int row = threadIdx.x / kPer, piece = threadIdx.x % kPer;
    // (TR: pieces 256 bytes apart write the two halves of a chunk in turn, so that
    // 16 lanes write to all 64 banks)
    const bool swap = TR && (piece & 4);
    uint32_t at = TR ? row * (SIZE * 2) + ((2 * piece ^ tswz<SIZE * 2>(row)) << 5) + (swap ? 16 : 0) : row * 128 + ((4 * piece ^ pswz(row)) << 4);
    asm volatile("" : "+v"(at));
    u32x4 v;
    const uint32_t codes = swap ? c[j ^ 1] : c[j];
    if (GRAN == 16) v = dq8_scaled_bf16(codes, e4m3_to_f32((s >> (8 * (j >> 1))) & 0xFFu));
    else v = __builtin_bit_cast(u32x4, dq8_bf16(codes, ue8m0_to_f32(s)));
    *reinterpret_cast<u32x4*>(lds + (TR ? at ^ ((j >> 1) << 5) ^ ((j & 1) << 4) : at ^ (j << 4))) = v;
  }
  __device__ __forceinline__ void load(int st, int n, uint8_t* lds) {
#pragma unroll
    for (int j = 0; j < kPieces; ++j) piece(stage(st, n), j, lds);
  }
};

template <bool TR, int SIZE, int NTH, int GRAN, bool FAR>
struct WeightOperand { typedef Fp4Operand<TR, SIZE, NTH, GRAN, FAR> type; };
template <bool TR, int SIZE, int NTH, bool FAR>
struct WeightOperand<TR, SIZE, NTH, 0, FAR> { typedef Operand<TR, SIZE, NTH> type; };

// A store, past the caches if asked for.  (The empty asm keeps the compiler from
// making one ordinary store of the two.)
template <class V>
__device__ __forceinline__ void store(const V& v, V* to, bool past) {
  if (past) {
    asm volatile("" ::: "memory");
    __builtin_nontemporal_store(v, to);
    asm volatile("" ::: "memory");
  } else {
    *to = v;
  }
}

// Every wave's LDS accesses done, and its memory accesses but the LEFT newest
// (LEFT <= 63), and a barrier.
template <int LEFT>
__device__ __forceinline__ void wait_all() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070 | (LEFT & 15) | (LEFT >> 4) << 14);  // vmcnt(LEFT) lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The wave's own loads but the LEFT newest.
template <int LEFT>
__device__ __forceinline__ void wait_vm() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (LEFT & 15) | (LEFT >> 4) << 14);
  asm volatile("" ::: "memory");
}

// Every wave's loads but the `left` (0, 4, 8 or 16) newest accesses done, and a barrier.
__device__ __forceinline__ void wait_loads(int left) {
  if (left == 0) wait_all<0>();
  else if (left == 4) wait_all<4>();
  else if (left == 8) wait_all<8>();
  else wait_all<16>();
}

// ---------------------------------------------------------------------------
// the tiled product

// What bounds it.  One expert of 8192 x 8192 x 6144: 607 us, 1.36 PFLOP/s, where a
// library's plain product of 8192^3 reaches 1.42 on the same card; the matrix
// instructions are busy in two cycles of three at a clock that the card's power holds
// at 1.85 GHz.  A wave takes 128 x 64 outputs (12 KB of LDS reads for 32
// products; with 64 x 64, as in the tiles of 128, LDS becomes the bound: the sums of
// dW of 65536 rows of 4 experts, N = 4096, K = 6144, 2692 us in tiles of 256, 3630 in
// tiles of 128).  With ragged experts the weights' bytes and short last tiles come on
// top: 16384 rows of 64 experts, N = 4096, K = 6144, 1031 us, of which the weights alone
// would take 655 and the products alone 600.  dW: 620 us for 16384 more rows and 270
// for writing 1.6 GB, which does not overlap with it: two tiles per CU (of 128 rows)
// have the same 260 us.
//
// P x Q outputs per workgroup: P along the rows (TN: along N), Q along the
// output's contiguous side; WP x WQ waves.  blockIdx.y: the part of the sum (more
// than one: to a.part as float32, which grouped_sum adds up).  GRAN: 0, or FP4 weights' group.  NB:
// 3 where the Q side is asked for two stages ahead (in LDS bfloat16 has three then, the
// P side two), else 2.  MANY: a workgroup takes a.many tiles next to each
// other along Q, the first loads of one on their way while the one before is
// stored: for short sums, where finding the expert and waiting for a lone stage is
// most of a tile's time.  (2: sums of one stage, whose room is that of one.)
template <int FORM, int GRAN, int P, int Q, int WP, int WQ, int NB, int MANY>
__global__ __launch_bounds__(WP * WQ * 64, P * Q / (WP * WQ) > 8192 ? 1 : 2) void grouped_tile_kernel(GroupedArgs a) {
  constexpr int NTH = WP * WQ * 64;
  constexpr int NP = P / WP / 16, NQ = Q / WQ / 16;  // a wave's 16-row tiles
  typedef Operand<FORM == TN, P, NTH> OpP;
  typedef typename WeightOperand<FORM != NT, Q, NTH, GRAN, NB == 3>::type OpQ;
  constexpr bool kFar = GRAN == 0 && NB == 3, kFarCodes = GRAN != 0 && NB == 3;
  constexpr int kQ = GRAN ? 2 : NB;  // stages of the Q side in LDS
  constexpr int kLeft = kFarCodes ? 2 : kFar ? OpQ::kPieces : 0;  // a later stage's loads on their way at a handover
  __shared__ __attribute__((aligned(4096))) uint8_t s_p[(MANY == 2 ? 1 : 2) * OpP::kBytes], s_q[kQ * OpQ::kBytes];
  __shared__ __attribute__((aligned(16))) uint8_t s_ring[kFarCodes ? 2 * NTH * 20 : 16];
  __shared__ __attribute__((aligned(16))) uint8_t s_turn[MANY ? WP * WQ * 4096 : 16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, q4 = lane >> 4;
  const int outs = FORM == NT ? a.N : a.K;  // the output's contiguous side
  const int nq = MANY ? ((outs + Q - 1) / Q + a.many - 1) / a.many : (outs + Q - 1) / Q;
  const int tile = tile_of(blockIdx.x, a.group);
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
  if constexpr (FORM == TN) {
    r.r0 = __builtin_amdgcn_readfirstlane(r.r0);
    r.n = __builtin_amdgcn_readfirstlane(r.n);
    // (an expert without rows is left as it is: a sum of nothing would make 0.0 of its -0.0, and
    // takes reading and writing it: 2048 rows of 8 of 64 experts, N = 4096, K = 6144, float32:
    // 3060 us so, 496 us without)
    if (a.accumulate && r.n == 0) return;
  }
  int tp, tq;
  tile_at(r.i, r.np, nq, &tp, &tq);
  const int p0 = tp * P;
  int q0 = tq * Q * (MANY ? a.many : 1);
  const int q_end = MANY ? min(outs, q0 + Q * a.many) : outs;
  const int pn = (FORM == TN ? a.N : r.n) - p0;  // what exists of the tile
  // the stages [s0, s1) of the sum, which ends at element `sum` here
  const int whole = FORM == NT ? a.K : FORM == NN ? a.N : r.n;
  const int per = ((whole + kS - 1) / kS + a.parts - 1) / a.parts;
  const int s0 = min((int)blockIdx.y * per, (whole + kS - 1) / kS), s1 = min(s0 + per, (whole + kS - 1) / kS);
  const int sum = min(whole, s1 * kS), tail = sum & (kS - 1);
  const int wp = (wave / WQ) * (P / WP), wq = (wave % WQ) * (Q / WQ);

  OpP op;
  OpQ oq;
  auto aim = [&]() __attribute__((always_inline)) {  // the Q side at q0
    const int qn = outs - q0;
    if constexpr (FORM == TN) {
      oq.init(a.q + (size_t)r.r0 * a.K + q0, 2 * a.K, qn);
    } else {
      // the weights' first row and column of the tile
      const size_t row = (size_t)r.e * a.N + (FORM == NT ? q0 : 0);
      const int col = FORM == NT ? 0 : q0;
      if constexpr (GRAN != 0) {
        oq.init(a.w + row * (a.K / 2) + col / 2, a.w_sf + row * (a.K / GRAN) + col / GRAN, a.K, qn, s_ring);
        if (s1 > s0) {
          oq.fetch(s0, sum);
          if constexpr (kFarCodes) oq.fetch(s0 + 1, sum);
        }
      } else {
        oq.init(a.q + row * a.K + col, 2 * a.K, qn);
      }
    }
  };
  if constexpr (FORM == TN) op.init(a.p + (size_t)r.r0 * a.N + p0, 2 * a.N, pn);
  else op.init(a.p + (size_t)(r.r0 + p0) * whole, 2 * whole, pn);
  aim();

  v4f acc[NQ][NP];
  // Half of the row tiles at a time (a phase): 16 products per wave at 128 x 64.
  constexpr int NH = NP / 2, kLess = NH > 2 ? NH / 2 : NH;
  u32x4 fq[2][NQ], fp[2][NH];
  const uint32_t at_q = OpQ::lane_at(wq) + lds_address(s_q), at_p = OpP::lane_at(wp) + lds_address(s_p);
  auto read_q = [&](uint32_t buf, int ks) __attribute__((always_inline)) {
    uint32_t at = at_q + buf;
    asm volatile("" : "+v"(at));  // (the tiles' addresses are formed anew: registers are short)
#pragma unroll
    for (int i = 0; i < NQ; ++i) fq[ks][i] = OpQ::frag(at, i, ks);
  };
  auto read_p = [&](uint32_t buf, int ks, int h, int n) __attribute__((always_inline)) {
    uint32_t at = at_p + buf;
    asm volatile("" : "+v"(at));
#pragma unroll
    for (int j = 0; j < n; ++j) fp[h][j] = OpP::frag(at, NH * h + j, ks);
  };
  auto multiply_one = [&](int ks, int h, int j, int i) __attribute__((always_inline)) {
    v4f& c = acc[i][NH * h + j];
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, fq[ks][i]), __builtin_bit_cast(v8bf, fp[h][j]), c, 0,
                                                0, 0);
  };
  auto multiply = [&](int ks, int h, int n) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < n; ++j)
#pragma unroll
      for (int i = 0; i < NQ; ++i) multiply_one(ks, h, j, i);
    __builtin_amdgcn_sched_barrier(0);
  };
  // A stage's loads have landed, and every wave has read the one before; what lies
  // behind the sum in its last stage is cleared.
  int stores = 0;  // newer than a tile's first loads
  bool lone = false;  // (a lone stage's P side is cleared once)
  auto handover = [&](bool last, uint32_t pb, uint32_t qb) __attribute__((always_inline)) {
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (MANY) wait_loads(stores);
    else wait_all<kLeft>();
    stores = 0;
    if ((OpQ::kClear || (OpP::kClear && !lone)) && tail && last) {
      if (OpP::kClear && !lone) OpP::clear(tail, s_p + pb);
      if constexpr (OpQ::kClear) OpQ::clear(tail, s_q + qb);
      wait_all<MANY ? 63 : kLeft>();
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  uint32_t pb = 0, qb = 0;  // where the stage at hand lies
  auto next_q = [](uint32_t b) __attribute__((always_inline)) { return b + OpQ::kBytes == kQ * OpQ::kBytes ? 0 : b + OpQ::kBytes; };
  // TILES: of a wave's row tiles, those that exist (by halves; by quarters of 8).
  // Others are neither read nor multiplied, so that an expert's short last tile takes
  // as much less time (halves of 8 only, 16384 rows of 64 experts, N = 4096, K = 6144:
  // 1050 us, quarters 1031; dx 1020 and 1000; of 4: quarters gain nothing).
  auto stages = [&](auto TILES) __attribute__((always_inline)) {
    constexpr int n0 = TILES.value < NH ? TILES.value : NH, n1 = TILES.value - n0;  // the phases' halves
    constexpr bool some = n0 > 0, both = n1 > 0;
    // A stage in four phases: the operands of a phase come while the one before
    // multiplies.  The one barrier lies before the last phase, whose operands are
    // in registers: behind it the next stage's first operands are read, and the
    // loads of a later stage go between the products.
    auto three = [&]() __attribute__((always_inline)) {
      if constexpr (both) read_p(pb, 0, 1, n1);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (some) {
        multiply(0, 0, n0);
        read_q(qb, 1);
        read_p(pb, 1, 0, n0);
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (both) {
        multiply(0, 1, n1);
        read_p(pb, 1, 1, n1);
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (some) multiply(1, 0, n0);
    };
    if constexpr (some) {
      read_q(0, 0);
      read_p(0, 0, 0, n0);
    }
    for (int s = s0; MANY < 2 && s < s1 - 1; ++s) {
      three();
      const uint32_t old_p = pb, old_q = qb;
      pb ^= OpP::kBytes;
      qb = next_q(qb);
      handover(s + 2 == s1, pb, qb);
      if constexpr (some) {
        read_q(qb, 0);
        read_p(pb, 0, 0, n0);
        __builtin_amdgcn_sched_barrier(0);
      }
      constexpr int pieces = OpP::kPieces + OpQ::kPieces, n = both ? n1 * NQ : 1;
      uint8_t* lds_q = s_q + (kFar ? old_q : next_q(qb));
      const typename OpP::Stage sp = op.stage(s + 2, sum);
      const typename OpQ::Stage sq = oq.stage(s + (kFar ? 3 : 2), sum);
#pragma unroll
      for (int i = 0; i < n; ++i) {
        if constexpr (both) multiply_one(1, 1, i / NQ, i % NQ);
#pragma unroll
        for (int k = i * pieces / n; k < (i + 1) * pieces / n; ++k) {
          if (k < OpP::kPieces) op.piece(sp, k, s_p + old_p);
          else oq.piece(sq, k - OpP::kPieces, lds_q);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
    three();
    if constexpr (both) multiply(1, 1, n1);
  };
  // The first stage's loads (the newest are the Q side's farthest stage).
  // (a lone stage's P side stays where it is)
  auto start = [&](bool first) __attribute__((always_inline)) {
    if (s1 <= s0) return;
    if (!kFar && (first || s1 - s0 > 1)) op.load(s0, sum, s_p);
    if constexpr (kFarCodes) wait_vm<OpP::kPieces + 2>();  // (the first stage's codes)
    oq.load(s0, sum, s_q);
    if constexpr (kFar) {
      op.load(s0, sum, s_p);
      oq.load(s0 + 1, sum, s_q + OpQ::kBytes);
    }
  };
  start(true);
  const float gs = GRAN && a.w_gs ? a.w_gs[r.e] : 1.0f;
  const size_t row0 = FORM == TN ? (size_t)r.e * a.N + p0 : (size_t)(r.r0 + p0);
  const bool one = a.parts == 1, f32 = a.out_f32 || !one, add = FORM == TN && one && a.accumulate, past = one && a.stream;
  void* out = one ? a.out : a.part + (size_t)blockIdx.y * (FORM == TN ? (size_t)a.E * a.N : (size_t)a.M) * outs;
  for (;;) {
#pragma unroll
  for (int i = 0; i < NQ; ++i)
#pragma unroll
    for (int j = 0; j < NP; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  if (s1 > s0) {
    pb = qb = 0;
    handover(s1 - s0 == 1, 0, 0);
    if constexpr (MANY < 2) {
      op.load(s0 + 1, sum, s_p + OpP::kBytes);
      if constexpr (kFar) oq.load(s0 + 2, sum, s_q + 2 * OpQ::kBytes);
      else oq.load(s0 + 1, sum, s_q + OpQ::kBytes);
    }
    if (FORM == TN || pn > wp + 16 * (NP - kLess)) stages(std::integral_constant<int, NP>{});
    else if (kLess < NH && pn > wp + 16 * NH) stages(std::integral_constant<int, kLess < NH ? NP - kLess : 0>{});
    else if (pn > wp + 16 * (NH - kLess)) stages(std::integral_constant<int, NH>{});
    else if (kLess < NH && pn > wp) stages(std::integral_constant<int, kLess < NH ? NH - kLess : 0>{});
    else stages(std::integral_constant<int, 0>{});
  }
  if constexpr (GRAN != 0) {
#pragma unroll
    for (int i = 0; i < NQ; ++i)
#pragma unroll
      for (int j = 0; j < NP; ++j) acc[i][j] *= gs;
  }
  // Out through LDS, 16 rows of a wave's 64 columns at a time, so that whole lines
  // are written (E = 16, N = 4096, K = 6144, float32: 8192 rows' dW 731 -> 704 us);
  // past the caches where the output is larger than the last one (687 us; 64
  // experts of 2048 x 2048, 16384 rows 367 -> 286 us).
  static_assert(Q / WQ == 64 && (MANY || WP * WQ * 4096 <= 2 * OpP::kBytes), "4 KB per wave");
  if constexpr (MANY) wait_all<63>();  // (every wave is done with the stages; `turn` lies elsewhere)
  else wait_all<0>();                  // (and no load is left that would write to it)
  v4f* turn = reinterpret_cast<v4f*>(MANY ? s_turn : s_p) + wave * 256;  // [16][16], piece c of row r at c ^ r
  const int q00 = q0, qn = outs - q0;
  const bool again = MANY && q0 + Q < q_end;
  if (again) {
    q0 += Q;
    aim();
    start(false);
    lone = s1 - s0 == 1;
  }
  // MANY: every store is issued, dropped where the tile has no such row or column,
  // so that their number is known to the next wait for loads.
  const int eb = f32 ? 4 : 2;
  const __amdgpu_buffer_rsrc_t to = __builtin_amdgcn_make_buffer_rsrc(static_cast<uint8_t*>(out) + (row0 * outs + q00) * eb, 0,
                                                                       min(pn, P) * outs * eb, 0x00020000);
  auto drop = [&](const u32x4& x, int row, int q) __attribute__((always_inline)) {
    const uint32_t at = q < qn ? (uint32_t)(row * outs + q) * eb : 0xFFFFFFFFu;
    __builtin_amdgcn_raw_buffer_store_b128(x, to, at, 0, 0);
  };
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    const int p16 = wp + 16 * j;
    if (!MANY && p16 >= pn) break;
#pragma unroll
    for (int i = 0; i < NQ; ++i) turn[r16 * 16 + ((4 * i + q4) ^ r16)] = acc[i][j];
    __builtin_amdgcn_wave_barrier();
    if (f32) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int row = 4 * k + q4, q = wq + 4 * r16;
        v4f v = turn[row * 16 + (r16 ^ row)];
        if constexpr (MANY) {
          drop(__builtin_bit_cast(u32x4, v), p16 + row, q);
          continue;
        }
        if (p16 + row >= pn || q >= qn) continue;
        v4f* o = reinterpret_cast<v4f*>(static_cast<float*>(out) + (row0 + p16 + row) * outs + q00 + q);
        if (add) v += *o;
        store(v, o, past);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int row = 8 * k + (lane >> 3), c = 2 * (lane & 7), q = wq + 4 * c;
        v4f v = turn[row * 16 + (c ^ row)], w = turn[row * 16 + ((c + 1) ^ row)];
        u32x4* o = reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out) + (row0 + p16 + row) * outs + q00 + q);
        const bool there = p16 + row < pn && q < qn;  // (a multiple of 8 columns exist)
        if (add && there) {
          const u32x4 b = *o;
          v += v4f{u2f(b[0] << 16), u2f(b[0] & 0xFFFF0000u), u2f(b[1] << 16), u2f(b[1] & 0xFFFF0000u)};
          w += v4f{u2f(b[2] << 16), u2f(b[2] & 0xFFFF0000u), u2f(b[3] << 16), u2f(b[3] & 0xFFFF0000u)};
        }
        const u32x4 x = {bf16_bits(v[0]) | (bf16_bits(v[1]) << 16), bf16_bits(v[2]) | (bf16_bits(v[3]) << 16),
                         bf16_bits(w[0]) | (bf16_bits(w[1]) << 16), bf16_bits(w[2]) | (bf16_bits(w[3]) << 16)};
        if constexpr (MANY) drop(x, p16 + row, q);
        else if (there) store(x, o, past);
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
  if constexpr (MANY) stores = f32 ? 4 * NP : 2 * NP;
  if (!again) break;
  }
  // (no load into LDS is left behind when the wave ends)
  if constexpr (MANY) wait_loads(stores);
}

// The sum of the parts, in order: eight outputs per thread.  Rows of no expert
// (TN: none) are left as they are.
template <bool TN_>
__global__ __launch_bounds__(256) void grouped_sum_kernel(GroupedArgs a, int outs) {
  const long long rows = TN_ ? (long long)a.E * a.N : a.M, i = ((long long)blockIdx.x * 256 + threadIdx.x) * 8;
  if (i >= rows * outs) return;
  if (!TN_) {
    const int r = (int)(i / outs);
    if (r < min(max(a.offsets[0], 0), a.M) || r >= min(max(a.offsets[a.E], 0), a.M)) return;
  }
  if (TN_ && a.accumulate) {
    const int e = (int)(i / outs / a.N);
    if (min(max(a.offsets[e + 1], 0), a.M) <= min(max(a.offsets[e], 0), a.M)) return;  // (nothing to add, no parts)
  }
  v4f v = {0.f, 0.f, 0.f, 0.f}, w = v;
#pragma unroll 4
  for (int p = 0; p < a.parts; ++p) {
    const v4f* q = reinterpret_cast<const v4f*>(a.part + p * rows * outs + i);
    v += q[0];
    w += q[1];
  }
  if (a.out_f32) {
    v4f* o = reinterpret_cast<v4f*>(static_cast<float*>(a.out) + i);
    if (TN_ && a.accumulate) v += o[0], w += o[1];
    o[0] = v;
    o[1] = w;
  } else {
    u32x4* o = reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.out) + i);
    if (TN_ && a.accumulate) {
      const u32x4 b = *o;
      v += v4f{u2f(b[0] << 16), u2f(b[0] & 0xFFFF0000u), u2f(b[1] << 16), u2f(b[1] & 0xFFFF0000u)};
      w += v4f{u2f(b[2] << 16), u2f(b[2] & 0xFFFF0000u), u2f(b[3] << 16), u2f(b[3] & 0xFFFF0000u)};
    }
    *o = u32x4{bf16_bits(v[0]) | (bf16_bits(v[1]) << 16), bf16_bits(v[2]) | (bf16_bits(v[3]) << 16),
               bf16_bits(w[0]) | (bf16_bits(w[1]) << 16), bf16_bits(w[2]) | (bf16_bits(w[3]) << 16)};
  }
}

// ---------------------------------------------------------------------------
// few rows per expert: the stream of the weights

// A wave's chunk of 16 weight rows: whole 128-byte lines (load j: rows 8 j + lane
// / 8, bytes 16 (lane & 7)) of 64 bfloat16 or 256 FP4 elements, and the scales of
// row lane % 16.
template <int GRAN>
struct FewChunk {
  u32x4 c[2];
  u32x4 s;  // GRAN 16: 16 scales; 32: 8
};

// Sixteen (GRAN 32: eight) scales of a row from element k on; byte by byte where
// the row may end before.
template <int GRAN, bool WHOLE>
__device__ __forceinline__ u32x4 few_scales(const uint8_t* base, uint32_t row, int k, int K) {
  constexpr int n = 256 / GRAN;
  u32x4 v = {0, 0, 0, 0};
  if (WHOLE || k + 256 <= K) {
    __builtin_memcpy(&v, base + (row + k / GRAN), n);
  } else {
#pragma unroll
    for (int i = 0; i < n; ++i) v[i >> 2] |= (uint32_t)base[row + min(k / GRAN + i, K / GRAN - 1)] << (8 * (i & 3));
  }
  return v;
}

// 16 NR weight rows x 16 NG rows of x per workgroup, the sum split over its 8
// waves, chunk by chunk in turn; NC chunks of weights in flight per wave.  WHOLE:
// the sum is whole chunks.  Bound by HBM: the weights go through registers in whole
// lines, past the caches, without a barrier; x comes from L2.  8 rows of 64 experts,
// bfloat16, N = 4096, K = 6144: 62 us, 6.2 TB/s.  128 rows, group16: 168 to 197 us, 4 to
// 4.7 TB/s; decoding the codes takes about as long as fetching them.
template <int GRAN, bool WHOLE, int NR, int NG, int NC>
__global__ __launch_bounds__(512, WHOLE && NG <= (GRAN ? 1 : 2) ? 4 : 2) void grouped_few_kernel(GroupedArgs a) {
  constexpr int CK = GRAN ? 256 : 64;  // elements per chunk
  constexpr int NJ = CK / 32;          // products of 32 elements
  constexpr int ROWS = 16 * NR, XR = 16 * NG;
  __shared__ v4f s_red[8][NR][NG][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, q = lane >> 4, K = a.K, N = a.N;
  const int nq = (N + ROWS - 1) / ROWS;
  Rows r = rows_of(a.offsets, a.E, a.M, XR, nq, blockIdx.y * gridDim.x + blockIdx.x);
  if (r.e < 0) return;
  const int e = __builtin_amdgcn_readfirstlane(r.e), i0 = __builtin_amdgcn_readfirstlane(r.i);
  const int m0 = i0 / nq * XR, n0 = i0 % nq * ROWS;
  const int rows = __builtin_amdgcn_readfirstlane(r.n) - m0;  // of x, from here on
  const size_t first = (size_t)__builtin_amdgcn_readfirstlane(r.r0) + m0;

  // weights: lane's row of each load, and its 16 bytes of a line
  const uint32_t ldw = GRAN ? K / 2 : 2 * K, line = 16 * (lane & 7), last = ldw - 16;
  const size_t wrow = (size_t)e * N + n0;
  const uint8_t* wbase = (GRAN ? a.w : reinterpret_cast<const uint8_t*>(a.q)) + wrow * ldw;
  const uint8_t* sbase = GRAN ? a.w_sf + wrow * (K / (GRAN ? GRAN : 1)) : nullptr;
  const int left = N - n0 - 1;
  const int nch = (K + CK - 1) / CK;
  typedef FewChunk<GRAN> Chunk;
  auto load = [&](int c, Chunk (&w)[NR]) __attribute__((always_inline)) {
    c = min(c, nch - 1);  // (behind the last: the last again, not used)
#pragma unroll
    for (int t = 0; t < NR; ++t) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t row = min(16 * t + 8 * j + (lane >> 3), left);
        w[t].c[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(wbase + row * ldw + (WHOLE ? c * 128 + line : min(c * 128 + line, last))));
      }
      if constexpr (GRAN != 0)
        w[t].s = few_scales<GRAN, WHOLE>(sbase, __umul24(min(16 * t + r16, left), K / GRAN), c * CK, K);
    }
  };
  Chunk w[NC][NR];
#pragma unroll
  for (int i = 0; i < NC; ++i) load(wave + 8 * i, w[i]);

  // x: row r16 of each 16, elements 32 j + 8 q .. + 7 of a chunk (rows behind the
  // last repeat it: their results are not stored)
  const uint16_t* xbase = a.p + first * K;
  uint32_t xr[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) xr[g] = (uint32_t)min(16 * g + r16, rows - 1) * K + 8 * q;
  u32x4 x[NG][NJ];
  auto load_x = [&](int g, int c, int j) __attribute__((always_inline)) {
    const int k = min(c, nch - 1) * CK + 32 * j;
    x[g][j] = *reinterpret_cast<const u32x4*>(xbase + (xr[g] + (WHOLE ? k : min(k, K - 8 - 8 * q))));
  };
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int g = 0; g < NG; ++g) load_x(g, wave, j);

  v4f acc[NR][NG];
#pragma unroll
  for (int t = 0; t < NR; ++t)
#pragma unroll
    for (int g = 0; g < NG; ++g) acc[t][g] = v4f{0.f, 0.f, 0.f, 0.f};
  // the lines turned into operand order through the wave's own LDS: 16 rows of
  // 128 bytes, 16-byte piece p of row r at p ^ pswz(r)
  uint8_t* turn = reinterpret_cast<uint8_t*>(&s_red[wave][0][0][0]);
  const int wr = lane >> 3;
  const uint32_t tw0 = wr * 128 + 16 * ((lane & 7) ^ pswz(wr)), tw1 = (wr + 8) * 128 + 16 * ((lane & 7) ^ pswz(wr + 8));
  for (int c0 = 0; c0 < nch; c0 += 8 * NC) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = c0 + wave + 8 * i;
      typedef typename std::conditional<GRAN == 0, u32x4, uint32_t>::type Raw;
      Raw raw[NR][NJ];
#pragma unroll
      for (int t = 0; t < NR; ++t) {
        *reinterpret_cast<u32x4*>(turn + tw0) = w[i][t].c[0];
        *reinterpret_cast<u32x4*>(turn + tw1) = w[i][t].c[1];
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const uint8_t* p = turn + r16 * 128 + (GRAN == 0 ? 16 * ((4 * j + q) ^ pswz(r16)) : 16 * (j ^ pswz(r16)) + 4 * q);
          raw[t][j] = *reinterpret_cast<const Raw*>(p);
        }
        __builtin_amdgcn_wave_barrier();
      }
      u32x4 s[NR];
#pragma unroll
      for (int t = 0; t < NR; ++t) {
        s[t] = w[i][t].s;
        if (GRAN == 16) {  // (the lane's elements lie in every other group)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[t][j] >>= 8 * (q >> 1);
        }
      }
      if (WHOLE && c >= nch) break;  // (the wave's last)
      // (the next chunk into these registers is asked for before this one multiplies)
      if (c0 + 8 * NC < nch) load(c + 8 * NC, w[i]);
      auto operand = [&](int t, int j) __attribute__((always_inline)) {
        u32x4 v;
        if constexpr (GRAN == 0) v = raw[t][j];
        else if constexpr (GRAN == 16) v = dq8_scaled_bf16(raw[t][j], __builtin_amdgcn_cvt_f32_fp8((int)(s[t][j >> 1] >> (16 * (j & 1))), 0));
        else v = __builtin_bit_cast(u32x4, dq8_bf16(raw[t][j], ue8m0_to_f32((s[t][j >> 2] >> (8 * (j & 3))) & 0xFFu)));
        return !WHOLE && c * CK + 32 * j + 8 * q >= K ? u32x4{0, 0, 0, 0} : v;
      };
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        u32x4 A[NR];
#pragma unroll
        for (int t = 0; t < NR; ++t) A[t] = operand(t, j);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          // (zeros on both sides behind the sum's last element)
          const u32x4 b = !WHOLE && c * CK + 32 * j + 8 * q >= K ? u32x4{0, 0, 0, 0} : x[g][j];
#pragma unroll
          for (int t = 0; t < NR; ++t)
            acc[t][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, A[t]), __builtin_bit_cast(v8bf, b),
                                                                acc[t][g], 0, 0, 0);
          load_x(g, c + 8, j);  // (into the registers just used)
        }
        if (GRAN) __builtin_amdgcn_sched_barrier(0);  // (one decoding after the other: registers are short)
      }
    }
  }
  const float gs = GRAN && a.w_gs ? a.w_gs[e] : 1.0f;
  __syncthreads();  // (every wave is done with its turning place)
#pragma unroll
  for (int t = 0; t < NR; ++t)
#pragma unroll
    for (int g = 0; g < NG; ++g) s_red[wave][t][g][lane] = acc[t][g];
  __syncthreads();
  // thread: output column n0 + rn of rows rt, rt + 512 / ROWS, ..
  const int rn = tid & (ROWS - 1);
  if (n0 + rn >= N) return;
  for (int t = tid / ROWS; t < min(rows, XR); t += 512 / ROWS) {
    float v = 0.0f;
#pragma unroll
    for (int p = 0; p < 8; ++p)
      v += reinterpret_cast<const float*>(&s_red[p][rn >> 4][t >> 4][(t & 15) + 16 * ((rn & 15) >> 2)])[rn & 3];
    if (GRAN) v *= gs;
    const size_t at = (first + t) * N + n0 + rn;
    if (a.out_f32) static_cast<float*>(a.out)[at] = v;
    else static_cast<uint16_t*>(a.out)[at] = (uint16_t)bf16_bits(v);
  }
}

template <int GRAN, int NR, int NG, int NC>
hipError_t launch_few(const GroupedArgs& a, hipStream_t s) {
  const long long nq = (a.N + 16 * NR - 1) / (16 * NR), most = a.E < a.M ? a.E : a.M;
  // (a dimension of a grid has less than 2^32 threads)
  const long long n = (a.M / (16 * NG) + most) * nq, x = n < (1 << 20) ? n : 1 << 20;
  const dim3 grid((unsigned)x, (unsigned)((n + x - 1) / x)), block(512);
  if (a.K % (GRAN ? 256 : 64) == 0) hipLaunchKernelGGL((grouped_few_kernel<GRAN, true, NR, NG, NC>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((grouped_few_kernel<GRAN, false, NR, NG, NC>), grid, block, 0, s, a);
  return hipGetLastError();
}

template <int FORM, int GRAN, int P, int Q, int WP, int WQ, int NB, int MANY = 0>
hipError_t launch_tile(const GroupedArgs& args, hipStream_t s) {
  const long long outs = FORM == NT ? args.N : args.K;
  const long long nq = MANY ? ((outs + Q - 1) / Q + args.many - 1) / args.many : (outs + Q - 1) / Q;
  const long long most = args.E < args.M ? args.E : args.M;  // experts with rows
  const long long tiles = FORM == TN ? (long long)args.E * ((args.N + P - 1) / P) * nq : (args.M / P + most) * nq;
  GroupedArgs a = args;
  // Consecutive tiles per XCD.  dW of 16 experts of 16384 rows, N = 4096, K = 6144: 32
  // 926 us, 16 901, 4 898, 1 907 (64 experts of 8000 rows: 32 1082 us, 4 1063).  The
  // other forms: 32 the best or within 1% of it (8 experts of 16384 rows: 718 us, 4 748).
  const int most_group = FORM == TN ? 4 : 32;
  // (Where tiles are few, shared out evenly in two turns: as many as there will be if every expert
  // has rows and half of its last tile is empty.)
  const long long rows = args.M / P + (most + 1) / 2, likely = FORM == TN ? tiles : (rows > most ? rows : most) * nq;
  a.group = (int)(likely >= 8 * most_group ? most_group : FORM == NT ? (likely + 15) / 16 : (likely + 7) / 8);
  const long long round = 8 * (long long)a.group;  // (tile_of)
  const dim3 grid((unsigned)((tiles + round - 1) / round * round), a.parts);
  hipLaunchKernelGGL((grouped_tile_kernel<FORM, GRAN, P, Q, WP, WQ, NB, MANY>), grid, dim3(WP * WQ * 64), 0, s, a);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || a.parts == 1) return err;
  const long long n = (FORM == TN ? (long long)a.E * a.N : a.M) * outs / 8;
  hipLaunchKernelGGL((grouped_sum_kernel<FORM == TN>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, a, (int)outs);
  return hipGetLastError();
}

template <int FORM, int GRAN>
hipError_t launch_form(const GroupedArgs& a, const GroupedPlan& plan, hipStream_t s) {
  if constexpr (FORM == NT) {
    if (plan.few == 1) return launch_few<GRAN, 2, 1, GRAN ? 1 : 3>(a, s);
    if constexpr (GRAN == 0) {
      if (plan.few == 2) return launch_few<GRAN, 2, 2, 3>(a, s);
    }
  }
  if constexpr (GRAN == 0 && FORM != TN) {
    if (plan.many > 0 && (FORM == NT ? a.K : a.N) <= kS) return launch_tile<FORM, GRAN, 64, 128, 2, 2, 1, 2>(a, s);
    if (plan.many > 0) return launch_tile<FORM, GRAN, 64, 128, 2, 2, 2, 1>(a, s);
  }
  if (plan.tile == 256) return launch_tile<FORM, GRAN, 256, 256, 2, 4, GRAN ? 2 : 3>(a, s);
  if constexpr (FORM == TN) {
    if (plan.tile == 64 && a.N > 64) return launch_tile<FORM, GRAN, 128, 64, 4, 1, 2>(a, s);
  }
  if (plan.tile == 64) {
    if constexpr (GRAN != 0) {
      if (FORM == NT || plan.far) return launch_tile<FORM, GRAN, 64, 128, 2, 2, 3>(a, s);
    }
    if constexpr (GRAN == 0 || FORM != NT) return launch_tile<FORM, GRAN, 64, 128, 2, 2, 2>(a, s);
  }
  return launch_tile<FORM, GRAN, 128, 128, 2, 2, FORM == TN ? 2 : 3>(a, s);
}

}  // namespace

// Stages of a sum (an average one's).
static long long stages_of(int form, long long M, long long E, long long N, long long K) {
  const long long most = E < M ? E : M;
  return ((form == NT ? K : form == NN ? N : most ? M / most : 0) + kS - 1) / kS;
}

static long long most_parts(int form, long long M, long long E, long long N, long long K) {
  const long long stages = stages_of(form, M, E, N, K);
  return stages < 16 ? 1 : stages / 4 > 32 ? 32 : stages / 4;
}

// Which kernel and tile, by the rows per expert with rows (M / most) and by how many
// tiles there are for the 256 CUs.  N = 4096, K = 6144 unless said; with smaller weights
// the borders move (1111 rows of 40 experts, 1000 x 696: 19.8 us in tiles of 128, as
// chosen, 17.3 of 64).  The host does not know the offsets: rows are taken to be spread
// over the experts within a factor of a few.  The stream of the weights reads an
// expert's matrix once per 16 or 32 of its rows, and is the slower the more of all rows
// one expert has (384 rows of 64 experts: 587 us spread evenly, 712 with three quarters
// in one; with all in one 217 us, where a call with that expert alone takes 41; 3000 rows
// of 512 experts, 2048 x 2048: 1065, 1168; 601 and 36).
// - the stream of the weights.  bfloat16, 64 experts: up to 6 rows with 16 rows of x
//   per workgroup (380 rows 465 us, with 32 463; 500 rows 496 and 485), up to 12 with 32
//   (750 rows 520 us, tiles of 64 564; 1000 rows 574 and 565).  FP4, 32 group16 experts:
//   up to 14 with 16 (400 rows 178 us, tiles of 64 185; 480 rows 208 and 190).
// - tiles of 256 x 256 where there are 256 of them, bfloat16 from the first row on
//   (64 experts, 4000 rows: 607 us, 128 x 128 674, 64 x 128 710; 1000 rows 579, 573,
//   565), FP4 from 192 rows per expert on (32 experts, 3500 rows, group32: 394 us, 128 x
//   128 321; 6000 rows 453 and 473).
// - tiles of 128 x 128 where there are 256, FP4 from 28 (dx 64) rows per expert on
//   (group16, 700 rows: 218 us, 64 x 128 190; 1000 rows 221 and 243; dx of 1500 rows 236
//   and 225, group32 dx of 2500 rows 257 and 273).
// - tiles of 64 x 128 else (dx of 600 rows of 8 experts, N = K = 4096: 70 us, 128 x 128
//   73).  dW: 128 x 128, and 64 x 128 or 128 x 64 for a factor no larger than 64.
//
// With fewer than 256 tiles the sums are split so that there are up to 512, four
// stages of 64 elements at least to a part (a stage of a lone workgroup takes 0.5
// us, its loads' latency), where that saves more than the 6 us of adding the parts:
// 60 rows of one expert, N = K = 4096: dx 44 -> 20 us; dW of 8192 rows of one
// expert, 64 x 4096: 94 -> 28 us.  (Up to 256 parts times tiles: 300 rows' dx 43 us,
// with up to 512 27 us.)
GroupedPlan grouped_plan(int form, long long M, long long E, long long N, long long K, int gran) {
  const long long most = E < M ? E : M, outs = form == NT ? N : K;
  // Row tiles over `most` experts with rows: about half of each expert's last one is empty.
  auto tiles = [&](int P, int Q) {
    const long long n = (M + P / 2 * most) / P, rows = form == TN ? E * ((N + P - 1) / P) : n > most ? n : most;
    return rows * ((outs + Q - 1) / Q);
  };
  GroupedPlan p{0, 128, 1, 0, 0};
  if (form == TN) {
    if (N > 128 && K > 128 && tiles(256, 256) >= 256) p.tile = 256;
    else if (N <= 64 || K <= 64) p.tile = 64;  // (a low-rank factor's: 4000 rows, 64 experts, 32 x 6144 28 -> 21 us)
  } else {
    if (form == NT && M <= (gran ? 14 : 6) * most) p.few = 1;
    else if (form == NT && M <= 12 * most) p.few = 2;
    if (p.few) return p;
  }
  // Short sums: several tiles per workgroup, so that there are about 768 (three per
  // CU), and for one stage this form in any case.  64 experts, bfloat16, N = 32, K =
  // 6144, dx of 4000 rows 45 -> 21 us (512 workgroups 24 us, 1024 22 us); two stages,
  // N = 128, K = 4096, float32: 37 -> 28 us.
  const long long stages = stages_of(form, M, E, N, K);
  if (form != TN && gran == 0 && stages <= 2) {
    const long long n = tiles(64, 128) / 768;
    p.many = n > 8 ? 8 : n > 1 || stages == 2 ? (int)n : 1;
    if (p.many > 1 || stages == 1) return p;
  }
  p.many = 0;
  if (form != TN) {
    if (tiles(256, 256) >= 256 && outs > 128 && (gran == 0 || M >= 192 * most)) p.tile = 256;
    else if (tiles(128, 128) >= 256 && (gran == 0 || M > (form == NT ? 28 : 64) * most)) p.tile = 128;
    else p.tile = 64;
  }
  const long long n = p.tile == 256 ? tiles(256, 256) : p.tile == 128 || form == TN ? tiles(128, 128) : tiles(64, 128);
  p.parts = (int)most_parts(form, M, E, N, K);  // (1 without rows)
  if (p.parts > 512 / n) p.parts = (int)(512 / n);
  if (n >= 256 || p.parts < 2 || stages * (p.parts - 1) < 18 * p.parts) p.parts = 1;
  p.far = n * p.parts <= 512;
  return p;
}

long long grouped_part_floats(int form, long long M, long long E, long long N, long long K) {
  const long long outs = form == NT ? N : K, nq = (outs + 127) / 128;
  const long long parts = most_parts(form, M, E, N, K);
  if (parts < 2) return 0;
  if (form == TN) {
    const long long n = E * ((N + 127) / 128) * nq;  // (N or K <= 64: tiles of 64 are as many)
    return n >= 256 ? 0 : (parts < 512 / n ? parts : 512 / n) * E * N * K;
  }
  // (fewer than 256 tiles have no more rows than this: one expert per tile at
  // least, 64 rows and half a tile of each expert at most)
  long long rows = E * nq < 256 ? M : 256 / nq;
  if (rows > M || form == NT) rows = M;
  if (form == NT && E * nq >= 256) return 0;  // (what is not `few` has rows for every expert)
  const long long all = parts * rows * outs, cap = 512LL * 96 * 128;
  return all < cap ? all : cap;
}

hipError_t launch_grouped(const GroupedArgs& args, int form, hipStream_t s) {
  GroupedArgs a = args;
  const GroupedPlan plan = grouped_plan(form, a.M, a.E, a.N, a.K, a.gran);
  const long long outs = form == TN ? (long long)a.E * a.N * a.K : (long long)a.M * (form == NT ? a.N : a.K);
  a.stream = outs * (a.out_f32 ? 4 : 2) > (256LL << 20);
  a.parts = plan.parts;
  a.many = plan.many;
  if (form == TN) return launch_form<TN, 0>(a, plan, s);
  if (a.gran == 16) return form == NT ? launch_form<NT, 16>(a, plan, s) : launch_form<NN, 16>(a, plan, s);
  if (a.gran == 32) return form == NT ? launch_form<NT, 32>(a, plan, s) : launch_form<NN, 32>(a, plan, s);
  return form == NT ? launch_form<NT, 0>(a, plan, s) : launch_form<NN, 0>(a, plan, s);
}

}  // namespace moefp4
