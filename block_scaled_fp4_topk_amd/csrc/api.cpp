// C-ABI entry points of libmoefp4: argument validation, workspace planning
// and the launch sequence on the caller's stream.  No allocation, no
// synchronisation; every check runs before the first launch.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <mutex>
#include <string>

#include "../../include/moefp4.h"
#include "kernels.h"

namespace {

thread_local std::string g_err;
thread_local hipEvent_t* g_stage_events = nullptr;
thread_local int g_wait_looks = moefp4::kFewLooks;


moefp4_status fail(moefp4_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_err = buf;
  return st;
}

moefp4_status ok() {
  g_err.clear();
  return MOEFP4_OK;
}

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

struct Layout {
  size_t flags, counts, offsets, sorted, slot_of, tiles, ntiles;
  size_t act_scale, x16, x8, x8_sf, sync, hmax, h, h_sf, y, route_hist, total;
  int sync_words, zero_words;  // decode: queue + done counters; + hmax words (all cleared by the route launch)
  int route_chunks, route_chunk;
  int tile_m, nt, max_tiles;
  bool a8, a4, quant_x, g16_a16;
};

moefp4_status check_problem(const moefp4_problem* p) {
  if (!p) return fail(MOEFP4_EINVAL, "problem is NULL");
  if (p->T < 0) return fail(MOEFP4_EINVAL, "T must be >= 0, got %d", p->T);
  if (p->E < 1 || p->E > moefp4::kMaxExperts)
    return fail(p->E < 1 ? MOEFP4_EINVAL : MOEFP4_EUNSUPPORTED, "E must be in [1, %d], got %d",
                moefp4::kMaxExperts, p->E);
  if (p->top_k < 1 || p->top_k > p->E)
    return fail(MOEFP4_EINVAL, "top_k must be in [1, E=%d], got %d", p->E, p->top_k);
  if (p->H <= 0 || p->I <= 0) return fail(MOEFP4_EINVAL, "H and I must be positive");
  if (p->gran_k != 16 && p->gran_k != 32)
    return fail(MOEFP4_EINVAL, "gran_k must be 16 or 32, got %d", p->gran_k);
  if (p->act_fmt < MOEFP4_ACT_BF16 || p->act_fmt > MOEFP4_ACT_BF16_QUANT_FP4_K32)
    return fail(MOEFP4_EINVAL, "unknown act_fmt %d", p->act_fmt);
  if (p->w13_order != MOEFP4_GATE_UP && p->w13_order != MOEFP4_UP_GATE)
    return fail(MOEFP4_EINVAL, "unknown w13_order %d", p->w13_order);
  if (p->out_fmt != MOEFP4_OUT_BF16 && p->out_fmt != MOEFP4_OUT_F32)
    return fail(MOEFP4_EINVAL, "unknown out_fmt %d", p->out_fmt);
  if (p->w_layout != MOEFP4_W_RAW && p->w_layout != MOEFP4_W_GEMM)
    return fail(MOEFP4_EINVAL, "unknown w_layout %d", p->w_layout);
  if (p->H % 32 || p->I % 32)
    return fail(MOEFP4_EINVAL, "H and I must be multiples of 32 (K blocks of the scale grid), got H=%d I=%d",
                p->H, p->I);
  if (p->act_fmt != MOEFP4_ACT_BF16 && p->gran_k == 16)
    return fail(MOEFP4_EUNSUPPORTED,
                "FP8 / FP4 activations with group16 weights (recipe (1,1,16)) are not computed: requantise "
                "the weights to group32 with fp4_requant_gran_k");
  if (p->H % 256 || p->I % 256)
    return fail(MOEFP4_EUNSUPPORTED, "this build tiles K in chunks of 256: H and I must be multiples of 256, got H=%d I=%d",
                p->H, p->I);
  const long long A = (long long)p->T * p->top_k;
  if (A > (1LL << 26)) return fail(MOEFP4_EUNSUPPORTED, "T*top_k = %lld exceeds 2^26", A);
  if (p->act_fmt == MOEFP4_ACT_FP4_UE8M0_K32 || p->act_fmt == MOEFP4_ACT_BF16_QUANT_FP4_K32) {
    // FP4 activations beyond decode sizes run on the 128-row GEMM tiles only
    if (p->H % 512 || p->I % 512)
      return fail(MOEFP4_EUNSUPPORTED, "FP4 activations need H and I multiples of 512, got H=%d I=%d", p->H,
                  p->I);
    if ((long long)p->T * p->H >= (1LL << 31) || A * p->I >= (1LL << 31) ||
        (long long)p->I * p->H >= (1LL << 31))
      return fail(MOEFP4_EUNSUPPORTED, "FP4 activations need T*H, T*top_k*I and I*H below 2^31");
  }
  return MOEFP4_OK;
}

moefp4_status plan(const moefp4_problem* p, Layout* L) {
  moefp4_status st = check_problem(p);
  if (st != MOEFP4_OK) return st;
  const size_t A = (size_t)p->T * p->top_k, E = p->E, T = p->T, H = p->H, I = p->I;
  L->a4 = p->act_fmt == MOEFP4_ACT_FP4_UE8M0_K32 || p->act_fmt == MOEFP4_ACT_BF16_QUANT_FP4_K32;
  L->quant_x = p->act_fmt == MOEFP4_ACT_BF16_QUANT_FP8_K32 || p->act_fmt == MOEFP4_ACT_BF16_QUANT_FP4_K32;
  // a8: block-scaled activations (FP8 or FP4) with h quantised the same way
  L->a8 = p->act_fmt != MOEFP4_ACT_BF16;
  L->g16_a16 = !L->a8 && p->gran_k == 16;
  const size_t active = A < E ? A : E;
  const double avg = active ? (double)A / (double)active : 0.0;
  // 16-row tiles for decode-shaped routing; 128-row tiles for the FP8 x FP4
  // prefill GEMM (needs 32-bit row offsets and its row-block shapes); else
  // 64-row tiles
  const bool gemm_ok = L->a8 && I % 512 == 0 && H % 512 == 0 &&
                       T * H < (1ull << 31) &&
                       A * I < (1ull << 31) && I * H < (1ull << 31);
  L->nt = avg > 16.0 ? (gemm_ok ? 8 : 4) : 1;
  // the decode kernels address an expert's weights and the fp16 rows of x
  // with 32-bit offsets
  if (L->nt == 1 && (I * H >= (1ull << 31) || (L->g16_a16 && T * H >= (1ull << 31))))
    return fail(MOEFP4_EUNSUPPORTED,
                "decode-shaped problem too large for the 16-row tiles: needs I*H and (16-bit activations with "
                "group16 weights) T*H below 2^31, got I*H=%zu T*H=%zu",
                I * H, T * H);
  if (p->w_layout == MOEFP4_W_GEMM && L->nt != 8)
    return fail(MOEFP4_EUNSUPPORTED,
                "GEMM-layout weights are read by the prefill GEMM only (FP8 / FP4 activations, group32, H and "
                "I multiples of 512, more than 16 assignments per active expert); this problem runs on the %s "
                "tiles: pass RAW weights",
                L->nt == 1 ? "16-row decode" : "64-row");
  L->tile_m = 16 * L->nt;
  L->max_tiles = (int)(A / L->tile_m + active);
  size_t o = 0;
  auto take = [&](size_t bytes) { const size_t at = o; o = align_up(o + bytes); return at; };
  L->flags = take(64);
  L->counts = take(E * 4);
  L->offsets = take((E + 1) * 4);
  L->sorted = take(A * 4);
  L->slot_of = take(A * 4);
  L->tiles = take((size_t)L->max_tiles * 8);
  L->ntiles = take(4);
  L->act_scale = take(L->g16_a16 ? T * 4 : 0);
  L->x16 = take(L->g16_a16 ? T * H * 2 : 0);
  L->x8 = take(L->quant_x ? (L->a4 ? T * H / 2 : T * H) : 0);
  L->x8_sf = take(L->quant_x ? T * (H / 32) : 0);
  // the single-launch decode kernel's counters, then the per-slot h maxima
  // (group16 with bf16 x): one region the route launch clears
  L->sync_words = L->nt == 1 ? moefp4::decode_sync_words(L->max_tiles) : 0;
  L->zero_words = L->sync_words + (L->g16_a16 ? (int)A : 0);
  L->sync = take((size_t)L->zero_words * 4);
  L->hmax = L->sync + (size_t)L->sync_words * 4;
  L->h = take(L->a4 ? A * I / 2 : L->a8 ? A * I : A * I * 2);
  L->h_sf = take(L->a8 ? A * (I / 32) : 0);
  L->y = take(A * H * 4);
  L->route_chunks = 0;
  L->route_chunk = 0;
  if ((long long)A > moefp4::kRouteSingleMax) {
    L->route_chunk = moefp4::route_chunk((long long)A);
    L->route_chunks = (int)((A + L->route_chunk - 1) / L->route_chunk);
  }
  L->route_hist = take((size_t)L->route_chunks * (E + 1) * 4);
  L->total = o;
  return MOEFP4_OK;
}

template <class T>
T* at(void* base, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(base) + off);
}

bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

moefp4_status hip_status(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(MOEFP4_EHIP, "%s: %s", what, hipGetErrorString(e));
  return MOEFP4_OK;
}

// stage boundary events of moefp4_set_stage_events (timing only)
moefp4_status stage_mark(int i, hipStream_t s) {
  return g_stage_events ? hip_status(hipEventRecord(g_stage_events[i], s), "stage event")
                        : MOEFP4_OK;
}

moefp4_status route_into(const moefp4_problem* p, const Layout& L, const int32_t* ids,
                         int32_t* counts, int32_t* offsets, int32_t* sorted, int32_t* slot_of,
                         void* ws, uint32_t* zero_words, int n_zero, const void* x, float* row_scale,
                         uint16_t* x16, uint8_t* x8, uint8_t* x8_sf, hipStream_t s) {
  moefp4::RouteOut o;
  o.counts = counts;
  o.offsets = offsets;
  o.sorted_assign = sorted;
  o.slot_of = slot_of;
  o.tiles = at<int32_t>(ws, L.tiles);
  o.ntiles = at<int32_t>(ws, L.ntiles);
  o.flags = at<int32_t>(ws, L.flags);
  o.zero_words = zero_words;
  o.n_zero = n_zero;
  o.x = static_cast<const uint16_t*>(x);
  o.T = p->T;
  o.H = p->H;
  o.row_scale = row_scale;
  o.x16 = x16;
  o.x8 = x8;
  o.xsf = x8_sf;
  o.x_fp4 = L.a4;
  o.nchunks = L.route_chunks;
  o.chunk = L.route_chunk;
  o.hist = L.route_chunks ? at<int32_t>(ws, L.route_hist) : nullptr;
  return hip_status(moefp4::launch_route(ids, p->T * p->top_k, p->E, L.tile_m, o, s), "route");
}

// The scratch of moe_fp4_forward_static: a file-scope device array, one copy
// per GPU, that holds the forward's workspace for callers that cannot
// allocate.  Host code uses only the per-device address hipGetSymbolAddress
// returns for it (the array's name is not a device address on the host).
constexpr size_t kStaticScratchBytes = (size_t)64 << 20;

}  // namespace

static __device__ __align__(256) uint8_t scratch[kStaticScratchBytes];

namespace {

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices] = {};

// This device's copy of the scratch array (resolved once per device, with
// that device current).
moefp4_status static_scratch(void** ptr) {
  int dev = -1;
  moefp4_status st = hip_status(hipGetDevice(&dev), "hipGetDevice");
  if (st != MOEFP4_OK) return st;
  if (dev < 0 || dev >= kMaxDevices) return fail(MOEFP4_EUNSUPPORTED, "device %d beyond %d", dev, kMaxDevices);
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch_ptr[dev]) {
    void* p = nullptr;
    st = hip_status(hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)), "hipGetSymbolAddress(scratch)");
    if (st != MOEFP4_OK) return st;
    if (!p) return fail(MOEFP4_EHIP, "hipGetSymbolAddress(scratch) returned NULL");
    g_scratch_ptr[dev] = p;
  }
  *ptr = g_scratch_ptr[dev];
  return MOEFP4_OK;
}

}  // namespace

namespace {

// The forward; fused: FC1 and FC2 in one persistent launch (16-row decode
// tiles only, checked by the caller).
moefp4_status forward_impl(const moefp4_problem* p, const Layout& L, const void* x, const uint8_t* x_sf,
                           const int32_t* topk_ids, const float* topk_w, const uint8_t* w13,
                           const uint8_t* w13_sf, const float* w13_gs, const uint8_t* w2,
                           const uint8_t* w2_sf, const float* w2_gs, void* out, void* workspace,
                           size_t ws_bytes, bool fused, hipStream_t stream) {
  moefp4_status st = MOEFP4_OK;
  if (p->T == 0) return ok();
  if (!x || !topk_ids || !topk_w || !w13 || !w13_sf || !w2 || !w2_sf || !out)
    return fail(MOEFP4_EINVAL, "x, topk_ids, topk_w, w13, w13_sf, w2, w2_sf and out must be non-NULL");
  if (L.a8 && !L.quant_x && !x_sf) return fail(MOEFP4_EINVAL, "FP8 / FP4 activations need x_sf");
  if ((!L.a8 || L.quant_x) && x_sf)
    return fail(MOEFP4_EINVAL, "x_sf must be NULL for bfloat16 activations");
  if (misaligned(x, 16) || misaligned(w13, 16) || misaligned(w2, 16) || misaligned(out, 16) ||
      misaligned(w13_sf, 16) || misaligned(w2_sf, 16) || (x_sf && misaligned(x_sf, 16)))
    return fail(MOEFP4_EINVAL, "x, x_sf, w13, w13_sf, w2, w2_sf and out must be 16-byte aligned");
  if (!workspace || ws_bytes < L.total)
    return fail(MOEFP4_EWORKSPACE, "workspace of %zu bytes needed, got %zu", L.total,
                workspace ? ws_bytes : (size_t)0);
  if (misaligned(workspace, 256)) return fail(MOEFP4_EINVAL, "workspace must be 256-byte aligned");

  const int A = p->T * p->top_k;
  int32_t* counts = at<int32_t>(workspace, L.counts);
  int32_t* offsets = at<int32_t>(workspace, L.offsets);
  int32_t* sorted = at<int32_t>(workspace, L.sorted);
  int32_t* slot_of = at<int32_t>(workspace, L.slot_of);
  uint32_t* hmax = L.g16_a16 ? at<uint32_t>(workspace, L.hmax) : nullptr;
  uint32_t* zero = L.zero_words ? at<uint32_t>(workspace, L.sync) : nullptr;
  if ((st = stage_mark(0, stream)) != MOEFP4_OK) return st;
  // group16 weights with bf16 x on 16-row tiles: the route launch also
  // computes the per-token fp16 staging scales and writes the rows converted
  // with them, which FC1 copies straight to LDS
  const bool stage_f16 = L.g16_a16 && L.nt == 1;
  float* xs = L.g16_a16 ? at<float>(workspace, L.act_scale) : nullptr;
  uint16_t* x16 = L.g16_a16 ? at<uint16_t>(workspace, L.x16) : nullptr;
  // bf16 x to be quantised to FP8 or MXFP4 (+ UE8M0 per 32): also done by
  // the route launch, into the workspace
  uint8_t* x8 = L.quant_x ? at<uint8_t>(workspace, L.x8) : nullptr;
  uint8_t* x8_sf = L.quant_x ? at<uint8_t>(workspace, L.x8_sf) : nullptr;
  st = route_into(p, L, topk_ids, counts, offsets, sorted, slot_of, workspace, zero,
                  L.zero_words, (stage_f16 || L.quant_x) ? x : nullptr,
                  stage_f16 ? xs : nullptr, stage_f16 ? x16 : nullptr, x8, x8_sf, stream);
  if (st != MOEFP4_OK) return st;
  if ((st = stage_mark(1, stream)) != MOEFP4_OK) return st;

  moefp4::FcArgs a;
  memset(&a, 0, sizeof a);
  a.tiles = at<int32_t>(workspace, L.tiles);
  a.ntiles = at<int32_t>(workspace, L.ntiles);
  a.counts = counts;
  a.offsets = offsets;
  a.sorted_assign = sorted;
  a.I = p->I;
  a.H = p->H;
  a.top_k = p->top_k;
  a.w13_order = p->w13_order;

  // FC1 + SwiGLU (+ h quantisation)
  a.w = w13;
  a.wsf = w13_sf;
  a.gs = w13_gs;
  a.K = p->H;
  a.N = 2 * p->I;
  a.h_out = at<void>(workspace, L.h);
  if (L.a8) {
    a.act = L.quant_x ? x8 : x;
    a.act_sf = L.quant_x ? x8_sf : x_sf;
    a.h_sf_out = at<uint8_t>(workspace, L.h_sf);
  } else if (stage_f16) {
    a.act = x16;
    a.act_scale = xs;
    a.hmax_out = hmax;
  } else if (L.g16_a16) {
    st = hip_status(moefp4::launch_rows_to_f16(static_cast<const uint16_t*>(x), p->T, p->H, x16, xs, stream),
                    "rows_to_f16");
    if (st != MOEFP4_OK) return st;
    a.act = x16;
    a.act_scale = xs;
    a.hmax_out = hmax;
  } else {
    a.act = x;
  }
  // FC2
  moefp4::FcArgs b = a;
  b.w = w2;
  b.wsf = w2_sf;
  b.gs = w2_gs;
  b.K = p->I;
  b.N = p->H;
  b.act = at<void>(workspace, L.h);
  b.act_sf = L.a8 ? at<uint8_t>(workspace, L.h_sf) : nullptr;
  b.act_scale = nullptr;
  b.hmax_in = hmax;
  b.hmax_out = nullptr;
  b.h_out = nullptr;
  b.h_sf_out = nullptr;
  b.y_out = at<float>(workspace, L.y);
  const int mode = L.a4 ? 3 : L.a8 ? 2 : (p->gran_k == 16 ? 0 : 1);
  if ((st = stage_mark(2, stream)) != MOEFP4_OK) return st;
  if (fused) {
    // FC1 and FC2 in one persistent launch (16-row decode tiles)
    moefp4::DecodeSync y;
    y.queue = at<int32_t>(workspace, L.sync);
    y.done = y.queue + 8;
    y.err = at<int32_t>(workspace, L.flags) + 1;
    y.nx = moefp4::xcd_count();
    y.nblk1 = p->I / 64;
    y.nblk2 = p->H / 128;
    st = hip_status(moefp4::launch_fc_decode_fused(a, b, mode, y, stream), "fc1+fc2");
    if (st != MOEFP4_OK) return st;
    if ((st = stage_mark(3, stream)) != MOEFP4_OK) return st;
  } else {
    st = hip_status(L.nt == 1   ? moefp4::launch_fc_decode(a, mode, true, L.max_tiles, stream)
                    : L.nt == 8 ? moefp4::launch_fc_gemm_a8(a, true, L.a4, p->w_layout == MOEFP4_W_GEMM,
                                                            L.max_tiles, stream)
                    : L.a8      ? moefp4::launch_fc1_a8(a, L.max_tiles, stream)
                                : moefp4::launch_fc1_a16(a, p->gran_k, L.max_tiles, stream),
                    "fc1");
    if (st != MOEFP4_OK) return st;
    if ((st = stage_mark(3, stream)) != MOEFP4_OK) return st;
    st = hip_status(L.nt == 1   ? moefp4::launch_fc_decode(b, mode, false, L.max_tiles, stream)
                    : L.nt == 8 ? moefp4::launch_fc_gemm_a8(b, false, L.a4, p->w_layout == MOEFP4_W_GEMM,
                                                            L.max_tiles, stream)
                    : L.a8      ? moefp4::launch_fc2_a8(b, L.max_tiles, stream)
                                : moefp4::launch_fc2_a16(b, p->gran_k, L.max_tiles, stream),
                    "fc2");
    if (st != MOEFP4_OK) return st;
  }
  if ((st = stage_mark(4, stream)) != MOEFP4_OK) return st;

  st = hip_status(moefp4::launch_combine(b.y_out, slot_of, topk_w, p->T, p->top_k, p->H, out,
                                         p->out_fmt == MOEFP4_OUT_F32, stream),
                  "combine");
  if (st != MOEFP4_OK) return st;
  if ((st = stage_mark(5, stream)) != MOEFP4_OK) return st;
  return ok();
}

// The router's argument checks and plan.
moefp4_status gate_check(const moefp4_gate* g, int64_t T, int64_t E, int64_t H, moefp4::GatePlan* plan) {
  if (!g) return fail(MOEFP4_EINVAL, "gate is NULL");
  if (T < 0 || E < 1 || H < 8 || H % 8)
    return fail(MOEFP4_EINVAL, "need T >= 0, E >= 1 and H a positive multiple of 8, got T=%lld E=%lld H=%lld",
                (long long)T, (long long)E, (long long)H);
  if (g->top_k < 1 || g->top_k > E || g->shared < 0)
    return fail(MOEFP4_EINVAL, "need 1 <= top_k <= E=%lld and shared >= 0, got top_k=%d shared=%d", (long long)E,
                g->top_k, g->shared);
  if (g->scoring != MOEFP4_SCORE_SOFTMAX && g->scoring != MOEFP4_SCORE_SIGMOID)
    return fail(MOEFP4_EINVAL, "unknown scoring %d", g->scoring);
  if (g->w_fmt != MOEFP4_GATE_W_BF16 && g->w_fmt != MOEFP4_GATE_W_F32)
    return fail(MOEFP4_EINVAL, "unknown gate weight format %d", g->w_fmt);
  if (E > moefp4::kMaxExperts || g->shared > moefp4::kMaxExperts - E)
    return fail(MOEFP4_EUNSUPPORTED, "E + shared must be at most %d, got %lld + %d", moefp4::kMaxExperts, (long long)E,
                g->shared);
  if (g->top_k > moefp4::kGateMaxTopK)
    return fail(MOEFP4_EUNSUPPORTED, "top_k must be at most %d, got %d", moefp4::kGateMaxTopK, g->top_k);
  if (T > (1 << 24) || H > (1 << 24) || T * H >= (1ll << 40))
    return fail(MOEFP4_EUNSUPPORTED, "T and H must be at most 2^24 and T*H below 2^40");
  *plan = moefp4::gate_plan((int)T, (int)E, (int)H, g->w_fmt == MOEFP4_GATE_W_F32);
  return MOEFP4_OK;
}

// Workspace of the router: the logits, then the planes of FP32 weights.
size_t gate_need(const moefp4::GatePlan& p) { return align_up(p.most_bytes) + align_up(p.planes_bytes); }

moefp4::GateSel gate_sel(const moefp4_gate* g, int E, const float* bias) {
  return moefp4::GateSel{E, g->top_k, g->shared, g->scoring, g->renormalize != 0, g->scale, bias};
}

// A layer's checks and the places of its two forms in the workspace.
struct LayerPlan {
  Layout L;                 // the forward's (at 0)
  moefp4::GatePlan gate;
  bool few;
  size_t part, planes, ids, wts;                        // gate + forward
  size_t flags, logits, xs, x16, h, hexp, sync, parts;  // few tokens
  int ld, nwg;
  size_t total;
};

moefp4_status layer_plan(const moefp4_problem* p, const moefp4_gate* g, LayerPlan* P) {
  moefp4_status st = plan(p, &P->L);
  if (st != MOEFP4_OK) return st;
  if (!g) return fail(MOEFP4_EINVAL, "gate is NULL");
  if (p->act_fmt != MOEFP4_ACT_BF16 && !P->L.quant_x)
    return fail(MOEFP4_EINVAL, "the router takes bfloat16 x: act_fmt must be BF16 or one of the BF16_QUANT formats");
  if (g->shared < 0 || g->shared >= p->E || g->top_k != p->top_k - g->shared)
    return fail(MOEFP4_EINVAL, "need 0 <= shared < E and top_k (with the shared experts) = %d + %d, got E=%d top_k=%d",
                g->top_k, g->shared, p->E, p->top_k);
  st = gate_check(g, p->T, p->E - g->shared, p->H, &P->gate);
  if (st != MOEFP4_OK) return st;
  const size_t T = p->T, H = p->H, I = p->I, A = T * p->top_k;
  const int most = p->gran_k == 16 ? moefp4::kFewTokens : moefp4::kFewTokensG32;
  bool small = p->act_fmt == MOEFP4_ACT_BF16 && p->H <= moefp4::kFewMaxH && p->top_k <= moefp4::kFewMaxK;
  P->nwg = moefp4::cu_count();
  // (launch 2 counts FC2's steps times workgroups in 31 bits)
  if ((H / 32) * ((size_t)p->E * (I / 256) / 8 + 1) * P->nwg >= (1ull << 31)) small = false;
  P->few = small && T >= 1 && p->T <= most && A * I * 4 < (1ull << 31);
  // The total is the most that T or fewer tokens need, so that a workspace
  // serves the batches below the one it was made for.
  size_t o = 0;
  auto take = [&](size_t bytes) { const size_t at = o; o = align_up(o + bytes); return at; };
  P->total = 0;
  if (small) {
    const size_t t = p->T < most ? T : most, a = t * p->top_k;
    P->ld = p->E - g->shared <= 256 ? 256 : 512;
    P->flags = take(64);
    P->logits = take(t * P->ld * 4);
    P->xs = take(P->L.g16_a16 ? t * 4 : 0);
    P->x16 = take(P->L.g16_a16 ? t * H * 2 : 0);
    P->h = take(P->L.g16_a16 ? a * I * 2 : a * I * 4);
    P->hexp = take(P->L.g16_a16 ? a * (I / 16) : 0);
    P->sync = take((size_t)moefp4::few_sync_words(p->H) * 4);
    P->parts = take((size_t)P->nwg * 2 * 512 * 4);
    P->total = o;
  }
  if (!P->few) {
    o = P->L.total;
    P->ids = take(A * 4);
    P->wts = take(A * 4);
    P->part = take(P->gate.most_bytes);
    P->planes = take(P->gate.planes_bytes);
    // (what of the forward's own shrinks with T: the tiles and counters of its
    // 16-row form, the chunks of its grouping)
    const size_t active = A < (size_t)p->E ? A : p->E, tiles = A / 16 + active;
    o += align_up(tiles * 8) - align_up((size_t)P->L.max_tiles * 8);
    o += align_up((moefp4::decode_sync_words((int)tiles) + (P->L.g16_a16 ? A : 0)) * 4) -
         align_up((size_t)P->L.zero_words * 4);
    o += align_up((size_t)(A > moefp4::kRouteSingleMax ? moefp4::kRouteMaxChunks : 0) * (p->E + 1) * 4) -
         align_up((size_t)P->L.route_chunks * (p->E + 1) * 4);
    if (o > P->total) P->total = o;
  }
  return MOEFP4_OK;
}

struct ProjectPlan {
  size_t x16, xs, u, part, total;
  bool group;  // u by matrix instructions
  size_t ids, counts, offsets, sorted, slot_of, tiles, ntiles, flags, hist;
  int chunk, chunks, ku;
};

moefp4_status project_check(const moefp4_linear* p, ProjectPlan* P) {
  if (!p) return fail(MOEFP4_EINVAL, "linear is NULL");
  if (p->T < 0 || p->N <= 0 || p->K <= 0) return fail(MOEFP4_EINVAL, "need T >= 0, N > 0 and K > 0");
  if (p->gran_k != 16 && p->gran_k != 32) return fail(MOEFP4_EINVAL, "gran_k must be 16 or 32, got %d", p->gran_k);
  if (p->out_fmt != MOEFP4_OUT_BF16 && p->out_fmt != MOEFP4_OUT_F32)
    return fail(MOEFP4_EINVAL, "unknown out_fmt %d", p->out_fmt);
  if (p->K % 32) return fail(MOEFP4_EINVAL, "K must be a multiple of 32, got %lld", (long long)p->K);
  if (p->adapters < 0) return fail(MOEFP4_EINVAL, "adapters must be >= 0, got %d", p->adapters);
  if (p->adapters > 0 && (p->rank <= 0 || p->rank % 8))
    return fail(MOEFP4_EINVAL, "rank must be a positive multiple of 8, got %d", p->rank);
  // (tokens without one are grouped as one more)
  if (p->adapters >= moefp4::kMaxExperts)
    return fail(MOEFP4_EUNSUPPORTED, "adapters must be below %d, got %d", moefp4::kMaxExperts, p->adapters);
  if (p->adapters > 0 && p->rank > 128) return fail(MOEFP4_EUNSUPPORTED, "rank must be at most 128, got %d", p->rank);
  if (p->K % 256 || p->N % 16)
    return fail(MOEFP4_EUNSUPPORTED, "K must be a multiple of 256 and N of 16, got K=%lld N=%lld", (long long)p->K,
                (long long)p->N);
  const int64_t lim = 1ll << 32;
  if (p->T >= (1 << 24) || p->N >= lim || p->K >= lim || p->N * p->K >= lim ||
      (p->T + 127) / 128 * ((p->N + 127) / 128) >= (1ll << 24) ||
      (p->adapters > 0 && (int64_t)p->adapters * p->rank >= lim / p->N))
    return fail(MOEFP4_EUNSUPPORTED,
                "T must be below 2^24, N*K and adapters*N*rank below 2^32 and T*N below 2^38, got T=%lld N=%lld K=%lld",
                (long long)p->T, (long long)p->N, (long long)p->K);
  // Every size is the most that T or fewer tokens need, so that a workspace
  // serves the batches below the one it was made for.
  // (few tokens: rows for whole groups of 16, as many as the launch multiplies)
  const size_t T = (size_t)p->T, Tg = T <= 16 ? 16 : T <= 32 ? 32 : T <= 64 ? 64 : 128;
  size_t o = 0;
  auto take = [&](size_t bytes) { const size_t at = o; o = align_up(o + bytes); return at; };
  static_assert(moefp4::kProjectFew == 128, "Tg");
  P->x16 = take(Tg * p->K * 2);
  P->xs = take(p->gran_k == 16 ? Tg * 4 : 0);
  P->ku = p->adapters > 0 ? moefp4::project_u_parts(p->T, p->K, p->rank) : 1;
  P->u = take(p->adapters > 0 ? moefp4::project_u_rows(p->T, p->K, p->rank) * p->rank * 4 : 0);
  P->part = take((size_t)moefp4::project_part_rows(p->T, p->N, p->K) * p->N * 4);
  P->group = p->adapters > 0 && !moefp4::project_dot(p->T, p->K, p->rank);
  P->chunk = P->chunks = 0;
  if (P->group) {
    const size_t L = p->adapters + 1;
    // (one workgroup takes 21 us to group 8192 tokens)
    if (p->T > 2048) {
      P->chunk = p->T > moefp4::kRouteSingleMax ? moefp4::route_chunk(p->T) : 1024;
      P->chunks = (int)((p->T + P->chunk - 1) / P->chunk);
    }
    P->ids = take(T * 4);
    P->counts = take(L * 4);
    P->offsets = take((L + 1) * 4);
    P->sorted = take(T * 4);
    P->slot_of = take(T * 4);
    P->tiles = take((T / 32 + L) * 8);
    P->ntiles = take(4);
    P->flags = take(64);
    P->hist = take((size_t)(p->T > moefp4::kRouteSingleMax ? moefp4::kRouteMaxChunks : P->chunks) * (L + 1) * 4);
  }
  // (never 0: a caller that allocates what it is told has something to pass)
  P->total = o > 0 ? o : kAlign;
  return MOEFP4_OK;
}

}  // namespace

extern "C" {

moefp4_status moe_fp4_workspace_bytes(const moefp4_problem* p, size_t* bytes) {
  if (!bytes) return fail(MOEFP4_EINVAL, "bytes is NULL");
  Layout L;
  moefp4_status st = plan(p, &L);
  if (st != MOEFP4_OK) return st;
  *bytes = L.total;
  return ok();
}

moefp4_status moe_fp4_workspace_offsets(const moefp4_problem* p, size_t* h, size_t* h_sf, size_t* slot_of) {
  if (!h || !h_sf || !slot_of) return fail(MOEFP4_EINVAL, "h, h_sf and slot_of must be non-NULL");
  Layout L;
  moefp4_status st = plan(p, &L);
  if (st != MOEFP4_OK) return st;
  *h = L.h;
  *h_sf = L.a8 ? L.h_sf : 0;
  *slot_of = L.slot_of;
  return ok();
}

moefp4_status moe_fp4_route(const moefp4_problem* p, const int32_t* topk_ids, int32_t* counts,
                            int32_t* offsets, int32_t* sorted_assign, int32_t* slot_of,
                            void* workspace, size_t ws_bytes, hipStream_t stream) {
  Layout L;
  moefp4_status st = plan(p, &L);
  if (st != MOEFP4_OK) return st;
  if (p->T > 0 && (!topk_ids || !sorted_assign || !slot_of))
    return fail(MOEFP4_EINVAL, "topk_ids, sorted_assign and slot_of must be non-NULL");
  if (!counts || !offsets) return fail(MOEFP4_EINVAL, "counts and offsets must be non-NULL");
  if (!workspace || ws_bytes < L.total)
    return fail(MOEFP4_EWORKSPACE, "workspace of %zu bytes needed, got %zu", L.total,
                workspace ? ws_bytes : (size_t)0);
  st = route_into(p, L, topk_ids, counts, offsets, sorted_assign, slot_of, workspace, nullptr, 0,
                  nullptr, nullptr, nullptr, nullptr, nullptr, stream);
  return st == MOEFP4_OK ? ok() : st;
}

moefp4_status moe_fp4_gate_workspace_bytes(const moefp4_gate* g, int64_t T, int64_t E, int64_t H, size_t* bytes) {
  if (!bytes) return fail(MOEFP4_EINVAL, "bytes is NULL");
  moefp4::GatePlan P;
  moefp4_status st = gate_check(g, T, E, H, &P);
  if (st != MOEFP4_OK) return st;
  *bytes = gate_need(P);
  return ok();
}

moefp4_status moe_fp4_gate(const moefp4_gate* g, int64_t T, int64_t E, int64_t H, const void* x, const void* w,
                           const float* bias, int32_t* topk_ids, float* topk_w, void* workspace, size_t ws_bytes,
                           hipStream_t stream) {
  moefp4::GatePlan P;
  moefp4_status st = gate_check(g, T, E, H, &P);
  if (st != MOEFP4_OK) return st;
  if (T == 0) return ok();
  if (!x || !w || !topk_ids || !topk_w)
    return fail(MOEFP4_EINVAL, "x, w, topk_ids and topk_w must be non-NULL");
  if (misaligned(x, 16) || misaligned(w, 16) || misaligned(bias, 4) || misaligned(topk_ids, 4) || misaligned(topk_w, 4))
    return fail(MOEFP4_EINVAL, "x and w must be 16-byte aligned, bias, topk_ids and topk_w 4-byte");
  const size_t need = gate_need(P);
  if (!workspace || ws_bytes < need)
    return fail(MOEFP4_EWORKSPACE, "workspace of %zu bytes needed, got %zu", need, workspace ? ws_bytes : (size_t)0);
  if (misaligned(workspace, 256)) return fail(MOEFP4_EINVAL, "workspace must be 256-byte aligned");
  st = hip_status(moefp4::launch_gate(P, gate_sel(g, (int)E, bias), w, g->w_fmt == MOEFP4_GATE_W_F32,
                                      static_cast<const uint16_t*>(x), (int)T, (int)H,
                                      at<uint16_t>(workspace, align_up(P.part_bytes)), at<float>(workspace, 0),
                                      topk_ids, topk_w, stream),
                  "gate");
  return st == MOEFP4_OK ? ok() : st;
}

moefp4_status moe_fp4_forward(const moefp4_problem* p, const void* x, const uint8_t* x_sf,
                              const int32_t* topk_ids, const float* topk_w, const uint8_t* w13,
                              const uint8_t* w13_sf, const float* w13_gs, const uint8_t* w2,
                              const uint8_t* w2_sf, const float* w2_gs, void* out,
                              void* workspace, size_t ws_bytes, hipStream_t stream) {
  Layout L;
  moefp4_status st = plan(p, &L);
  if (st != MOEFP4_OK) return st;
  return forward_impl(p, L, x, x_sf, topk_ids, topk_w, w13, w13_sf, w13_gs, w2, w2_sf, w2_gs, out, workspace,
                      ws_bytes, false, stream);
}

moefp4_status moe_fp4_forward_fused(const moefp4_problem* p, const void* x, const uint8_t* x_sf,
                                    const int32_t* topk_ids, const float* topk_w, const uint8_t* w13,
                                    const uint8_t* w13_sf, const float* w13_gs, const uint8_t* w2,
                                    const uint8_t* w2_sf, const float* w2_gs, void* out, void* workspace,
                                    size_t ws_bytes, hipStream_t stream) {
  Layout L;
  moefp4_status st = plan(p, &L);
  if (st != MOEFP4_OK) return st;
  if (L.nt != 1)
    return fail(MOEFP4_EUNSUPPORTED,
                "the single-launch forward runs the 16-row decode tiles only (at most 16 assignments per active "
                "expert); this problem runs on the %s tiles: use moe_fp4_forward",
                L.nt == 8 ? "128-row GEMM" : "64-row");
  return forward_impl(p, L, x, x_sf, topk_ids, topk_w, w13, w13_sf, w13_gs, w2, w2_sf, w2_gs, out, workspace,
                      ws_bytes, true, stream);
}

moefp4_status moe_fp4_layer_workspace_bytes(const moefp4_problem* p, const moefp4_gate* g, size_t* bytes) {
  if (!bytes) return fail(MOEFP4_EINVAL, "bytes is NULL");
  LayerPlan P;
  moefp4_status st = layer_plan(p, g, &P);
  if (st != MOEFP4_OK) return st;
  *bytes = P.total;
  return ok();
}

moefp4_status moe_fp4_layer(const moefp4_problem* p, const moefp4_gate* g, const void* x, const void* gate_w,
                            const float* bias, const uint8_t* w13, const uint8_t* w13_sf, const float* w13_gs,
                            const uint8_t* w2, const uint8_t* w2_sf, const float* w2_gs, void* out,
                            int32_t* topk_ids, float* topk_w, void* workspace, size_t ws_bytes, hipStream_t stream) {
  LayerPlan P;
  moefp4_status st = layer_plan(p, g, &P);
  if (st != MOEFP4_OK) return st;
  if (p->T == 0) return ok();
  if (!x || !gate_w || !w13 || !w13_sf || !w2 || !w2_sf || !out)
    return fail(MOEFP4_EINVAL, "x, gate_w, w13, w13_sf, w2, w2_sf and out must be non-NULL");
  if (misaligned(x, 16) || misaligned(gate_w, 16) || misaligned(w13, 16) || misaligned(w2, 16) || misaligned(out, 16) ||
      misaligned(w13_sf, 16) || misaligned(w2_sf, 16))
    return fail(MOEFP4_EINVAL, "x, gate_w, w13, w13_sf, w2, w2_sf and out must be 16-byte aligned");
  if (misaligned(bias, 4) || misaligned(w13_gs, 4) || misaligned(w2_gs, 4) || misaligned(topk_ids, 4) ||
      misaligned(topk_w, 4))
    return fail(MOEFP4_EINVAL, "bias, w13_gs, w2_gs, topk_ids and topk_w must be 4-byte aligned");
  if (!workspace || ws_bytes < P.total)
    return fail(MOEFP4_EWORKSPACE, "workspace of %zu bytes needed, got %zu", P.total,
                workspace ? ws_bytes : (size_t)0);
  if (misaligned(workspace, 256)) return fail(MOEFP4_EINVAL, "workspace must be 256-byte aligned");
  const moefp4::GateSel sel = gate_sel(g, p->E - g->shared, bias);
  const bool w_f32 = g->w_fmt == MOEFP4_GATE_W_F32;
  const uint16_t* xb = static_cast<const uint16_t*>(x);
  if (!P.few) {
    int32_t* ids = topk_ids ? topk_ids : at<int32_t>(workspace, P.ids);
    float* wts = topk_w ? topk_w : at<float>(workspace, P.wts);
    st = hip_status(moefp4::launch_gate(P.gate, sel, gate_w, w_f32, xb, p->T, p->H, at<uint16_t>(workspace, P.planes),
                                        at<float>(workspace, P.part), ids, wts, stream),
                    "gate");
    if (st != MOEFP4_OK) return st;
    return forward_impl(p, P.L, x, nullptr, ids, wts, w13, w13_sf, w13_gs, w2, w2_sf, w2_gs, out, workspace, ws_bytes,
                        false, stream);
  }
  moefp4::FewArgs a;
  memset(&a, 0, sizeof a);
  a.g = sel;
  a.T = p->T;
  a.H = p->H;
  a.I = p->I;
  a.w13_order = p->w13_order;
  a.g16 = P.L.g16_a16;
  a.w_f32 = w_f32;
  a.out_f32 = p->out_fmt == MOEFP4_OUT_F32;
  a.x = xb;
  a.gate_w = gate_w;
  a.w13 = w13;
  a.w13_sf = w13_sf;
  a.w13_gs = w13_gs;
  a.w2 = w2;
  a.w2_sf = w2_sf;
  a.w2_gs = w2_gs;
  a.out = out;
  a.ids = topk_ids;
  a.wts = topk_w;
  a.flags = at<int32_t>(workspace, P.flags);
  a.logits = at<float>(workspace, P.logits);
  a.ld = P.ld;
  a.x16 = at<uint16_t>(workspace, P.x16);
  a.xs = at<float>(workspace, P.xs);
  a.h = at<uint16_t>(workspace, P.h);
  a.hexp = at<int8_t>(workspace, P.hexp);
  a.sync = at<int32_t>(workspace, P.sync);
  a.part = at<float>(workspace, P.parts);
  a.nwg = P.nwg;
  a.looks = g_wait_looks;
  st = hip_status(moefp4::launch_few(a, stream), "layer");
  return st == MOEFP4_OK ? ok() : st;
}

moefp4_status moe_fp4_project_workspace_bytes(const moefp4_linear* p, size_t* bytes) {
  if (!bytes) return fail(MOEFP4_EINVAL, "bytes is NULL");
  ProjectPlan P;
  moefp4_status st = project_check(p, &P);
  if (st != MOEFP4_OK) return st;
  *bytes = P.total;
  return ok();
}

moefp4_status moe_fp4_project(const moefp4_linear* p, const void* x, const uint8_t* w, const uint8_t* w_sf,
                              const float* w_gs, const void* lora_a, const void* lora_b, const int32_t* id,
                              const float* scale, void* out, void* workspace, size_t ws_bytes, hipStream_t stream) {
  ProjectPlan P;
  moefp4_status st = project_check(p, &P);
  if (st != MOEFP4_OK) return st;
  if (p->T == 0) return ok();
  if (!x || !w || !w_sf || !out) return fail(MOEFP4_EINVAL, "x, w, w_sf and out must be non-NULL");
  if (p->adapters > 0 && (!lora_a || !lora_b || !id || !scale))
    return fail(MOEFP4_EINVAL, "lora_a, lora_b, id and scale must be non-NULL with adapters");
  if (p->adapters == 0 && (lora_a || lora_b || id || scale))
    return fail(MOEFP4_EINVAL, "lora_a, lora_b, id and scale must be NULL without adapters");
  if (misaligned(x, 16) || misaligned(w, 16) || misaligned(w_sf, 16) || misaligned(out, 16) || misaligned(lora_a, 16) ||
      misaligned(lora_b, 16) || misaligned(w_gs, 4) || misaligned(id, 4) || misaligned(scale, 4))
    return fail(MOEFP4_EINVAL, "x, w, w_sf, lora_a, lora_b and out must be 16-byte aligned, w_gs, id and scale 4-byte");
  if (!workspace || ws_bytes < P.total)
    return fail(MOEFP4_EWORKSPACE, "workspace of %zu bytes needed, got %zu", P.total,
                workspace ? ws_bytes : (size_t)0);
  if (misaligned(workspace, 256)) return fail(MOEFP4_EINVAL, "workspace must be 256-byte aligned");
  // (workgroups store while others still read)
  const size_t N = p->N, K = p->K, LR = (size_t)p->adapters * p->rank;
  const struct { const void* p; size_t n; } in[] = {{x, p->T * K * 2}, {w, N * K / 2}, {w_sf, N * (K / p->gran_k)}, {w_gs, 4},
                                                    {lora_a, LR * K * 2}, {lora_b, LR * N * 2}, {id, (size_t)p->T * 4},
                                                    {scale, (size_t)p->adapters * 4}};
  const char* o = static_cast<const char*>(out);
  const size_t on = p->T * N * (p->out_fmt == MOEFP4_OUT_F32 ? 4 : 2);
  for (const auto& b : in) {
    const char* q = static_cast<const char*>(b.p);
    if (q && q < o + on && o < q + b.n) return fail(MOEFP4_EINVAL, "out overlaps an input");
  }
  moefp4::ProjectArgs a;
  memset(&a, 0, sizeof a);
  a.T = (int)p->T;
  a.N = (int)p->N;
  a.K = (int)p->K;
  a.L = p->adapters;
  a.R = p->rank;
  a.g16 = p->gran_k == 16;
  a.out_f32 = p->out_fmt == MOEFP4_OUT_F32;
  a.x = static_cast<const uint16_t*>(x);
  a.w = w;
  a.w_sf = w_sf;
  a.w_gs = w_gs;
  a.a = static_cast<const uint16_t*>(lora_a);
  a.b = static_cast<const uint16_t*>(lora_b);
  a.id = id;
  a.scale = scale;
  a.out = out;
  a.x16 = at<uint16_t>(workspace, P.x16);
  a.xs = at<float>(workspace, P.xs);
  a.u = at<float>(workspace, P.u);
  a.ku = P.ku;
  a.part = at<float>(workspace, P.part);
  if (P.group) {
    a.ids = at<int32_t>(workspace, P.ids);
    a.route.counts = at<int32_t>(workspace, P.counts);
    a.route.offsets = at<int32_t>(workspace, P.offsets);
    a.route.sorted_assign = at<int32_t>(workspace, P.sorted);
    a.route.slot_of = at<int32_t>(workspace, P.slot_of);
    a.route.tiles = at<int32_t>(workspace, P.tiles);
    a.route.ntiles = at<int32_t>(workspace, P.ntiles);
    a.route.flags = at<int32_t>(workspace, P.flags);
    a.route.nchunks = P.chunks;
    a.route.chunk = P.chunk;
    a.route.hist = P.chunks ? at<int32_t>(workspace, P.hist) : nullptr;
    if (p->T > moefp4::kProjectFew) a.order = a.route.sorted_assign;
  }
  st = hip_status(moefp4::launch_project(a, stream), "project");
  return st == MOEFP4_OK ? ok() : st;
}

static moefp4_status grouped_check(const moefp4_grouped* p, bool weights) {
  if (!p) return fail(MOEFP4_EINVAL, "problem is NULL");
  if (p->M < 0 || p->E < 1 || p->N < 1 || p->K < 1)
    return fail(MOEFP4_EINVAL, "M must be >= 0, E, N and K positive; got M=%lld E=%d N=%lld K=%lld", (long long)p->M, p->E,
                (long long)p->N, (long long)p->K);
  if (p->N % 8 || p->K % 8)
    return fail(MOEFP4_EINVAL, "N and K must be multiples of 8, got N=%lld K=%lld", (long long)p->N, (long long)p->K);
  if (p->gran_k != 0 && p->gran_k != 16 && p->gran_k != 32)
    return fail(MOEFP4_EINVAL, "gran_k must be 0 (bfloat16 weights), 16 or 32, got %d", p->gran_k);
  if (!weights && p->gran_k != 0) return fail(MOEFP4_EINVAL, "weight gradients have gran_k 0, got %d", p->gran_k);
  if (p->gran_k != 0 && p->K % 32) return fail(MOEFP4_EINVAL, "FP4 weights need K a multiple of 32, got %lld", (long long)p->K);
  if (p->out_fmt != MOEFP4_OUT_BF16 && p->out_fmt != MOEFP4_OUT_F32) return fail(MOEFP4_EINVAL, "unknown out_fmt %d", p->out_fmt);
  const long long lim = 1LL << 40;
  if (p->E > moefp4::kMaxExperts || p->M > (1LL << 24) || p->N > (1LL << 20) || p->K > (1LL << 20) || p->M * p->N >= lim ||
      p->M * p->K >= lim || p->N * p->K >= lim / p->E)
    return fail(MOEFP4_EUNSUPPORTED, "E up to %d, M up to 2^24, N and K up to 2^20, M*N, M*K and E*N*K below 2^40", moefp4::kMaxExperts);
  return MOEFP4_OK;
}

struct Span { const void* p; size_t n; };

static bool overlaps(const void* out, size_t bytes, const Span* in, int n) {
  const char* o = static_cast<const char*>(out);
  for (int i = 0; i < n; ++i) {
    const char* q = static_cast<const char*>(in[i].p);
    if (q && o < q + in[i].n && q < o + bytes) return true;
  }
  return false;
}

static size_t grouped_floats(const moefp4_grouped* p, int form) {
  return (size_t)moefp4::grouped_part_floats(form, p->M, p->E, p->N, p->K);
}

moefp4_status moe_fp4_grouped_workspace_bytes(const moefp4_grouped* p, int32_t direction, size_t* bytes) {
  if (direction < MOEFP4_GROUPED || direction > MOEFP4_GROUPED_DW) return fail(MOEFP4_EINVAL, "unknown direction %d", direction);
  const moefp4_status st = grouped_check(p, direction != MOEFP4_GROUPED_DW);
  if (st != MOEFP4_OK) return st;
  if (!bytes) return fail(MOEFP4_EINVAL, "bytes is NULL");
  *bytes = align_up(4 * grouped_floats(p, direction));
  return ok();
}

// out and the workspace (what this call itself takes of it) against each other and the inputs.
static moefp4_status grouped_room(const moefp4_grouped* p, int form, const Span* in, int n, void* out, size_t outputs, void* workspace,
                                  size_t ws_bytes, moefp4::GroupedArgs* a) {
  const moefp4::GroupedPlan plan = moefp4::grouped_plan(form, p->M, p->E, p->N, p->K, p->gran_k);
  const size_t need = plan.parts > 1 ? 4 * outputs * plan.parts : 0;
  const Span to = {out, outputs * (p->out_fmt == MOEFP4_OUT_F32 ? 4 : 2)};
  if (need && (!workspace || ws_bytes < need))
    return fail(MOEFP4_EWORKSPACE, "workspace of %zu bytes needed, got %zu", need, workspace ? ws_bytes : (size_t)0);
  if (need && misaligned(workspace, 256)) return fail(MOEFP4_EINVAL, "workspace must be 256-byte aligned");
  if (overlaps(out, to.n, in, n)) return fail(MOEFP4_EINVAL, "out overlaps an input");
  if (need && (overlaps(workspace, need, in, n) || overlaps(workspace, need, &to, 1)))
    return fail(MOEFP4_EINVAL, "the workspace overlaps an input or out");
  a->part = need ? static_cast<float*>(workspace) : nullptr;
  return MOEFP4_OK;
}

// form 0: the product, 1: towards the rows
static moefp4_status grouped_product(const moefp4_grouped* p, int form, const void* x, const void* w, const uint8_t* w_sf,
                                     const float* w_gs, const int32_t* offsets, void* out, void* workspace, size_t ws_bytes,
                                     hipStream_t stream) {
  moefp4_status st = grouped_check(p, true);
  if (st != MOEFP4_OK) return st;
  if (p->M == 0) return ok();
  if (!x || !w || !offsets || !out) return fail(MOEFP4_EINVAL, "%s, w, offsets and out must be non-NULL", form ? "dy" : "x");
  if (p->gran_k ? !w_sf : (w_sf || w_gs)) return fail(MOEFP4_EINVAL, "w_sf goes with FP4 weights, and w_gs with them only");
  if (misaligned(x, 16) || misaligned(w, 16) || misaligned(w_sf, 16) || misaligned(out, 16) || misaligned(w_gs, 4) ||
      misaligned(offsets, 4))
    return fail(MOEFP4_EINVAL, "%s, w, w_sf and out must be 16-byte aligned, w_gs and offsets 4-byte", form ? "dy" : "x");
  const size_t M = p->M, N = p->N, K = p->K, E = p->E, g = p->gran_k;
  const Span in[] = {{x, 2 * M * (form ? N : K)}, {w, g ? E * N * (K / 2) : 2 * E * N * K}, {w_sf, g ? E * N * (K / g) : 0},
                     {w_gs, 4 * E}, {offsets, 4 * (E + 1)}};
  moefp4::GroupedArgs a;
  memset(&a, 0, sizeof a);
  st = grouped_room(p, form, in, 5, out, M * (form ? K : N), workspace, ws_bytes, &a);
  if (st != MOEFP4_OK) return st;
  a.M = (int)M;
  a.E = (int)E;
  a.N = (int)N;
  a.K = (int)K;
  a.gran = p->gran_k;
  a.out_f32 = p->out_fmt == MOEFP4_OUT_F32;
  a.p = static_cast<const uint16_t*>(x);
  if (g) a.w = static_cast<const uint8_t*>(w);
  else a.q = static_cast<const uint16_t*>(w);
  a.w_sf = w_sf;
  a.w_gs = w_gs;
  a.offsets = offsets;
  a.out = out;
  st = hip_status(moefp4::launch_grouped(a, form, stream), form ? "grouped_dx" : "grouped");
  return st == MOEFP4_OK ? ok() : st;
}

moefp4_status moe_fp4_grouped(const moefp4_grouped* p, const void* x, const void* w, const uint8_t* w_sf,
                              const float* w_gs, const int32_t* offsets, void* out, void* workspace, size_t ws_bytes,
                              hipStream_t stream) {
  return grouped_product(p, 0, x, w, w_sf, w_gs, offsets, out, workspace, ws_bytes, stream);
}

moefp4_status moe_fp4_grouped_dx(const moefp4_grouped* p, const void* dy, const void* w, const uint8_t* w_sf,
                                 const float* w_gs, const int32_t* offsets, void* out, void* workspace, size_t ws_bytes,
                                 hipStream_t stream) {
  return grouped_product(p, 1, dy, w, w_sf, w_gs, offsets, out, workspace, ws_bytes, stream);
}

moefp4_status moe_fp4_grouped_dw(const moefp4_grouped* p, const void* dy, const void* x, const int32_t* offsets,
                                 void* out, int32_t accumulate, void* workspace, size_t ws_bytes, hipStream_t stream) {
  moefp4_status st = grouped_check(p, false);
  if (st != MOEFP4_OK) return st;
  if (!offsets || !out || (p->M > 0 && (!dy || !x))) return fail(MOEFP4_EINVAL, "dy, x, offsets and out must be non-NULL");
  if (misaligned(dy, 16) || misaligned(x, 16) || misaligned(out, 16) || misaligned(offsets, 4))
    return fail(MOEFP4_EINVAL, "dy, x and out must be 16-byte aligned, offsets 4-byte");
  const size_t M = p->M, N = p->N, K = p->K, E = p->E;
  const Span in[] = {{dy, 2 * M * N}, {x, 2 * M * K}, {offsets, 4 * (E + 1)}};
  moefp4::GroupedArgs a;
  memset(&a, 0, sizeof a);
  st = grouped_room(p, 2, in, 3, out, E * N * K, workspace, ws_bytes, &a);
  if (st != MOEFP4_OK) return st;
  a.M = (int)M;
  a.E = (int)E;
  a.N = (int)N;
  a.K = (int)K;
  a.out_f32 = p->out_fmt == MOEFP4_OUT_F32;
  a.accumulate = accumulate != 0;
  a.p = static_cast<const uint16_t*>(dy);
  a.q = static_cast<const uint16_t*>(x);
  a.offsets = offsets;
  a.out = out;
  st = hip_status(moefp4::launch_grouped(a, 2, stream), "grouped_dw");
  return st == MOEFP4_OK ? ok() : st;
}

static moefp4_status norm_check(const moefp4_norm* p) {
  if (!p) return fail(MOEFP4_EINVAL, "problem is NULL");
  if (p->T < 0 || p->H < 8 || p->H % 8)
    return fail(MOEFP4_EINVAL, "T must be >= 0 and H a positive multiple of 8, got T=%lld H=%lld", (long long)p->T, (long long)p->H);
  for (int32_t f : {p->h_fmt, p->post_fmt, p->pre_fmt, p->gate_fmt})
    if (f != MOEFP4_OUT_BF16 && f != MOEFP4_OUT_F32) return fail(MOEFP4_EINVAL, "unknown format %d", f);
  if (p->gate_kind < MOEFP4_GATE_NONE || p->gate_kind > MOEFP4_GATE_ELEMENT)
    return fail(MOEFP4_EINVAL, "unknown gate_kind %d", p->gate_kind);
  if (p->gate_sigmoid != 0 && p->gate_sigmoid != 1) return fail(MOEFP4_EINVAL, "gate_sigmoid must be 0 or 1, got %d", p->gate_sigmoid);
  if (!isfinite(p->scale) || !isfinite(p->h_scale)) return fail(MOEFP4_EINVAL, "scale and h_scale must be finite");
  // (squares below FP32's smallest number are nothing beside it, and it is nothing beside a mean beyond the largest one)
  if (!(p->eps >= 1e-20f && p->eps <= 1.0f)) return fail(MOEFP4_EINVAL, "eps must be in [1e-20, 1], got %g", (double)p->eps);
  if (p->H > moefp4::kNormMostH || p->T > (1LL << 24) || p->T * p->H >= (1LL << 40))
    return fail(MOEFP4_EUNSUPPORTED, "H up to %d, T up to 2^24, T*H below 2^40", moefp4::kNormMostH);
  return MOEFP4_OK;
}

static size_t gate_elements(const moefp4_norm* p) {
  return p->gate_kind == MOEFP4_GATE_CHANNEL ? p->H : p->gate_kind == MOEFP4_GATE_TOKEN ? p->T :
         p->gate_kind == MOEFP4_GATE_ELEMENT ? (size_t)p->T * p->H : 0;
}

// What both directions take: y, the gate and the weights go together as the problem says.
static moefp4_status norm_operands(const moefp4_norm* p, const void* y, const void* post_w, const void* gate, const void* pre_w) {
  if (!y && (post_w || gate || p->gate_kind != MOEFP4_GATE_NONE)) return fail(MOEFP4_EINVAL, "post_w and a gate need y");
  if ((gate != nullptr) != (p->gate_kind != MOEFP4_GATE_NONE)) return fail(MOEFP4_EINVAL, "the gate goes with a gate_kind");
  if (!y && !pre_w) return fail(MOEFP4_EINVAL, "y or pre_w must be non-NULL");
  if (misaligned(y, 16) || misaligned(post_w, 16) || misaligned(pre_w, 16) ||
      misaligned(gate, p->gate_kind == MOEFP4_GATE_TOKEN ? 4 : 16))
    return fail(MOEFP4_EINVAL, "y, the weights and the gate must be 16-byte aligned (a gate per token 4-byte)");
  return MOEFP4_OK;
}

static moefp4::NormArgs norm_args(const moefp4_norm* p) {
  moefp4::NormArgs a;
  memset(&a, 0, sizeof a);
  a.T = p->T;
  a.H = (int)p->H;
  a.h_f32 = p->h_fmt == MOEFP4_OUT_F32;
  a.post_f32 = p->post_fmt == MOEFP4_OUT_F32;
  a.pre_f32 = p->pre_fmt == MOEFP4_OUT_F32;
  a.gate_f32 = p->gate_fmt == MOEFP4_OUT_F32;
  a.gate_kind = p->gate_kind;
  a.gate_act = p->gate_sigmoid;
  a.scale = p->scale;
  a.h_scale = p->h_scale;
  a.eps = p->eps;
  return a;
}

moefp4_status moe_fp4_block_norm(const moefp4_norm* p, const void* h, const void* y, const void* post_w,
                                 const void* gate, const void* pre_w, void* h_out, void* n, hipStream_t stream) {
  moefp4_status st = norm_check(p);
  if (st != MOEFP4_OK) return st;
  if (p->T == 0) return ok();
  st = norm_operands(p, y, post_w, gate, pre_w);
  if (st != MOEFP4_OK) return st;
  if (!h || (y != nullptr) != (h_out != nullptr) || (pre_w != nullptr) != (n != nullptr))
    return fail(MOEFP4_EINVAL, "h must be non-NULL, h_out go with y and n with pre_w");
  if (misaligned(h, 16) || misaligned(h_out, 16) || misaligned(n, 16))
    return fail(MOEFP4_EINVAL, "h, h_out and n must be 16-byte aligned");
  const size_t TH = (size_t)p->T * p->H, hb = p->h_fmt == MOEFP4_OUT_F32 ? 4 : 2;
  const size_t wb[2] = {(size_t)p->H * (p->post_fmt == MOEFP4_OUT_F32 ? 4 : 2), (size_t)p->H * (p->pre_fmt == MOEFP4_OUT_F32 ? 4 : 2)};
  const Span in[] = {{y, 2 * TH}, {post_w, wb[0]}, {gate, gate_elements(p) * (p->gate_fmt == MOEFP4_OUT_F32 ? 4 : 2)},
                     {pre_w, wb[1]}, {h, h == h_out ? 0 : hb * TH}};
  const Span out_h = {h_out, hb * TH}, in_h = {h, hb * TH};
  if ((h_out && overlaps(h_out, hb * TH, in, 5)) || (n && (overlaps(n, 2 * TH, in, 4) || overlaps(n, 2 * TH, &in_h, 1) ||
                                                           overlaps(n, 2 * TH, &out_h, 1))))
    return fail(MOEFP4_EINVAL, "an output overlaps an input or the other output (h_out may be h itself)");
  moefp4::NormArgs a = norm_args(p);
  a.h = h;
  a.y = y;
  a.post_w = post_w;
  a.gate = gate;
  a.pre_w = pre_w;
  a.h_out = h_out;
  a.n = n;
  st = hip_status(moefp4::launch_block_norm(a, stream), "block_norm");
  return st == MOEFP4_OK ? ok() : st;
}

static size_t norm_grad_bytes(const moefp4_norm* p) {
  // (rows of a smaller T take no more parts)
  const size_t n = (size_t)moefp4::norm_grad_parts(p->T, (int)p->H) * p->H * 3 * 4;
  return n > 256 ? align_up(n) : 256;
}

moefp4_status moe_fp4_block_norm_grad_workspace_bytes(const moefp4_norm* p, size_t* bytes) {
  const moefp4_status st = norm_check(p);
  if (st != MOEFP4_OK) return st;
  if (!bytes) return fail(MOEFP4_EINVAL, "bytes is NULL");
  *bytes = norm_grad_bytes(p);
  return ok();
}

moefp4_status moe_fp4_block_norm_grad(const moefp4_norm* p, const void* dh, const void* dn, const void* h, const void* y,
                                      const void* post_w, const void* gate, const void* pre_w, void* d_h, void* d_y,
                                      float* d_post_w, void* d_gate, float* d_pre_w, void* workspace, size_t ws_bytes,
                                      hipStream_t stream) {
  moefp4_status st = norm_check(p);
  if (st != MOEFP4_OK) return st;
  const bool rows = p->T > 0;  // (tensors without elements may have no address)
  if (rows) {
    st = norm_operands(p, y, post_w, gate, pre_w);
    if (st != MOEFP4_OK) return st;
    if (!d_h || (y != nullptr) != (d_y != nullptr) || (gate != nullptr) != (d_gate != nullptr))
      return fail(MOEFP4_EINVAL, "d_h must be non-NULL, d_y go with y and d_gate with the gate");
    if ((pre_w != nullptr) != (dn != nullptr) || (pre_w != nullptr) != (h != nullptr))
      return fail(MOEFP4_EINVAL, "dn and h go with pre_w");
    if (!pre_w && !dh) return fail(MOEFP4_EINVAL, "dh or pre_w (and dn) must be non-NULL");
  }
  if ((post_w != nullptr) != (d_post_w != nullptr) || (pre_w != nullptr) != (d_pre_w != nullptr))
    return fail(MOEFP4_EINVAL, "d_post_w goes with post_w and d_pre_w with pre_w");
  if (p->gate_kind == MOEFP4_GATE_CHANNEL && !d_gate) return fail(MOEFP4_EINVAL, "d_gate must be non-NULL with a gate");
  if (misaligned(dh, 16) || misaligned(dn, 16) || misaligned(h, 16) || misaligned(d_h, 16) || misaligned(d_y, 16) ||
      misaligned(d_post_w, 16) || misaligned(d_pre_w, 16) || misaligned(d_gate, p->gate_kind == MOEFP4_GATE_TOKEN ? 4 : 16))
    return fail(MOEFP4_EINVAL, "dh, dn, h, d_h, d_y, d_post_w, d_pre_w and d_gate must be 16-byte aligned (a gate per token 4-byte)");
  const size_t need = norm_grad_bytes(p);
  if (!workspace || ws_bytes < need)
    return fail(MOEFP4_EWORKSPACE, "workspace of %zu bytes needed, got %zu", need, workspace ? ws_bytes : (size_t)0);
  if (misaligned(workspace, 256)) return fail(MOEFP4_EINVAL, "workspace must be 256-byte aligned");
  const size_t T = p->T, H = p->H, TH = T * H, hb = p->h_fmt == MOEFP4_OUT_F32 ? 4 : 2, gb = p->gate_fmt == MOEFP4_OUT_F32 ? 4 : 2;
  const size_t ge = gate_elements(p);
  const Span in[] = {{dn, 2 * TH}, {h, hb * TH}, {y, 2 * TH}, {post_w, H * (p->post_fmt == MOEFP4_OUT_F32 ? 4 : 2)}, {gate, ge * gb},
                     {pre_w, H * (p->pre_fmt == MOEFP4_OUT_F32 ? 4 : 2)}, {dh, hb * TH}};
  const Span out[] = {{d_h, hb * TH}, {d_y, 2 * TH}, {d_post_w, 4 * H}, {d_gate, ge * (p->gate_kind == MOEFP4_GATE_ELEMENT ? gb : 4)},
                      {d_pre_w, 4 * H}, {workspace, need}};
  for (int i = 0; i < 6; ++i) {
    if (!out[i].p) continue;
    // (d_h may be dh, the last input)
    if (overlaps(out[i].p, out[i].n, in, i == 0 && d_h == dh ? 6 : 7) || overlaps(out[i].p, out[i].n, out + i + 1, 5 - i))
      return fail(MOEFP4_EINVAL, "an output or the workspace overlaps an input or another output (d_h may be dh itself)");
  }
  moefp4::NormArgs a = norm_args(p);
  a.h = h;
  a.y = y;
  a.post_w = post_w;
  a.gate = gate;
  a.pre_w = pre_w;
  a.dh = dh;
  a.dn = dn;
  a.d_h = d_h;
  a.d_y = d_y;
  a.d_gate = d_gate;
  a.d_post_w = d_post_w;
  a.d_pre_w = d_pre_w;
  a.part = static_cast<float*>(workspace);
  st = hip_status(moefp4::launch_block_norm_grad(a, stream), "block_norm_grad");
  return st == MOEFP4_OK ? ok() : st;
}

moefp4_status moe_fp4_forward_static(const moefp4_problem* p, const void* x, const uint8_t* x_sf,
                                     const int32_t* topk_ids, const float* topk_w, const uint8_t* w13,
                                     const uint8_t* w13_sf, const float* w13_gs, const uint8_t* w2,
                                     const uint8_t* w2_sf, const float* w2_gs, void* out, hipStream_t stream) {
  Layout L;
  moefp4_status st = plan(p, &L);
  if (st != MOEFP4_OK) return st;
  if (L.total > kStaticScratchBytes)
    return fail(MOEFP4_EWORKSPACE,
                "this problem needs %zu bytes of scratch; the static scratch of moe_fp4_forward_static holds %zu "
                "(use moe_fp4_forward with a caller workspace)",
                L.total, kStaticScratchBytes);
  void* ws = nullptr;
  if ((st = static_scratch(&ws)) != MOEFP4_OK) return st;
  return moe_fp4_forward(p, x, x_sf, topk_ids, topk_w, w13, w13_sf, w13_gs, w2, w2_sf, w2_gs, out, ws,
                         kStaticScratchBytes, stream);
}

moefp4_status fp4_requant_gran_k(int64_t E, int64_t N, int64_t K, const uint8_t* src,
                                 const uint8_t* src_sf, int32_t src_gran, const float* src_gs,
                                 uint8_t* dst, uint8_t* dst_sf, int32_t dst_gran,
                                 hipStream_t stream) {
  if (E < 0 || N < 0 || K < 0) return fail(MOEFP4_EINVAL, "E, N, K must be >= 0");
  if ((src_gran != 16 && src_gran != 32) || (dst_gran != 16 && dst_gran != 32))
    return fail(MOEFP4_EINVAL, "granularities must be 16 or 32, got %d -> %d", src_gran, dst_gran);
  if (src_gran != 16 || dst_gran != 32)
    return fail(MOEFP4_EUNSUPPORTED, "only group16 -> group32 requantisation is computed, got %d -> %d",
                src_gran, dst_gran);
  if (K % 32) return fail(MOEFP4_EINVAL, "K must be a multiple of 32, got %lld", (long long)K);
  if (N * (K / 32) > (int64_t)1 << 30 || E > 65535)
    return fail(MOEFP4_EUNSUPPORTED, "N*K/32 must be <= 2^30 and E <= 65535");
  const int64_t n = E * N * K;
  if (n == 0) return ok();
  if (!src || !src_sf || !dst || !dst_sf)
    return fail(MOEFP4_EINVAL, "src, src_sf, dst and dst_sf must be non-NULL");
  if (misaligned(src, 16) || misaligned(dst, 16) || misaligned(src_sf, 8) || misaligned(dst_sf, 4))
    return fail(MOEFP4_EINVAL, "src/dst must be 16-byte aligned, src_sf 8-byte, dst_sf 4-byte");
  // overlap rules: dst == src allowed; everything else disjoint
  struct R { uintptr_t b, e; } r[4] = {
      {(uintptr_t)src, (uintptr_t)src + (uintptr_t)(n / 2)},
      {(uintptr_t)src_sf, (uintptr_t)src_sf + (uintptr_t)(n / 16)},
      {(uintptr_t)dst, (uintptr_t)dst + (uintptr_t)(n / 2)},
      {(uintptr_t)dst_sf, (uintptr_t)dst_sf + (uintptr_t)(n / 32)}};
  for (int i = 0; i < 4; ++i)
    for (int j = i + 1; j < 4; ++j) {
      if (i == 0 && j == 2 && src == dst) continue;
      if (r[i].b < r[j].e && r[j].b < r[i].e)
        return fail(MOEFP4_EINVAL, "buffers overlap (only dst == src is allowed)");
    }
  moefp4_status st = hip_status(
      moefp4::launch_requant_g16_g32(src, src_sf, src_gs, dst, dst_sf, E, N, K, stream), "requant");
  return st == MOEFP4_OK ? ok() : st;
}

moefp4_status moe_fp4_prepare_gemm_weights(int64_t E, int64_t N, int64_t K, int32_t which,
                                           int32_t w13_order, const uint8_t* src, const uint8_t* src_sf,
                                           uint8_t* dst, uint8_t* dst_sf, hipStream_t stream) {
  if (E < 0 || N < 0 || K < 0) return fail(MOEFP4_EINVAL, "E, N, K must be >= 0");
  if (which != 0 && which != 1) return fail(MOEFP4_EINVAL, "which must be 0 (w13) or 1 (w2), got %d", which);
  if (w13_order != MOEFP4_GATE_UP && w13_order != MOEFP4_UP_GATE)
    return fail(MOEFP4_EINVAL, "unknown w13_order %d", w13_order);
  if (N % 512 || K % 512)
    return fail(MOEFP4_EINVAL, "N and K must be multiples of 512, got N=%lld K=%lld", (long long)N,
                (long long)K);
  if (N * K / 32 >= ((int64_t)1 << 31) || E > 65535)
    return fail(MOEFP4_EUNSUPPORTED, "N*K/32 must be below 2^31 and E <= 65535");
  const int64_t n = E * N * K;
  if (n == 0) return ok();
  if (!src || !src_sf || !dst || !dst_sf)
    return fail(MOEFP4_EINVAL, "src, src_sf, dst and dst_sf must be non-NULL");
  if (misaligned(src, 16) || misaligned(dst, 16) || misaligned(src_sf, 16) || misaligned(dst_sf, 16))
    return fail(MOEFP4_EINVAL, "src, src_sf, dst and dst_sf must be 16-byte aligned");
  struct R { uintptr_t b, e; } r[4] = {
      {(uintptr_t)src, (uintptr_t)src + (uintptr_t)(n / 2)},
      {(uintptr_t)src_sf, (uintptr_t)src_sf + (uintptr_t)(n / 32)},
      {(uintptr_t)dst, (uintptr_t)dst + (uintptr_t)(n / 2)},
      {(uintptr_t)dst_sf, (uintptr_t)dst_sf + (uintptr_t)(n / 32)}};
  for (int i = 0; i < 4; ++i)
    for (int j = i + 1; j < 4; ++j)
      if (r[i].b < r[j].e && r[j].b < r[i].e) return fail(MOEFP4_EINVAL, "buffers overlap");
  moefp4_status st = hip_status(
      moefp4::launch_prepare_gemm(src, src_sf, dst, dst_sf, E, N, K, which == 0, w13_order, stream),
      "prepare_gemm_weights");
  return st == MOEFP4_OK ? ok() : st;
}

moefp4_status moe_fp4_prepare_gemm_weights_g16(int64_t E, int64_t N, int64_t K, int32_t which,
                                               int32_t w13_order, const uint8_t* src, const uint8_t* src_sf,
                                               const float* src_gs, uint8_t* dst, uint8_t* dst_sf,
                                               hipStream_t stream) {
  if (E < 0 || N < 0 || K < 0) return fail(MOEFP4_EINVAL, "E, N, K must be >= 0");
  if (which != 0 && which != 1) return fail(MOEFP4_EINVAL, "which must be 0 (w13) or 1 (w2), got %d", which);
  if (w13_order != MOEFP4_GATE_UP && w13_order != MOEFP4_UP_GATE)
    return fail(MOEFP4_EINVAL, "unknown w13_order %d", w13_order);
  if (N % 512 || K % 512)
    return fail(MOEFP4_EINVAL, "N and K must be multiples of 512, got N=%lld K=%lld", (long long)N,
                (long long)K);
  if (N * K / 32 >= ((int64_t)1 << 31) || E > 65535)
    return fail(MOEFP4_EUNSUPPORTED, "N*K/32 must be below 2^31 and E <= 65535");
  const int64_t n = E * N * K;
  if (n == 0) return ok();
  if (!src || !src_sf || !dst || !dst_sf)
    return fail(MOEFP4_EINVAL, "src, src_sf, dst and dst_sf must be non-NULL");
  if (misaligned(src, 16) || misaligned(dst, 16) || misaligned(src_sf, 16) || misaligned(dst_sf, 16))
    return fail(MOEFP4_EINVAL, "src, src_sf, dst and dst_sf must be 16-byte aligned");
  struct R { uintptr_t b, e; } r[4] = {
      {(uintptr_t)src, (uintptr_t)src + (uintptr_t)(n / 2)},
      {(uintptr_t)src_sf, (uintptr_t)src_sf + (uintptr_t)(n / 16)},
      {(uintptr_t)dst, (uintptr_t)dst + (uintptr_t)(n / 2)},
      {(uintptr_t)dst_sf, (uintptr_t)dst_sf + (uintptr_t)(n / 32)}};
  for (int i = 0; i < 4; ++i)
    for (int j = i + 1; j < 4; ++j)
      if (r[i].b < r[j].e && r[j].b < r[i].e) return fail(MOEFP4_EINVAL, "buffers overlap");
  moefp4_status st = hip_status(moefp4::launch_requant_prepare_gemm(src, src_sf, src_gs, dst, dst_sf, E, N, K,
                                                                    which == 0, w13_order, stream),
                                "prepare_gemm_weights_g16");
  return st == MOEFP4_OK ? ok() : st;
}

moefp4_status moe_fp4_quantize_act(int64_t T, int64_t H, const void* x, uint8_t* x_fp8,
                                   uint8_t* x_sf, hipStream_t stream) {
  if (T < 0 || H <= 0 || H % 32) return fail(MOEFP4_EINVAL, "need T >= 0 and H a positive multiple of 32, got T=%lld H=%lld", (long long)T, (long long)H);
  if (H > (1 << 30) || T > (1ll << 40) / H) return fail(MOEFP4_EUNSUPPORTED, "T*H too large");
  if (T == 0) return ok();
  if (!x || !x_fp8 || !x_sf) return fail(MOEFP4_EINVAL, "x, x_fp8 and x_sf must be non-NULL");
  if (misaligned(x, 16) || misaligned(x_fp8, 16))
    return fail(MOEFP4_EINVAL, "x and x_fp8 must be 16-byte aligned");
  moefp4_status st = hip_status(moefp4::launch_quantize_act(static_cast<const uint16_t*>(x), T, (int)H,
                                                            x_fp8, x_sf, false, stream),
                                "quantize_act");
  return st == MOEFP4_OK ? ok() : st;
}

moefp4_status moe_fp4_quantize_act_fp4(int64_t T, int64_t H, const void* x, uint8_t* x_fp4,
                                       uint8_t* x_sf, hipStream_t stream) {
  if (T < 0 || H <= 0 || H % 32) return fail(MOEFP4_EINVAL, "need T >= 0 and H a positive multiple of 32, got T=%lld H=%lld", (long long)T, (long long)H);
  if (H > (1 << 30) || T > (1ll << 40) / H) return fail(MOEFP4_EUNSUPPORTED, "T*H too large");
  if (T == 0) return ok();
  if (!x || !x_fp4 || !x_sf) return fail(MOEFP4_EINVAL, "x, x_fp4 and x_sf must be non-NULL");
  if (misaligned(x, 16) || misaligned(x_fp4, 16))
    return fail(MOEFP4_EINVAL, "x and x_fp4 must be 16-byte aligned");
  moefp4_status st = hip_status(moefp4::launch_quantize_act(static_cast<const uint16_t*>(x), T, (int)H,
                                                            x_fp4, x_sf, true, stream),
                                "quantize_act_fp4");
  return st == MOEFP4_OK ? ok() : st;
}

moefp4_status moefp4_mfma_peak_probe(int32_t a4, int32_t iters, int32_t blocks, float* sink, double* flops,
                                     hipStream_t stream) {
  if (iters < 1 || blocks < 1 || !flops) return fail(MOEFP4_EINVAL, "iters, blocks >= 1 and flops non-NULL needed");
  if (!sink) return fail(MOEFP4_EINVAL, "sink must be non-NULL (blocks * 256 floats)");
  *flops = (double)blocks * 4 * (double)iters * 64 * 2.0 * 16 * 16 * 128;
  moefp4_status st = hip_status(moefp4::launch_mfma_peak(a4 != 0, iters, blocks, sink, stream), "mfma_peak");
  return st == MOEFP4_OK ? ok() : st;
}

moefp4_status moefp4_set_stage_events(hipEvent_t* events, int32_t n) {
  if (events && n < 6) return fail(MOEFP4_EINVAL, "stage events need an array of 6, got %d", n);
  g_stage_events = events;
  return ok();
}

moefp4_status moefp4_set_wait_looks(int32_t looks) {
  g_wait_looks = looks < 0 ? moefp4::kFewLooks : looks;
  return ok();
}

const char* moefp4_last_error(void) { return g_err.c_str(); }

const char* moefp4_version(void) { return "moefp4 0.1 gfx950"; }

}  // extern "C"
