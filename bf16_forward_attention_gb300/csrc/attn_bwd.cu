// attn_bwd.cu - host side of the backward pass declared in include/attn_fwd.h:
// checks the call, lays out the workspace and launches, on the caller's stream, dQ
// with the row statistics, then dK with dV (attn_bwd_kernel.cuh), then the join of the results
// that several CTAs share the streamed axis of, where there are any; the second and
// the third each a programmatic dependent of the one before.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "attn_bwd_kernel.cuh"
#include "attn_fwd.h"
#include "host_common.h"

namespace attn_host {

bool bwd_take_status(unsigned int* s) { return take_status(attn::g_attn_status, s); }

}  // namespace attn_host

namespace {

using namespace attn_host;
namespace bwd = attn::bwd;

std::mutex g_mutex;
int g_state[kMaxDevices];  // 0 = not set up, 1 = ready, negative = status to return

// The kernels by variant_of.
using DkvKernel = void (*)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const CUtensorMap,
                           const bwd::BwdParams);
using DqKernel = void (*)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const CUtensorMap,
                          const CUtensorMap, const bwd::BwdParams);
constexpr DkvKernel kDkv[8] = {
    bwd::attn_bwd_dkv<false, false, false>, bwd::attn_bwd_dkv<true, false, false>,
    bwd::attn_bwd_dkv<false, true, false>,  bwd::attn_bwd_dkv<true, true, false>,
    bwd::attn_bwd_dkv<false, false, true>,  bwd::attn_bwd_dkv<true, false, true>,
    bwd::attn_bwd_dkv<false, true, true>,   bwd::attn_bwd_dkv<true, true, true>};
constexpr DqKernel kDq[8] = {
    bwd::attn_bwd_dq<false, false, false>, bwd::attn_bwd_dq<true, false, false>,
    bwd::attn_bwd_dq<false, true, false>,  bwd::attn_bwd_dq<true, true, false>,
    bwd::attn_bwd_dq<false, false, true>,  bwd::attn_bwd_dq<true, false, true>,
    bwd::attn_bwd_dq<false, true, true>,   bwd::attn_bwd_dq<true, true, true>};
int variant_of(bool causal, bool varlen, bool is_long) { return causal + 2 * varlen + 4 * is_long; }

template <typename F>
bool raise_smem(F* fn, int bytes) {
  return cudaFuncSetAttribute(reinterpret_cast<const void*>(fn),
                              cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
}

// Once per device: check the architecture and raise the shared-memory limits.
int device_ready(int dev) {
  if (dev < 0 || dev >= kMaxDevices) return ATTN_ERR_NO_DEVICE;
  std::lock_guard<std::mutex> lock(g_mutex);
  if (g_state[dev] != 0) return g_state[dev] > 0 ? ATTN_OK : g_state[dev];
  int major = 0, minor = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) {
    cudaGetLastError();
    return ATTN_ERR_NO_DEVICE;
  }
  if (major != 10 || minor != 3) return g_state[dev] = ATTN_ERR_ARCH;
  for (int i = 0; i < 8; ++i)
    if (!raise_smem(kDkv[i], bwd::kDkvSmem) || !raise_smem(kDq[i], bwd::kDqSmem)) {
      cudaGetLastError();
      return ATTN_ERR_LAUNCH;
    }
  g_state[dev] = 1;
  return ATTN_OK;
}

constexpr int kJoinPer = bwd::kTile / bwd::kJoinRows;  // join blocks per tile

int64_t tiles_of(int64_t n) { return (n + bwd::kTile - 1) / bwd::kTile; }

// How many CTAs share one owned tile's streamed tiles: the count with the least
// estimated time, in units of one streamed tile (about 1 us). A wave costs its
// tiles, 2 units of start and end, and for a shared result `part` units to write
// and read back its fp32 terms; the join kernel's launch costs 3.
int choose_splits(int64_t items, int64_t tiles, int64_t sms, int part) {
  int best = 1;
  double least = 1e30;
  for (int s = 1; s <= 32 && s <= tiles; ++s) {
    const int64_t waves = (items * s + sms - 1) / sms;
    const double cost =
        static_cast<double>(waves) * ((tiles + s - 1) / s + 2 + (s > 1 ? part : 0)) + (s > 1 ? 3 : 0);
    if (cost < least) {
      least = cost;
      best = s;
    }
  }
  return best;
}

// What an item's number means (BH, n_tiles and n_splits are set).
void place(bwd::BwdParams* p, int heads, int64_t owners) {
  p->n_groups = (p->BH + heads - 1) / heads;
  p->heads = bwd::Div::by(heads);
  p->last = bwd::Div::by(p->BH - int64_t(p->n_groups - 1) * heads);
  p->span = bwd::Div::by(int64_t(p->n_tiles) * heads);
  p->splits = bwd::Div::by(p->n_splits);
  p->owners = bwd::Div::by(owners);
}

struct Plan {
  int64_t q_tiles, k_tiles;  // per sequence (grid)
  int64_t q_slots, k_slots;  // tile slots per head
  int64_t q_all, k_all;      // slots of all heads
  int dq_splits, dkv_splits;
  bool dq_long, dkv_long;    // an item may have more tiles than one accumulator takes
  int64_t stats_bytes, dq_bytes, dkv_bytes;
  int64_t bytes() const { return stats_bytes + dq_bytes + dkv_bytes; }
};

constexpr int64_t kLim31 = (int64_t(1) << 31) - 1;

// Sizes are checked (each at least 1 and below 2^31). False: beyond the launch limits.
bool make_plan(Plan* pl, bool varlen, int64_t B, int64_t Hq, int64_t Hkv, int64_t Sq, int64_t Sk,
               int64_t max_sq, int64_t max_sk) {
  pl->q_tiles = tiles_of(max_sq);
  pl->k_tiles = tiles_of(max_sk);
  pl->q_slots = varlen ? Sq / bwd::kTile + B + 1 : pl->q_tiles;
  pl->k_slots = varlen ? Sk / bwd::kTile + B + 1 : pl->k_tiles;
  const int64_t rep = varlen ? 1 : B;
  // Grids and slot numbers are ints; 32 is the most splits.
  if (B > kLim31 / Hq / pl->q_tiles / 32 || B > kLim31 / Hkv / pl->k_tiles / 32) return false;
  if (rep > kLim31 / Hq / pl->q_slots || rep > kLim31 / Hkv / pl->k_slots) return false;
  if (Hq / Hkv > kLim31 / pl->q_tiles) return false;
  pl->q_all = rep * Hq * pl->q_slots;
  pl->k_all = rep * Hkv * pl->k_slots;
  // A packed batch's sequences are taken at their average length.
  const int64_t sms = sms_here();
  const int64_t nq = varlen ? tiles_of((Sq + B - 1) / B) : pl->q_tiles;
  const int64_t nk = varlen ? tiles_of((Sk + B - 1) / B) : pl->k_tiles;
  pl->dq_splits = choose_splits(B * Hq * nq, nk, sms, 3);
  pl->dkv_splits = choose_splits(B * Hkv * nk, nq * (Hq / Hkv), sms, 5);
  const int64_t tile_bytes = int64_t(bwd::kTile) * attn::kD * 4;
  pl->stats_bytes = pl->q_all * bwd::kStatFloats * 4;
  // fp32 terms of results that several items share, and of items that take several accumulators.
  auto longer = [](int64_t n, int splits) { return (n + splits - 1) / splits > bwd::kAccTiles; };
  pl->dq_long = longer(pl->k_tiles, pl->dq_splits);
  pl->dkv_long = longer(pl->q_tiles * (Hq / Hkv), pl->dkv_splits);
  pl->dq_bytes = pl->dq_splits > 1 || pl->dq_long ? pl->dq_splits * pl->q_all * tile_bytes : 0;
  pl->dkv_bytes = pl->dkv_splits > 1 || pl->dkv_long ? 2 * pl->dkv_splits * pl->k_all * tile_bytes : 0;
  return true;
}

struct Span {
  const void* p;
  uint64_t n;
};

int bwd_impl(const void* dout, const void* q, const void* k, const void* v, const void* out,
             const float* lse, void* dq, void* dk, void* dv, const int32_t* cu_q, const int32_t* cu_k,
             int layout, int64_t B, int64_t Hq, int64_t Hkv, int64_t Sq, int64_t Sk, int64_t max_sq,
             int64_t max_sk, int64_t d, float scale, int rounding_mode, int flags, void* workspace,
             int64_t workspace_bytes, void* stream, unsigned long long timeout_ns = kTimeoutNs,
             int withhold = -1) {
  const bool varlen = cu_q != nullptr;
  // ---- host-side validation (nothing is launched on failure)
  if (!dout || !q || !k || !v || !out || !lse || !dq || !dk || !dv || !workspace)
    return ATTN_ERR_INVALID_ARG;
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Sq < 1 || Sk < 1) return ATTN_ERR_INVALID_ARG;
  if (max_sq < 1 || max_sk < 1 || max_sq > Sq || max_sk > Sk) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  if (flags & ~ATTN_FLAG_CAUSAL) return ATTN_ERR_UNSUPPORTED;
  if (d != attn::kD) return ATTN_ERR_UNSUPPORTED;
  if (layout != ATTN_LAYOUT_BHSD && layout != ATTN_LAYOUT_BSHD) return ATTN_ERR_UNSUPPORTED;
  if (rounding_mode < ATTN_ROUND_RTNE || rounding_mode > ATTN_ROUND_RTZ) return ATTN_ERR_UNSUPPORTED;
  if (Sq > kLim31 || Sk > kLim31 || Hq > kLim31 || B > kLim31) return ATTN_ERR_TOO_LARGE;
  const int64_t kStrideLim = int64_t(1) << 40;  // TMA strides
  if (Hq > kStrideLim / 256 / Sq || Hkv > kStrideLim / 256 / Sk) return ATTN_ERR_TOO_LARGE;
  const int64_t rep = varlen ? 1 : B;
  if (rep > (int64_t(1) << 54) / Hq / (Sq > Sk ? Sq : Sk)) return ATTN_ERR_TOO_LARGE;
  Plan pl;
  if (!make_plan(&pl, varlen, B, Hq, Hkv, Sq, Sk, max_sq, max_sk)) return ATTN_ERR_TOO_LARGE;
  if (workspace_bytes < pl.bytes()) return ATTN_ERR_INVALID_ARG;
  const void* aligned[] = {dout, q, k, v, out, dq, dk, dv, workspace};
  for (const void* p : aligned)
    if (reinterpret_cast<uintptr_t>(p) & 15u) return ATTN_ERR_MISALIGNED;
  if ((reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(cu_q) |
       reinterpret_cast<uintptr_t>(cu_k)) & 3u)
    return ATTN_ERR_MISALIGNED;
  const uint64_t nq = uint64_t(rep) * Hq * Sq * 256, nk = uint64_t(rep) * Hkv * Sk * 256;
  const uint64_t ncu = varlen ? uint64_t(B + 1) * 4 : 0;
  const Span in[] = {{dout, nq}, {q, nq}, {k, nk}, {v, nk}, {out, nq}, {lse, nq / 64}, {cu_q, ncu}, {cu_k, ncu}};
  const Span written[] = {{dq, nq}, {dk, nk}, {dv, nk}, {workspace, uint64_t(pl.bytes())}};
  for (int i = 0; i < 4; ++i) {
    for (const Span& s : in)
      if (s.n && overlaps(written[i].p, written[i].n, s.p, s.n)) return ATTN_ERR_ALIASING;
    for (int j = 0; j < i; ++j)
      if (overlaps(written[i].p, written[i].n, written[j].p, written[j].n)) return ATTN_ERR_ALIASING;
  }

  // ---- device
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return ATTN_ERR_NO_DEVICE;
  }
  const int st = device_ready(dev);
  if (st != ATTN_OK) return st;

  CUtensorMap tq, tk, tv, tdo, tout;
  if (!make_map(&tq, q, layout, rep, Hq, Sq, bwd::kTile) || !make_map(&tk, k, layout, rep, Hkv, Sk, bwd::kTile) ||
      !make_map(&tv, v, layout, rep, Hkv, Sk, bwd::kTile) ||
      !make_map(&tdo, dout, layout, rep, Hq, Sq, bwd::kTile) ||
      !make_map(&tout, out, layout, rep, Hq, Sq, bwd::kTile))
    return ATTN_ERR_LAUNCH;

  char* ws = static_cast<char*>(workspace);
  float* stats = reinterpret_cast<float*>(ws);
  float* dq_part = reinterpret_cast<float*>(ws + pl.stats_bytes);
  float* dkv_part = reinterpret_cast<float*>(ws + pl.stats_bytes + pl.dq_bytes);
  const bool causal = (flags & ATTN_FLAG_CAUSAL) != 0;

  bwd::BwdParams p;
  p.Sq = static_cast<int>(Sq);
  p.Sk = static_cast<int>(Sk);
  p.Hq = static_cast<int>(Hq);
  p.Hkv = static_cast<int>(Hkv);
  p.group = static_cast<int>(Hq / Hkv);
  p.layout = layout;
  p.mode = rounding_mode;
  p.c = scale * 1.4426950408889634f;
  p.scale = scale;
  p.timeout_ns = timeout_ns;
  p.cu_q = cu_q;
  p.cu_k = cu_k;
  p.max_sq = static_cast<int>(max_sq);
  p.max_sk = static_cast<int>(max_sk);
  p.q_slots = static_cast<int>(pl.q_slots);
  p.k_slots = static_cast<int>(pl.k_slots);
  p.lse = lse;
  p.stats = stats;
  p.dq = static_cast<uint16_t*>(dq);
  p.dk = static_cast<uint16_t*>(dk);
  p.dv = static_cast<uint16_t*>(dv);
  // The same for the two products; what differs is set at each.
  const int64_t keys_per_head = varlen ? (Sk + B - 1) / B : Sk;
  const int64_t rows_per_head = varlen ? (Sq + B - 1) / B : Sq;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);

  p.BH = static_cast<int>(B * Hq);
  p.n_tiles = static_cast<int>(pl.q_tiles);
  p.n_splits = pl.dq_splits;
  p.withhold = withhold == 0;
  place(&p, causal ? heads_together(B * Hq, 512 * keys_per_head * Hkv / Hq) : 1, Hq);
  p.part = dq_part;
  if (!launch(kDq[variant_of(causal, varlen, pl.dq_long)], B * Hq * pl.q_tiles * pl.dq_splits, attn::kThreads,
              bwd::kDqSmem, cs, false, tq, tk, tv, tdo, tout, p))
    return ATTN_ERR_LAUNCH;

  p.BH = static_cast<int>(B * Hkv);
  p.n_tiles = static_cast<int>(pl.k_tiles);
  p.n_splits = pl.dkv_splits;
  p.withhold = withhold == 1;
  place(&p, causal ? heads_together(B * Hkv, 512 * rows_per_head * (Hq / Hkv)) : 1, Hkv);
  p.part = dkv_part;
  if (!launch(kDkv[variant_of(causal, varlen, pl.dkv_long)], B * Hkv * pl.k_tiles * pl.dkv_splits,
              attn::kThreads, bwd::kDkvSmem, cs, true, tq, tk, tv, tdo, p))
    return ATTN_ERR_LAUNCH;
  if (pl.dq_splits > 1 || pl.dkv_splits > 1) {
    bwd::JoinParams jp;
    jp.layout = layout;
    jp.mode = rounding_mode;
    jp.B = static_cast<int>(B);
    jp.dq.part = dq_part;
    jp.dq.out[0] = jp.dq.out[1] = p.dq;
    jp.dq.factor[0] = jp.dq.factor[1] = scale;
    jp.dq.results = 1;
    jp.dq.cu = jp.dkv.cu2 = cu_q;
    jp.dq.cu2 = jp.dkv.cu = cu_k;
    jp.dq.S = jp.dkv.S2 = p.Sq;
    jp.dq.S2 = jp.dkv.S = p.Sk;
    jp.dq.max_s = jp.dkv.max_s2 = p.max_sq;
    jp.dq.max_s2 = jp.dkv.max_s = p.max_sk;
    jp.dq.H = p.Hq;
    jp.dkv.H = p.Hkv;
    jp.dq.slots = p.q_slots;
    jp.dkv.slots = p.k_slots;
    jp.dq.n_tiles = static_cast<int>(pl.q_tiles);
    jp.dkv.n_tiles = static_cast<int>(pl.k_tiles);
    jp.dq.n_splits = pl.dq_splits;
    jp.dkv.n_splits = pl.dkv_splits;
    jp.dkv.part = dkv_part;
    jp.dkv.out[0] = p.dk;
    jp.dkv.out[1] = p.dv;
    jp.dkv.factor[0] = scale;
    jp.dkv.factor[1] = 1.f;
    jp.dkv.results = 2;
    const int64_t dq_blocks = pl.dq_splits > 1 ? B * Hq * pl.q_tiles * kJoinPer : 0;
    const int64_t dkv_blocks = pl.dkv_splits > 1 ? 2 * B * Hkv * pl.k_tiles * kJoinPer : 0;
    jp.dq_blocks = static_cast<int>(dq_blocks);
    if (!launch(varlen ? bwd::attn_bwd_join<true> : bwd::attn_bwd_join<false>, dq_blocks + dkv_blocks,
                16 * bwd::kJoinRows, 0, cs, true, jp))
      return ATTN_ERR_LAUNCH;
  }
  return ATTN_OK;
}

int64_t workspace_of(bool varlen, int64_t B, int64_t Hq, int64_t Hkv, int64_t Sq, int64_t Sk, int64_t max_sq,
                     int64_t max_sk, int64_t d) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Sq < 1 || Sk < 1) return ATTN_ERR_INVALID_ARG;
  if (max_sq < 1 || max_sk < 1 || max_sq > Sq || max_sk > Sk) return ATTN_ERR_INVALID_ARG;
  if (d != attn::kD) return ATTN_ERR_UNSUPPORTED;
  if (Sq > kLim31 || Sk > kLim31 || Hq > kLim31 || B > kLim31) return ATTN_ERR_TOO_LARGE;
  Plan pl;
  if (!make_plan(&pl, varlen, B, Hq, Hkv, Sq, Sk, max_sq, max_sk)) return ATTN_ERR_TOO_LARGE;
  return pl.bytes();
}

}  // namespace

extern "C" {

int attn_bwd(const void* dout, const void* q, const void* k, const void* v, const void* out, const float* lse,
             void* dq, void* dk, void* dv, int layout, int64_t B, int64_t Hq, int64_t Hkv, int64_t Sq,
             int64_t Sk, int64_t d, float scale, int rounding_mode, int flags, void* workspace,
             int64_t workspace_bytes, void* stream) {
  return bwd_impl(dout, q, k, v, out, lse, dq, dk, dv, nullptr, nullptr, layout, B, Hq, Hkv, Sq, Sk, Sq, Sk, d,
                  scale, rounding_mode, flags, workspace, workspace_bytes, stream);
}

int64_t attn_bwd_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t Sq, int64_t Sk, int64_t d) {
  return workspace_of(false, B, Hq, Hkv, Sq, Sk, Sq, Sk, d);
}

int attn_bwd_varlen(const void* dout, const void* q, const void* k, const void* v, const void* out,
                    const float* lse, void* dq, void* dk, void* dv, const int32_t* cu_seqlens_q,
                    const int32_t* cu_seqlens_k, int64_t B, int64_t Hq, int64_t Hkv, int64_t total_q,
                    int64_t total_k, int64_t max_seqlen_q, int64_t max_seqlen_k, int64_t d, float scale,
                    int rounding_mode, int flags, void* workspace, int64_t workspace_bytes, void* stream) {
  if (!cu_seqlens_q || !cu_seqlens_k) return ATTN_ERR_INVALID_ARG;
  return bwd_impl(dout, q, k, v, out, lse, dq, dk, dv, cu_seqlens_q, cu_seqlens_k, ATTN_LAYOUT_BSHD, B, Hq, Hkv,
                  total_q, total_k, max_seqlen_q, max_seqlen_k, d, scale, rounding_mode, flags, workspace,
                  workspace_bytes, stream);
}

int attn_bwd_timeout_selftest(const void* dout, const void* q, const void* k, const void* v, const void* out,
                              const float* lse, void* dq, void* dk, void* dv, int layout, int64_t B,
                              int64_t Hq, int64_t Hkv, int64_t Sq, int64_t Sk, int64_t d, float scale,
                              int rounding_mode, int flags, void* workspace, int64_t workspace_bytes,
                              void* stream, uint64_t timeout_ns, int kernel) {
  if (timeout_ns < 1 || timeout_ns > kTimeoutNs || kernel < 0 || kernel > 1) return ATTN_ERR_INVALID_ARG;
  return bwd_impl(dout, q, k, v, out, lse, dq, dk, dv, nullptr, nullptr, layout, B, Hq, Hkv, Sq, Sk, Sq, Sk, d,
                  scale, rounding_mode, flags, workspace, workspace_bytes, stream, timeout_ns, kernel);
}

int64_t attn_bwd_varlen_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t total_q, int64_t total_k,
                                        int64_t max_seqlen_q, int64_t max_seqlen_k, int64_t d) {
  return workspace_of(true, B, Hq, Hkv, total_q, total_k, max_seqlen_q, max_seqlen_k, d);
}

}  // extern "C"
