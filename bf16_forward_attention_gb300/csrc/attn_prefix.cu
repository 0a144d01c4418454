// attn_prefix.cu - host side of attention on a shared prefix, declared in
// include/attn_fwd.h: checks the call, lays out the workspace (packed queries and
// the parts' unnormalised rows) and launches, on the caller's stream, the
// prefix (the fused kernel's split form), beside it the sequences' own keys, and the join.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "attn_fwd.h"
#include "attn_prefix_kernel.cuh"
#include "host_common.h"

namespace attn_host {

bool prefix_take_status(unsigned int* s) { return take_status(attn::g_attn_status, s); }

}  // namespace attn_host

namespace {

using namespace attn_host;
namespace pre = attn::prefix;

std::mutex g_mutex;
int g_state[kMaxDevices];  // 0 = not set up, 1 = ready, negative = status to return

using OwnKernel = void (*)(const pre::OwnParams);
// By 8-row tiles of a block; the second four for long parts.
constexpr OwnKernel kOwn[8] = {pre::attn_prefix_own<1, false>, pre::attn_prefix_own<2, false>,
                               pre::attn_prefix_own<3, false>, pre::attn_prefix_own<4, false>,
                               pre::attn_prefix_own<1, true>,  pre::attn_prefix_own<2, true>,
                               pre::attn_prefix_own<3, true>,  pre::attn_prefix_own<4, true>};

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
  for (OwnKernel fn : kOwn)
    if (cudaFuncSetAttribute(reinterpret_cast<const void*>(fn), cudaFuncAttributeMaxDynamicSharedMemorySize,
                             pre::kOwnSmem) != cudaSuccess) {
      cudaGetLastError();
      return ATTN_ERR_LAUNCH;
    }
  g_state[dev] = 1;
  return ATTN_OK;
}

constexpr int64_t kLim31 = (int64_t(1) << 31) - 1;

struct Plan {
  int64_t rows, rows_pad;  // packed rows of a kv head
  int64_t block_rows;      // of a block of the own keys' kernel, at most 32
  int64_t blocks;          // blocks per (sequence, kv head)
  bool prefix_here;        // few packed rows: the own keys' kernel takes the prefix as well
  int prefix_splits, own_splits;
  int64_t packed_bytes, o_bytes, rl_bytes;
  int64_t bytes() const { return packed_bytes + o_bytes + rl_bytes; }
};

int64_t up256(int64_t n) { return (n + 255) & ~int64_t(255); }

bool make_plan(Plan* pl, int64_t B, int64_t Hq, int64_t Hkv, int64_t Sq, int64_t Sp, int64_t cap) {
  const int64_t group = Hq / Hkv;
  if (B > kLim31 / Sq / group / 2) return false;
  pl->rows = B * Sq * group;
  pl->rows_pad = up256(pl->rows);
  const int64_t per_seq = Sq * group;
  // A sequence's rows in blocks of equal size; a batch of up to 32 rows in one (the
  // block then takes the prefix as well, below).
  pl->blocks = (per_seq + pre::kMaxRows - 1) / pre::kMaxRows;
  pl->block_rows = (per_seq + pl->blocks - 1) / pl->blocks;
  if (Sp > 0 && pl->rows <= pre::kMaxRows) pl->block_rows = pl->rows;
  // 128 parts at most: rows, grids and row numbers then stay ints.
  if (Hkv > kLim31 / pl->rows_pad / 128 || B > kLim31 / Hkv / pl->blocks / 64) return false;
  const int64_t sms = sms_here();
  // Own keys: two blocks for every SM (what it holds at once), of at least 256 keys of
  // the cache each (lengths are on the device; a short sequence's parts are shorter).
  const int64_t items = B * Hkv * pl->blocks;
  // Blocks of more than 16 rows are bound by their instructions, and the additions of kFold
  // would cost them 5 to 28%: their parts are kept short instead.
  const bool cut_short = pl->block_rows > 16;
  auto parts_of = [](int64_t keys) { return (keys + pre::kFoldKeys - 1) / pre::kFoldKeys; };
  int64_t s = (2 * sms + items - 1) / items;
  const int64_t most = (cap + 255) / 256;
  if (s > most) s = most;
  if (cut_short && s < parts_of(cap)) s = parts_of(cap);
  if (s > 64) s = 64;
  pl->own_splits = static_cast<int>(s);
  pl->prefix_here = Sp > 0 && pl->rows <= pre::kMaxRows;
  pl->prefix_splits = 0;
  if (pl->prefix_here) {
    // All packed rows of a kv head fit one block: the kernel of the own keys takes the
    // prefix as well, in the same launch, read once. (The fused kernel's 256-row items
    // would be nearly empty, and it needs the rows packed first.)
    int64_t n = (2 * sms + Hkv - 1) / Hkv;
    const int64_t cut = (Sp + 255) / 256;
    if (n > cut) n = cut;
    if (cut_short && n < parts_of(Sp)) n = parts_of(Sp);
    if (n > 64) n = 64;
    pl->prefix_splits = static_cast<int>(n);
  } else if (Sp > 0) {
    // The prefix product runs beside the own keys' kernel, on one SM per CTA. The split
    // count with the least estimated time: the product takes 1.9 us per key tile of 128
    // keys and 256 rows, and 8 us a CTA to start and end; meanwhile the own keys (half
    // of each cache, as lengths are on the device) are read by the other SMs, of which 105
    // reach the full 6.5 TB/s (an SM takes 62 GB/s from L2); what is left is read
    // afterwards. A split more costs the join 1040 bytes a row.
    const int64_t tiles = (Sp + attn::kBN - 1) / attn::kBN;
    const int64_t cta = Hkv * (pl->rows_pad / 256);
    const double own_us = static_cast<double>(B) * Hkv * cap * 256 / 6.5e6;
    double least = 1e30;
    for (int n = 1; n <= 64 && n <= tiles; ++n) {
      const int64_t waves = (cta * n + sms - 1) / sms;
      const double us = static_cast<double>(waves) * (1.9 * ((tiles + n - 1) / n) + 8);
      const double rate = cta * n >= sms ? 0.0 : (sms - cta * n >= 105 ? 1.0 : (sms - cta * n) / 105.0);
      const double left = own_us > us * rate ? own_us - us * rate : 0.0;
      const double cost = us + left + static_cast<double>(cta) * n * 256 * 1040 * 2 / 6.5e6;
      if (cost < least) {
        least = cost;
        pl->prefix_splits = n;
      }
    }
  }
  const int64_t parts = pl->prefix_splits + pl->own_splits;
  pl->packed_bytes = Sp > 0 && !pl->prefix_here ? up256(pl->rows * Hkv * 256) : 0;
  pl->o_bytes = parts * Hkv * pl->rows_pad * attn::kD * 4;
  pl->rl_bytes = parts * Hkv * pl->rows_pad * 8;
  return true;
}

int check_sizes(int64_t B, int64_t Hq, int64_t Hkv, int64_t Sq, int64_t Sp, int64_t cap, int64_t d, Plan* pl) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Sq < 1 || Sp < 0 || cap < 1) return ATTN_ERR_INVALID_ARG;
  if (d != attn::kD) return ATTN_ERR_UNSUPPORTED;
  if (B > kLim31 || Hq > kLim31 || Sq > kLim31 || Sp > kLim31 || cap > kLim31) return ATTN_ERR_TOO_LARGE;
  const int64_t kStrideLim = int64_t(1) << 40;  // TMA strides
  if (Sp > 0 && Hkv > kStrideLim / 256 / Sp) return ATTN_ERR_TOO_LARGE;
  if (B > (int64_t(1) << 54) / Hkv / cap) return ATTN_ERR_TOO_LARGE;
  return make_plan(pl, B, Hq, Hkv, Sq, Sp, cap) ? ATTN_OK : ATTN_ERR_TOO_LARGE;
}

}  // namespace

extern "C" {

int64_t attn_fwd_prefix_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t Sq, int64_t Sp,
                                        int64_t cap, int64_t d) {
  Plan pl;
  const int st = check_sizes(B, Hq, Hkv, Sq, Sp, cap, d, &pl);
  return st != ATTN_OK ? st : pl.bytes();
}

int attn_fwd_prefix(const void* q, const void* k_prefix, const void* v_prefix, const void* k, const void* v,
                    const int32_t* seqlens, void* out, float* lse, int layout, int64_t B, int64_t Hq,
                    int64_t Hkv, int64_t Sq, int64_t Sp, int64_t cap, int64_t d, float scale,
                    int rounding_mode, int flags, void* workspace, int64_t workspace_bytes, void* stream) {
  // ---- host-side validation (nothing is launched on failure)
  if (!q || !k || !v || !seqlens || !out || !lse || !workspace) return ATTN_ERR_INVALID_ARG;
  if (Sp > 0 && (!k_prefix || !v_prefix)) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  if (flags & ~ATTN_FLAG_CAUSAL) return ATTN_ERR_UNSUPPORTED;
  if (layout != ATTN_LAYOUT_BHSD && layout != ATTN_LAYOUT_BSHD) return ATTN_ERR_UNSUPPORTED;
  if (rounding_mode < ATTN_ROUND_RTNE || rounding_mode > ATTN_ROUND_RTZ) return ATTN_ERR_UNSUPPORTED;
  Plan pl;
  int st = check_sizes(B, Hq, Hkv, Sq, Sp, cap, d, &pl);
  if (st != ATTN_OK) return st;
  if (workspace_bytes < pl.bytes()) return ATTN_ERR_INVALID_ARG;
  if (Sp == 0) k_prefix = v_prefix = nullptr;
  for (const void* p : {q, k_prefix, v_prefix, k, v, static_cast<const void*>(out),
                        static_cast<const void*>(workspace)})
    if (reinterpret_cast<uintptr_t>(p) & 15u) return ATTN_ERR_MISALIGNED;
  if ((reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(seqlens)) & 3u) return ATTN_ERR_MISALIGNED;
  const uint64_t nq = uint64_t(B) * Hq * Sq * 256, np = uint64_t(Hkv) * Sp * 256,
                 nk = uint64_t(B) * Hkv * cap * 256, nl = nq / 64, nw = uint64_t(pl.bytes());
  struct Span {
    const void* p;
    uint64_t n;
  };
  const Span in[] = {{q, nq}, {k_prefix, np}, {v_prefix, np}, {k, nk}, {v, nk}, {seqlens, uint64_t(B) * 4}};
  const Span written[] = {{out, nq}, {lse, nl}, {workspace, nw}};
  for (int i = 0; i < 3; ++i) {
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
  st = device_ready(dev);
  if (st != ATTN_OK) return st;

  char* ws = static_cast<char*>(workspace);
  uint16_t* packed = reinterpret_cast<uint16_t*>(ws);
  float* part_o = reinterpret_cast<float*>(ws + pl.packed_bytes);
  float* part_rl = reinterpret_cast<float*>(ws + pl.packed_bytes + pl.o_bytes);
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);

  pre::OwnParams p;
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.seqlens = seqlens;
  p.kp = static_cast<const uint16_t*>(k_prefix);
  p.vp = static_cast<const uint16_t*>(v_prefix);
  const bool fused_prefix = Sp > 0 && !pl.prefix_here;
  p.beside_prefix = fused_prefix ? 1 : 0;
  p.part_o = part_o;
  p.part_rl = part_rl;
  p.B = static_cast<int>(B);
  p.Hq = static_cast<int>(Hq);
  p.Hkv = static_cast<int>(Hkv);
  p.group = static_cast<int>(Hq / Hkv);
  p.Sq = static_cast<int>(Sq);
  p.cap = static_cast<int>(cap);
  p.layout = layout;
  p.causal = (flags & ATTN_FLAG_CAUSAL) ? 1 : 0;
  p.rows = static_cast<int>(pl.rows);
  p.rows_pad = static_cast<int>(pl.rows_pad);
  p.Sp = static_cast<int>(Sp);
  p.own_splits = pl.own_splits;
  p.own_blocks = static_cast<int>(pl.blocks);
  p.prefix_splits = pl.prefix_splits;
  const int64_t prefix_items = pl.prefix_here ? Hkv * pl.prefix_splits : 0;
  p.prefix_items = static_cast<int>(prefix_items);
  p.c = scale * 1.4426950408889634f;
  if (fused_prefix) {
    pre::PackParams k;
    k.q = p.q;
    k.packed = packed;
    k.Hq = p.Hq;
    k.Hkv = p.Hkv;
    k.group = p.group;
    k.Sq = p.Sq;
    k.layout = layout;
    k.rows = p.rows;
    constexpr int kPackRows = pre::kPackThreads / 16;
    if (!launch(pre::attn_prefix_pack, (pl.rows * Hkv + kPackRows - 1) / kPackRows, pre::kPackThreads, 0, cs, false,
                k))
      return ATTN_ERR_LAUNCH;
    st = split_parts(packed, k_prefix, v_prefix, layout, 1, Hkv, pl.rows, Sp, scale, pl.prefix_splits, part_o,
                     part_rl, cs);
    if (st != ATTN_OK) return st;
  }
  p.block_rows = static_cast<int>(pl.block_rows);
  const bool fold = cap > int64_t(pre::kFoldKeys) * pl.own_splits ||
                    (prefix_items > 0 && Sp > int64_t(pre::kFoldKeys) * pl.prefix_splits);
  if (!launch(kOwn[(pl.block_rows + 7) / 8 - 1 + (fold ? 4 : 0)],
              prefix_items + B * Hkv * pl.blocks * pl.own_splits, pre::kOwnThreads, pre::kOwnSmem, cs, fused_prefix,
              p))
    return ATTN_ERR_LAUNCH;
  pre::JoinParams j;
  j.part_o = part_o;
  j.part_rl = part_rl;
  j.seqlens = seqlens;
  j.out = static_cast<uint16_t*>(out);
  j.lse = lse;
  j.Hq = p.Hq;
  j.Hkv = p.Hkv;
  j.group = p.group;
  j.Sq = p.Sq;
  j.cap = p.cap;
  j.layout = layout;
  j.mode = rounding_mode;
  j.rows = p.rows;
  j.rows_pad = p.rows_pad;
  j.n_parts = pl.prefix_splits + pl.own_splits;
  const int64_t join_blocks = (pl.rows * Hkv + pre::kJoinRows - 1) / pre::kJoinRows;
  if (!launch(pre::attn_prefix_join, join_blocks, 32 * pre::kJoinRows, 0, cs, true, j)) return ATTN_ERR_LAUNCH;
  return ATTN_OK;
}

}  // extern "C"
