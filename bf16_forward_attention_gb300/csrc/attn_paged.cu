// attn_paged.cu - host side of attention over a paged cache, declared in include/attn_fwd.h:
// checks the call, lays out the workspace and launches, on the caller's stream, the runs of
// units, then the join of the items they cut with, beside it, the keys' masses where they are wanted.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "attn_fwd.h"
#include "attn_paged_kernel.cuh"
#include "host_common.h"

namespace {

std::atomic<bool> g_launched{false};

}

namespace attn_host {

bool paged_take_status(unsigned int* s) { return take_status(attn::g_attn_status, g_launched, s); }

}  // namespace attn_host

namespace {

using namespace attn_host;
namespace paged = attn::paged;

std::mutex g_mutex;
bool g_ready[kMaxDevices];

using Kernel = void (*)(const paged::Params);
// A block's rows, and the kernel for them, with and without the keys' masses.
struct Form {
  int rows, threads, smem, ctas, cost;
  bool waits;  // for the tensor cores
  Kernel fwd[2];
};
template <int kGroups>
constexpr Form form() {
  using S = paged::Shape<kGroups>;
  return {S::kRows, S::kThreads, S::kSmem, 2, paged::kItemCost, false,
          {paged::attn_paged_fwd<kGroups, false>, paged::attn_paged_fwd<kGroups, true>}};
}
template <int kCopies>
constexpr Form rows_form() {
  return {128 / kCopies, paged::kRowsThreads, paged::kRowsSmem, 2, paged::kRowsItemCost, true,
          {paged::attn_paged_rows<kCopies, false>, paged::attn_paged_rows<kCopies, true>}};
}
// The first that holds a block's rows. Up to 16 the warp-level form, from 17 on the tensor cores: us a call with
// the one / the other at 1, 8, 9 and 16 rows a kv head, pages of 16:
//   64 caches of up to 8192 keys, 8 kv heads  178 / 199  178 / 199  197 / 200  201 / 202
//   64 of up to 300                            23 / 34    25 / 34    29 / 35    31 / 35
//   one of 100000                              75 / 85    75 / 85    81 / 87    81 / 86
constexpr Form kForms[] = {form<1>(), form<2>(), rows_form<4>(), rows_form<2>(), rows_form<1>()};

int device_ready() {
  const int st = arch_here();
  if (st != ATTN_OK) return st;
  int dev = -1;
  cudaGetDevice(&dev);
  std::lock_guard<std::mutex> lock(g_mutex);
  if (g_ready[dev]) return ATTN_OK;
  for (const Form& form : kForms)
    for (Kernel fn : form.fwd)
      if (cudaFuncSetAttribute(reinterpret_cast<const void*>(fn), cudaFuncAttributeMaxDynamicSharedMemorySize,
                               form.smem) != cudaSuccess) {
        cudaGetLastError();
        return ATTN_ERR_LAUNCH;
      }
  g_ready[dev] = true;
  return ATTN_OK;
}

constexpr int64_t kLim31 = (int64_t(1) << 31) - 1;

struct Plan {
  const Form* form;
  int64_t rows, rows4, blocks, block_rows, cap, runs;
  int64_t o_bytes, rl_bytes, cut_bytes, lse2_bytes, logit_bytes;
  int64_t bytes() const { return o_bytes + rl_bytes + cut_bytes + lse2_bytes + logit_bytes; }
};

int64_t up256(int64_t n) { return (n + 255) & ~int64_t(255); }

int make_plan(Plan* pl, int64_t B, int64_t Hq, int64_t Hkv, int64_t Sq, int64_t page_size, int64_t max_pages,
              int64_t d, bool mass) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Sq < 1 || page_size < 1 || max_pages < 1)
    return ATTN_ERR_INVALID_ARG;
  if (d != attn::kD) return ATTN_ERR_UNSUPPORTED;
  const int64_t group = Hq / Hkv;
  if (B > kLim31 || Hq > (1 << 20) || Sq > kLim31 / Hq || page_size > kLim31 || max_pages > (kLim31 - 64) / page_size)
    return ATTN_ERR_TOO_LARGE;  // a tile past the last key still has an int's number
  pl->cap = page_size * max_pages;
  // Blocks of equal size, an even number of rows where there are several (pairs of logits).
  pl->rows = Sq * group;
  pl->rows4 = (pl->rows + 3) & ~int64_t(3);
  pl->blocks = (pl->rows + paged::kMaxRows - 1) / paged::kMaxRows;
  pl->block_rows = pl->blocks == 1 ? pl->rows : ((pl->rows + pl->blocks - 1) / pl->blocks + 1) & ~int64_t(1);
  pl->form = kForms;
  while (pl->form->rows < pl->block_rows) ++pl->form;
  if (Hkv * pl->blocks > kLim31 || B > (int64_t(1) << 40) / (Hkv * pl->blocks)) return ATTN_ERR_TOO_LARGE;
  const int64_t items = B * Hkv * pl->blocks;
  // Places of all items (see find_run) below 2^47: a run's bounds are products with the number of runs.
  const int64_t units = (pl->cap + paged::kUnit - 1) / paged::kUnit + paged::kRowsItemCost;
  if (items > (int64_t(1) << 47) / units) return ATTN_ERR_TOO_LARGE;
  // The CTAs that the GPU holds at once; fewer where the caches are too small for as many runs.
  const int64_t most = items * units;
  const int64_t fill = pl->form->ctas * int64_t(sms_here());
  pl->runs = most < fill ? most : fill;
  pl->o_bytes = 2 * pl->runs * pl->form->rows * attn::kD * 4;
  pl->rl_bytes = up256(2 * pl->runs * pl->form->rows * 8);
  pl->cut_bytes = up256(pl->runs * int64_t(sizeof(paged::Cut)));
  pl->lse2_bytes = pl->logit_bytes = 0;
  if (mass) {
    const int64_t row_bytes = B * Hkv * pl->rows4 * 4;
    if (row_bytes > (int64_t(1) << 50) / pl->cap) return ATTN_ERR_TOO_LARGE;
    pl->lse2_bytes = up256(row_bytes);
    pl->logit_bytes = up256(row_bytes * pl->cap);
  }
  return ATTN_OK;
}

int run(const void* q, const void* k_pages, const void* v_pages, const int32_t* page_table,
                   const int32_t* seqlens, void* out, float* lse, float* mass, int layout, int64_t B, int64_t Hq,
                   int64_t Hkv, int64_t Sq, int64_t n_pages, int64_t page_size, int64_t page_stride,
                   int64_t max_pages, int64_t d, float scale, int rounding_mode, int flags, void* workspace,
                   int64_t workspace_bytes, void* stream, uint64_t timeout_ns, bool withhold) {
  // ---- host-side validation (nothing is launched on failure)
  if (!q || !page_table || !seqlens || !out || !lse || !workspace) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  if (flags & ~ATTN_FLAG_CAUSAL) return ATTN_ERR_UNSUPPORTED;
  if (layout != ATTN_LAYOUT_BHSD && layout != ATTN_LAYOUT_BSHD) return ATTN_ERR_UNSUPPORTED;
  if (rounding_mode < ATTN_ROUND_RTNE || rounding_mode > ATTN_ROUND_RTZ) return ATTN_ERR_UNSUPPORTED;
  Plan pl;
  int st = make_plan(&pl, B, Hq, Hkv, Sq, page_size, max_pages, d, mass != nullptr);
  if (st != ATTN_OK) return st;
  st = check_pages(k_pages, v_pages, n_pages, page_size, page_stride, Hkv);
  if (st != ATTN_OK) return st;
  if (workspace_bytes < pl.bytes()) return ATTN_ERR_INVALID_ARG;
  if (withhold && !pl.form->waits) return ATTN_ERR_UNSUPPORTED;
  for (const void* p : {q, static_cast<const void*>(out), static_cast<const void*>(workspace)})
    if (reinterpret_cast<uintptr_t>(p) & 15u) return ATTN_ERR_MISALIGNED;
  if ((reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(seqlens) |
       reinterpret_cast<uintptr_t>(page_table) | reinterpret_cast<uintptr_t>(mass)) & 3u)
    return ATTN_ERR_MISALIGNED;
  const uint64_t nq = uint64_t(B) * Hq * Sq * 256;
  const uint64_t np = uint64_t(PageSet{k_pages, n_pages, page_stride, page_size * Hkv}.bytes());
  struct Span {
    const void* p;
    uint64_t n;
  };
  const Span in[] = {{q, nq}, {k_pages, np}, {v_pages, np}, {page_table, uint64_t(B) * max_pages * 4},
                     {seqlens, uint64_t(B) * 4}};
  const Span written[] = {{out, nq}, {lse, nq / 64}, {workspace, uint64_t(pl.bytes())},
                          {mass, mass ? uint64_t(B) * Hkv * pl.cap * 4 : 0}};
  for (int i = 0; i < 4; ++i) {
    if (!written[i].n) continue;
    for (const Span& s : in)
      if (overlaps(written[i].p, written[i].n, s.p, s.n)) return ATTN_ERR_ALIASING;
    for (int j = 0; j < i; ++j)
      if (overlaps(written[i].p, written[i].n, written[j].p, written[j].n)) return ATTN_ERR_ALIASING;
  }

  // ---- device
  st = device_ready();
  if (st != ATTN_OK) return st;
  paged::Params p = {};
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k_pages);
  p.v = static_cast<const uint16_t*>(v_pages);
  p.table = page_table;
  p.seqlens = seqlens;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.mass = mass;
  char* ws = static_cast<char*>(workspace);
  p.part_o = reinterpret_cast<float*>(ws);
  p.part_rl = reinterpret_cast<float*>(ws + pl.o_bytes);
  p.cuts = reinterpret_cast<paged::Cut*>(ws + pl.o_bytes + pl.rl_bytes);
  p.lse2 = reinterpret_cast<float*>(ws + pl.o_bytes + pl.rl_bytes + pl.cut_bytes);
  p.logits = reinterpret_cast<float*>(ws + pl.o_bytes + pl.rl_bytes + pl.cut_bytes + pl.lse2_bytes);
  p.B = static_cast<int>(B);
  p.Hq = static_cast<int>(Hq);
  p.Hkv = static_cast<int>(Hkv);
  p.group = static_cast<int>(Hq / Hkv);
  p.Sq = static_cast<int>(Sq);
  p.cap = static_cast<int>(pl.cap);
  p.layout = layout;
  p.causal = (flags & ATTN_FLAG_CAUSAL) ? 1 : 0;
  p.mode = rounding_mode;
  p.n_pages = static_cast<int>(n_pages);
  p.page_size = static_cast<int>(page_size);
  const PageDivisor div = page_divisor(page_size);
  p.page_mul = div.mul;
  p.page_shift = div.shift;
  p.max_pages = static_cast<int>(max_pages);
  p.page_rows = static_cast<int>(page_stride / attn::kD);
  p.rows = static_cast<int>(pl.rows);
  p.rows4 = static_cast<int>(pl.rows4);
  p.blocks = static_cast<int>(pl.blocks);
  p.block_rows = static_cast<int>(pl.block_rows);
  p.rows8 = pl.form->rows;
  p.cost = pl.form->cost;
  p.runs = static_cast<int>(pl.runs);
  p.join_groups = static_cast<int>((pl.block_rows + 7) / 8);
  p.c = scale * 1.4426950408889634f;
  p.timeout_ns = timeout_ns;
  p.withhold = withhold ? 1 : 0;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  g_launched.store(true);
  if (!launch(pl.form->fwd[mass ? 1 : 0], pl.runs, pl.form->threads, pl.form->smem, cs, false, p))
    return ATTN_ERR_LAUNCH;
  // The blocks of the masses: what the join's leave of an SM at once.
  const bool few = pl.runs / (Hkv * pl.blocks) + 2 <= paged::kJoinFew;
  const int64_t blocks = pl.runs * p.join_groups + (mass ? (few ? 3 : 1) * int64_t(sms_here()) : 0);
  const Kernel finish = few ? (mass ? paged::attn_paged_finish<1, true> : paged::attn_paged_finish<1, false>)
                            : (mass ? paged::attn_paged_finish<4, true> : paged::attn_paged_finish<4, false>);
  if (!launch(finish, blocks, paged::kJoinThreads * (few ? 1 : 4), static_cast<int>(pl.runs) * 32, cs, true, p))
    return ATTN_ERR_LAUNCH;
  return ATTN_OK;
}

}  // namespace

extern "C" {

int64_t attn_fwd_paged_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t Sq, int64_t page_size,
                                       int64_t max_pages, int64_t d, int with_mass) {
  Plan pl;
  const int st = make_plan(&pl, B, Hq, Hkv, Sq, page_size, max_pages, d, with_mass != 0);
  return st != ATTN_OK ? st : pl.bytes();
}

int attn_fwd_paged(const void* q, const void* k_pages, const void* v_pages, const int32_t* page_table,
                   const int32_t* seqlens, void* out, float* lse, float* mass, int layout, int64_t B, int64_t Hq,
                   int64_t Hkv, int64_t Sq, int64_t n_pages, int64_t page_size, int64_t page_stride,
                   int64_t max_pages, int64_t d, float scale, int rounding_mode, int flags, void* workspace,
                   int64_t workspace_bytes, void* stream) {
  return run(q, k_pages, v_pages, page_table, seqlens, out, lse, mass, layout, B, Hq, Hkv, Sq, n_pages, page_size,
             page_stride, max_pages, d, scale, rounding_mode, flags, workspace, workspace_bytes, stream, kTimeoutNs,
             false);
}

int attn_fwd_paged_timeout_selftest(const void* q, const void* k_pages, const void* v_pages,
                                    const int32_t* page_table, const int32_t* seqlens, void* out, float* lse,
                                    float* mass, int layout, int64_t B, int64_t Hq, int64_t Hkv, int64_t Sq,
                                    int64_t n_pages, int64_t page_size, int64_t page_stride, int64_t max_pages,
                                    int64_t d, float scale, int rounding_mode, int flags, void* workspace,
                                    int64_t workspace_bytes, void* stream, uint64_t timeout_ns) {
  if (timeout_ns < 1 || timeout_ns > 2000000000ull) return ATTN_ERR_INVALID_ARG;
  return run(q, k_pages, v_pages, page_table, seqlens, out, lse, mass, layout, B, Hq, Hkv, Sq, n_pages, page_size,
             page_stride, max_pages, d, scale, rounding_mode, flags, workspace, workspace_bytes, stream, timeout_ns,
             true);
}

}  // extern "C"
