// attn_evict.cu - host side of a paged cache's eviction, declared in include/attn_fwd.h: checks
// the call, lays out the workspace and launches the selection and the moves.
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "attn_evict_kernel.cuh"
#include "attn_fwd.h"
#include "host_common.h"

namespace {

std::atomic<bool> g_launched{false};

}

namespace attn_host {

bool evict_take_status(unsigned int* s) { return take_status(attn::g_attn_status, g_launched, s); }

}  // namespace attn_host

namespace {

using namespace attn_host;
namespace evict = attn::evict;

constexpr int64_t kLim31 = (int64_t(1) << 31) - 1;

struct Plan {
  int64_t cap, keep, listed_bytes, head_bytes, src_bytes;
  int64_t bytes() const { return listed_bytes + head_bytes + 2 * src_bytes; }
};

int64_t up256(int64_t n) { return (n + 255) & ~int64_t(255); }

int make_plan(Plan* pl, int64_t B, int64_t Hkv, int64_t n_pages, int64_t page_size, int64_t max_pages, int64_t budget) {
  if (B < 1 || Hkv < 1 || n_pages < 1 || page_size < 1 || max_pages < 1 || budget < 1) return ATTN_ERR_INVALID_ARG;
  if (B > kLim31 / evict::kCluster / Hkv || n_pages > kLim31 || page_size > kLim31 ||
      max_pages > (kLim31 - (1 << 16)) / page_size || budget > kLim31 - (1 << 16))
    return ATTN_ERR_TOO_LARGE;  // places up to a round past the last still have an int's number
  pl->cap = page_size * max_pages;
  pl->keep = budget < pl->cap ? budget : pl->cap;
  if (B * Hkv > (int64_t(1) << 50) / pl->keep) return ATTN_ERR_TOO_LARGE;
  pl->listed_bytes = up256(n_pages * 4);
  pl->head_bytes = up256(B * Hkv * int64_t(sizeof(int2)));
  pl->src_bytes = up256(B * Hkv * pl->keep * 4);
  return ATTN_OK;
}

}  // namespace

extern "C" {

int64_t attn_cache_evict_workspace_bytes(int64_t B, int64_t Hkv, int64_t n_pages, int64_t page_size,
                                         int64_t max_pages, int64_t budget) {
  Plan pl;
  const int st = make_plan(&pl, B, Hkv, n_pages, page_size, max_pages, budget);
  return st != ATTN_OK ? st : pl.bytes();
}

int attn_cache_evict(void* k_pages, void* v_pages, const int32_t* page_table, const int32_t* seqlens,
                     const float* mass, float* mass_out, int32_t* seqlens_out, int layout, int64_t B, int64_t Hkv,
                     int64_t n_pages, int64_t page_size, int64_t page_stride, int64_t max_pages, int64_t d,
                     int64_t budget, int64_t recent, void* workspace, int64_t workspace_bytes, void* stream) {
  // ---- host-side validation (nothing is launched on failure)
  if (!page_table || !seqlens || !mass || !mass_out || !seqlens_out || !workspace) return ATTN_ERR_INVALID_ARG;
  if (recent < 0 || recent > budget) return ATTN_ERR_INVALID_ARG;
  if (d != attn::kD) return ATTN_ERR_UNSUPPORTED;
  if (layout != ATTN_LAYOUT_BHSD && layout != ATTN_LAYOUT_BSHD) return ATTN_ERR_UNSUPPORTED;
  Plan pl;
  int st = make_plan(&pl, B, Hkv, n_pages, page_size, max_pages, budget);
  if (st != ATTN_OK) return st;
  st = check_pages(k_pages, v_pages, n_pages, page_size, page_stride, Hkv);
  if (st != ATTN_OK) return st;
  if (workspace_bytes < pl.bytes()) return ATTN_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(workspace) & 15u) return ATTN_ERR_MISALIGNED;
  for (const void* p : {static_cast<const void*>(page_table), static_cast<const void*>(seqlens),
                        static_cast<const void*>(mass), static_cast<const void*>(mass_out),
                        static_cast<const void*>(seqlens_out)})
    if (reinterpret_cast<uintptr_t>(p) & 3u) return ATTN_ERR_MISALIGNED;
  const PageSet kp = {k_pages, n_pages, page_stride, page_size * Hkv}, vp = {v_pages, n_pages, page_stride,
                                                                            page_size * Hkv};
  if (pages_meet(kp, vp)) return ATTN_ERR_ALIASING;
  struct Span {
    const void* p;
    uint64_t n;
  };
  const uint64_t n_mass = uint64_t(B) * Hkv * pl.cap * 4, n_lens = uint64_t(B) * 4;
  const Span pages[] = {{k_pages, uint64_t(kp.bytes())}, {v_pages, uint64_t(vp.bytes())}};
  const Span rest[] = {{page_table, uint64_t(B) * max_pages * 4}, {seqlens, n_lens}, {mass, n_mass},
                       {workspace, uint64_t(pl.bytes())}, {mass_out, n_mass}, {seqlens_out, n_lens}};
  auto meet = [](const Span& a, const Span& b) { return overlaps(a.p, a.n, b.p, b.n); };
  for (int i = 0; i < 6; ++i) {
    if (meet(rest[i], pages[0]) || meet(rest[i], pages[1])) return ATTN_ERR_ALIASING;
    for (int j = 0; j < i; ++j) {
      if (i < 3) continue;  // inputs may overlap each other
      const bool in_place = (i == 4 && j == 2 && mass_out == mass) || (i == 5 && j == 1 && seqlens_out == seqlens);
      if (!in_place && meet(rest[i], rest[j])) return ATTN_ERR_ALIASING;
    }
  }

  // ---- device
  st = arch_here();
  if (st != ATTN_OK) return st;
  char* ws = static_cast<char*>(workspace);
  evict::Params p = {};
  p.k = static_cast<uint16_t*>(k_pages);
  p.v = static_cast<uint16_t*>(v_pages);
  p.table = page_table;
  p.seqlens = seqlens;
  p.mass = mass;
  p.mass_out = mass_out;
  p.seqlens_out = seqlens_out;
  p.listed = reinterpret_cast<int*>(ws);
  p.head = reinterpret_cast<int2*>(ws + pl.listed_bytes);
  p.src = reinterpret_cast<int*>(ws + pl.listed_bytes + pl.head_bytes);
  p.src_mass = reinterpret_cast<float*>(ws + pl.listed_bytes + pl.head_bytes + pl.src_bytes);
  p.page_rows = static_cast<int>(page_stride / attn::kD);
  p.B = static_cast<int>(B);
  p.Hkv = static_cast<int>(Hkv);
  p.cap = static_cast<int>(pl.cap);
  p.layout = layout;
  p.n_pages = static_cast<int>(n_pages);
  p.page_size = static_cast<int>(page_size);
  const PageDivisor div = page_divisor(page_size);
  p.page_mul = div.mul;
  p.page_shift = div.shift;
  p.max_pages = static_cast<int>(max_pages);
  p.budget = static_cast<int>(budget);
  p.recent = static_cast<int>(recent);
  p.keep = static_cast<int>(pl.keep);
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  g_launched.store(true);
  if (cudaMemsetAsync(p.listed, 0, static_cast<size_t>(n_pages) * 4, cs) != cudaSuccess) {
    cudaGetLastError();
    return ATTN_ERR_LAUNCH;
  }
  if (!launch(evict::attn_evict_select, B * Hkv, evict::kSelectThreads, 0, cs, false, p)) return ATTN_ERR_LAUNCH;
  if (!launch(evict::attn_evict_move, B * Hkv * evict::kCluster, evict::kMoveThreads, 0, cs, true, p))
    return ATTN_ERR_LAUNCH;
  return ATTN_OK;
}

}  // extern "C"
