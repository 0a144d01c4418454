// attn_rope.cu - host side of the per-head norms with rotation, declared in
// include/attn_fwd.h: checks the call and launches on the caller's stream.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "attn_fwd.h"
#include "attn_rope_kernel.cuh"
#include "host_common.h"
#include "rows.h"

namespace {

std::atomic<bool> g_launched{false};

}

namespace attn_host {

bool rope_take_status(unsigned int* s) { return take_status(attn::g_attn_status, g_launched, s); }

}  // namespace attn_host

namespace {

using namespace attn_host;
namespace rope = attn::rope;

constexpr int64_t kLim31 = (int64_t(1) << 31) - 1;
constexpr int64_t kFwdWarps = 48;  // an SM's, three times what it holds at once: with one wave and a half, 16384 tokens took 70 us for 66
constexpr int64_t kMaxHeads = 1 << 18;  // chunks of a token: a grid's y

// A dimension of one entry has no stride: what is given for it is not looked at (a batch of
// single tokens counts as tokens one batch stride apart).
RowSet row_set(const void* p, const int64_t* strides, int64_t B, int64_t S, int64_t H) {
  const int64_t batch = B > 1 ? strides[0] : 0;
  return {p, batch, S > 1 ? strides[1] : batch, H > 1 ? strides[2] : 0, B, S, H};
}

rope::Rows rows_of(const RowSet& r) {
  return {static_cast<uint16_t*>(const_cast<void*>(r.p)), r.batch, r.token, r.head};
}

struct Span {
  const void* p;
  uint64_t n;
};

// What the three entry points share.
struct Call {
  const void *q_weight, *k_weight, *cos, *sin;
  const int32_t* positions;
  int64_t B, S, Hq, Hkv, d, max_pos, rotary_dim;
  float eps;
  int mode, flags;
};

int check_call(const Call& c, const RowSet* tensors, int n) {
  if (!c.q_weight || !c.k_weight || !c.cos || !c.sin || !c.positions) return ATTN_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    if (!tensors[i].p) return ATTN_ERR_INVALID_ARG;
  if (c.B < 1 || c.S < 1 || c.Hq < 1 || c.Hkv < 1 || c.max_pos < 1) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(c.eps) || c.eps < 0) return ATTN_ERR_INVALID_ARG;
  if (c.d != attn::kD || c.rotary_dim < 16 || c.rotary_dim > c.d || c.rotary_dim % 16 != 0)
    return ATTN_ERR_UNSUPPORTED;
  if (c.flags & ~ATTN_FLAG_INTERLEAVED) return ATTN_ERR_UNSUPPORTED;
  if (c.mode < ATTN_ROUND_RTNE || c.mode > ATTN_ROUND_RTZ) return ATTN_ERR_UNSUPPORTED;
  if (c.B > kLim31 || c.S > kLim31 / c.B || c.Hq > kMaxHeads || c.Hkv > kMaxHeads || c.max_pos > kLim31)
    return ATTN_ERR_TOO_LARGE;
  for (int i = 0; i < n; ++i) {
    if (!strides_in_range(tensors[i])) return ATTN_ERR_INVALID_ARG;
    if (!extent_in_range(tensors[i])) return ATTN_ERR_TOO_LARGE;
  }
  for (int i = 0; i < n; ++i)
    if ((reinterpret_cast<uintptr_t>(tensors[i].p) & 15u) || !strides_aligned(tensors[i]))
      return ATTN_ERR_MISALIGNED;
  for (const void* p : {c.q_weight, c.k_weight, c.cos, c.sin})
    if (reinterpret_cast<uintptr_t>(p) & 15u) return ATTN_ERR_MISALIGNED;
  if (reinterpret_cast<uintptr_t>(c.positions) & 3u) return ATTN_ERR_MISALIGNED;
  return ATTN_OK;
}

// The dense inputs that no output may overlap.
void plain_inputs(const Call& c, Span (&s)[5]) {
  const uint64_t table = uint64_t(c.max_pos) * (c.rotary_dim / 2) * 4;
  s[0] = {c.q_weight, 256};
  s[1] = {c.k_weight, 256};
  s[2] = {c.cos, table};
  s[3] = {c.sin, table};
  s[4] = {c.positions, uint64_t(c.B) * c.S * 4};
}

uint64_t bytes_of(const RowSet& r) { return uint64_t(extent(r)) * r.elem; }

// Whether written tensor w overlaps a plain input or one of the row tensors (other than
// `same`, which may be w's own rows).
bool hits(const RowSet& w, const Span* plain, int n_plain, const RowSet* rows, int n_rows, int same) {
  for (int i = 0; i < n_plain; ++i)
    if (spans_meet(w.p, bytes_of(w), plain[i].p, plain[i].n)) return true;
  for (int i = 0; i < n_rows; ++i)
    if (rows_meet(w, rows[i]) && !(i == same && same_rows(w, rows[i]))) return true;
  return false;
}

void fill(rope::Params* p, const Call& c) {
  p->wq = static_cast<const uint16_t*>(c.q_weight);
  p->wk = static_cast<const uint16_t*>(c.k_weight);
  p->cos = static_cast<const float*>(c.cos);
  p->sin = static_cast<const float*>(c.sin);
  p->positions = c.positions;
  p->S = static_cast<int>(c.S);
  p->Hq = static_cast<int>(c.Hq);
  p->Hkv = static_cast<int>(c.Hkv);
  p->max_pos = static_cast<int>(c.max_pos);
  p->half = static_cast<int>(c.rotary_dim / 2);
  p->mode = c.mode;
  p->eps = c.eps;
  p->q_chunks = static_cast<int>((c.Hq + rope::kHeads - 1) / rope::kHeads);
  p->kv_chunks = static_cast<int>((c.Hkv + rope::kHeads - 1) / rope::kHeads);
  p->chunks = p->q_chunks + p->kv_chunks;
  p->tokens = static_cast<int>(c.B * c.S);
}

// Warps that share four tokens: as many as fill the GPU with `warps` of them, at most one a chunk.
int parts_of(int64_t tokens, int64_t chunks, int64_t warps) {
  const int64_t groups = (tokens + rope::kTokens - 1) / rope::kTokens, want = (warps + groups - 1) / groups;
  return static_cast<int>(want < chunks ? want : chunks);
}

rope::Form form_of(const Call& c) {
  if (c.flags & ATTN_FLAG_INTERLEAVED) return rope::kNext;
  return c.rotary_dim == attn::kD ? rope::kWhole : rope::kApart;
}

bool launch_fwd(rope::Params& p, bool paged, rope::Form form, void* stream) {
  using Kernel = void (*)(const rope::Params);
  static constexpr Kernel kFwd[3][2] = {
      {rope::attn_rope_fwd<rope::kWhole, false>, rope::attn_rope_fwd<rope::kWhole, true>},
      {rope::attn_rope_fwd<rope::kNext, false>, rope::attn_rope_fwd<rope::kNext, true>},
      {rope::attn_rope_fwd<rope::kApart, false>, rope::attn_rope_fwd<rope::kApart, true>}};
  p.parts = parts_of(p.tokens, p.chunks, kFwdWarps * int64_t(sms_here()));
  constexpr int64_t kBlock = rope::kWarps * rope::kTokens;
  const dim3 grid(static_cast<unsigned>((int64_t(p.tokens) + kBlock - 1) / kBlock), static_cast<unsigned>(p.parts));
  g_launched.store(true);
  return launch(kFwd[form][paged], grid, rope::kThreads, 0, static_cast<cudaStream_t>(stream), false, p);
}

struct BwdGrid {
  int64_t blocks;
  int parts;
};
BwdGrid bwd_grid(int64_t B, int64_t S, int64_t Hq, int64_t Hkv, int ctas) {
  const int64_t fill = ctas * int64_t(sms_here()), groups = (B * S + rope::kTokens - 1) / rope::kTokens;
  BwdGrid g;
  g.parts = parts_of(B * S, Hq + Hkv, fill * rope::kWarps);
  const int64_t need = (groups * g.parts + rope::kWarps - 1) / rope::kWarps;
  g.blocks = need < fill ? need : fill;
  return g;
}
// The form that has the most blocks.
int64_t bwd_bytes(int64_t B, int64_t S, int64_t Hq, int64_t Hkv) {
  int64_t most = 0;
  for (int ctas : {rope::kBwdCtas<rope::kWhole>, rope::kBwdCtas<rope::kApart>}) {
    const int64_t blocks = bwd_grid(B, S, Hq, Hkv, ctas).blocks;
    if (blocks > most) most = blocks;
  }
  return most * 2 * attn::kD * 4;
}

}  // namespace

extern "C" {

int attn_qk_norm_rope(const void* q, const void* k, const void* q_weight, const void* k_weight, const float* cos,
                      const float* sin, const int32_t* positions, void* q_out, void* k_out,
                      const int64_t* q_strides, const int64_t* k_strides, const int64_t* q_out_strides,
                      const int64_t* k_out_strides, int64_t B, int64_t S, int64_t Hq, int64_t Hkv, int64_t d,
                      int64_t max_pos, int64_t rotary_dim, float eps, int rounding_mode, int flags, void* stream) {
  if (!q_strides || !k_strides || !q_out_strides || !k_out_strides) return ATTN_ERR_INVALID_ARG;
  const Call c = {q_weight, k_weight, cos, sin, positions, B, S, Hq, Hkv, d, max_pos, rotary_dim, eps, rounding_mode,
                  flags};
  const RowSet t[] = {row_set(q, q_strides, B, S, Hq), row_set(k, k_strides, B, S, Hkv),
                      row_set(q_out, q_out_strides, B, S, Hq), row_set(k_out, k_out_strides, B, S, Hkv)};
  int st = check_call(c, t, 4);
  if (st != ATTN_OK) return st;
  Span plain[5];
  plain_inputs(c, plain);
  for (int w = 2; w < 4; ++w)
    if (!rows_distinct(t[w]) || hits(t[w], plain, 5, t, 2, w - 2)) return ATTN_ERR_ALIASING;
  if (rows_meet(t[2], t[3])) return ATTN_ERR_ALIASING;
  rope::Params p = {};
  fill(&p, c);
  st = arch_here();
  if (st != ATTN_OK) return st;
  p.q = rows_of(t[0]);
  p.k = rows_of(t[1]);
  p.q_out = rows_of(t[2]);
  p.k_out = rows_of(t[3]);
  return launch_fwd(p, false, form_of(c), stream) ? ATTN_OK : ATTN_ERR_LAUNCH;
}

int attn_qk_norm_rope_paged(const void* q, const void* k, const void* v, const void* q_weight, const void* k_weight,
                            const float* cos, const float* sin, const int32_t* positions, const int32_t* slots,
                            void* q_out, void* k_pages, void* v_pages, const int64_t* q_strides,
                            const int64_t* k_strides, const int64_t* v_strides, const int64_t* q_out_strides,
                            int layout, int64_t B, int64_t S, int64_t Hq, int64_t Hkv, int64_t n_pages,
                            int64_t page_size, int64_t page_stride, int64_t d, int64_t max_pos, int64_t rotary_dim,
                            float eps, int rounding_mode, int flags, void* stream) {
  if (!q_strides || !k_strides || !v_strides || !q_out_strides || !slots || !k_pages || !v_pages)
    return ATTN_ERR_INVALID_ARG;
  const Call c = {q_weight, k_weight, cos, sin, positions, B, S, Hq, Hkv, d, max_pos, rotary_dim, eps, rounding_mode,
                  flags};
  const RowSet t[] = {row_set(q, q_strides, B, S, Hq), row_set(k, k_strides, B, S, Hkv),
                      row_set(v, v_strides, B, S, Hkv), row_set(q_out, q_out_strides, B, S, Hq)};
  int st = check_call(c, t, 4);
  if (st != ATTN_OK) return st;
  if (layout != ATTN_LAYOUT_BHSD && layout != ATTN_LAYOUT_BSHD) return ATTN_ERR_UNSUPPORTED;
  st = check_pages(k_pages, v_pages, n_pages, page_size, page_stride, Hkv);
  if (st != ATTN_OK) return st;
  if (reinterpret_cast<uintptr_t>(slots) & 3u) return ATTN_ERR_MISALIGNED;
  Span plain[6];
  Span five[5];
  plain_inputs(c, five);
  for (int i = 0; i < 5; ++i) plain[i] = five[i];
  plain[5] = {slots, uint64_t(B) * S * 4};
  if (!rows_distinct(t[3]) || hits(t[3], plain, 6, t, 3, 0)) return ATTN_ERR_ALIASING;
  const PageSet kp = {k_pages, n_pages, page_stride, page_size * Hkv}, vp = {v_pages, n_pages, page_stride,
                                                                            page_size * Hkv};
  if (pages_meet(kp, vp)) return ATTN_ERR_ALIASING;
  for (const PageSet& w : {kp, vp}) {
    for (const Span& s : plain)
      if (spans_meet(w.p, w.bytes(), s.p, s.n)) return ATTN_ERR_ALIASING;
    for (const RowSet& r : t)
      if (spans_meet(w.p, w.bytes(), r.p, bytes_of(r))) return ATTN_ERR_ALIASING;
  }
  rope::Params p = {};
  fill(&p, c);
  p.chunks += p.kv_chunks;  // the values
  st = arch_here();
  if (st != ATTN_OK) return st;
  p.q = rows_of(t[0]);
  p.k = rows_of(t[1]);
  p.v = rows_of(t[2]);
  p.q_out = rows_of(t[3]);
  p.slots = slots;
  p.k_pages = static_cast<uint16_t*>(k_pages);
  p.v_pages = static_cast<uint16_t*>(v_pages);
  p.page_stride = page_stride;
  p.page_size = static_cast<int>(page_size);
  p.n_slots = static_cast<int>(n_pages * page_size);
  p.layout = layout;
  return launch_fwd(p, true, form_of(c), stream) ? ATTN_OK : ATTN_ERR_LAUNCH;
}

int64_t attn_qk_norm_rope_bwd_workspace_bytes(int64_t B, int64_t S, int64_t Hq, int64_t Hkv, int64_t d) {
  if (B < 1 || S < 1 || Hq < 1 || Hkv < 1) return ATTN_ERR_INVALID_ARG;
  if (d != attn::kD) return ATTN_ERR_UNSUPPORTED;
  if (B > kLim31 || S > kLim31 / B || Hq > kMaxHeads || Hkv > kMaxHeads) return ATTN_ERR_TOO_LARGE;
  return bwd_bytes(B, S, Hq, Hkv);
}

int attn_qk_norm_rope_bwd(const void* dq_out, const void* dk_out, const void* q, const void* k, const void* q_weight,
                          const void* k_weight, const float* cos, const float* sin, const int32_t* positions,
                          void* dq, void* dk, float* dq_weight, float* dk_weight, const int64_t* dq_out_strides,
                          const int64_t* dk_out_strides, const int64_t* q_strides, const int64_t* k_strides,
                          const int64_t* dq_strides, const int64_t* dk_strides, int64_t B, int64_t S, int64_t Hq,
                          int64_t Hkv, int64_t d, int64_t max_pos, int64_t rotary_dim, float eps, int rounding_mode,
                          int flags, void* workspace, int64_t workspace_bytes, void* stream) {
  if (!dq_out_strides || !dk_out_strides || !q_strides || !k_strides || !dq_strides || !dk_strides || !dq_weight ||
      !dk_weight || !workspace)
    return ATTN_ERR_INVALID_ARG;
  const Call c = {q_weight, k_weight, cos, sin, positions, B, S, Hq, Hkv, d, max_pos, rotary_dim, eps, rounding_mode,
                  flags};
  const RowSet t[] = {row_set(dq_out, dq_out_strides, B, S, Hq), row_set(dk_out, dk_out_strides, B, S, Hkv),
                      row_set(q, q_strides, B, S, Hq),           row_set(k, k_strides, B, S, Hkv),
                      row_set(dq, dq_strides, B, S, Hq),         row_set(dk, dk_strides, B, S, Hkv)};
  int st = check_call(c, t, 6);
  if (st != ATTN_OK) return st;
  const int64_t need = bwd_bytes(B, S, Hq, Hkv);
  if (workspace_bytes < need) return ATTN_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(workspace) & 15u) return ATTN_ERR_MISALIGNED;
  if ((reinterpret_cast<uintptr_t>(dq_weight) | reinterpret_cast<uintptr_t>(dk_weight)) & 3u)
    return ATTN_ERR_MISALIGNED;
  Span plain[5];
  plain_inputs(c, plain);
  for (int w = 4; w < 6; ++w)
    if (!rows_distinct(t[w]) || hits(t[w], plain, 5, t, 4, w - 4)) return ATTN_ERR_ALIASING;
  if (rows_meet(t[4], t[5])) return ATTN_ERR_ALIASING;
  const Span more[] = {{dq_weight, 512}, {dk_weight, 512}, {workspace, uint64_t(need)}};
  for (int i = 0; i < 3; ++i) {
    for (const Span& s : plain)
      if (spans_meet(more[i].p, more[i].n, s.p, s.n)) return ATTN_ERR_ALIASING;
    for (const RowSet& r : t)
      if (spans_meet(more[i].p, more[i].n, r.p, bytes_of(r))) return ATTN_ERR_ALIASING;
    for (int j = 0; j < i; ++j)
      if (spans_meet(more[i].p, more[i].n, more[j].p, more[j].n)) return ATTN_ERR_ALIASING;
  }
  st = arch_here();
  if (st != ATTN_OK) return st;
  rope::BwdParams p = {};
  fill(&p.f, c);
  p.dq_out = rows_of(t[0]);
  p.dk_out = rows_of(t[1]);
  p.f.q = rows_of(t[2]);
  p.f.k = rows_of(t[3]);
  p.dq = rows_of(t[4]);
  p.dk = rows_of(t[5]);
  const rope::Form form = form_of(c);
  const BwdGrid grid = bwd_grid(B, S, Hq, Hkv, form == rope::kWhole ? rope::kBwdCtas<rope::kWhole>
                                                                    : rope::kBwdCtas<rope::kApart>);
  p.f.parts = grid.parts;
  p.part = static_cast<float*>(workspace);
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const auto fn = form == rope::kWhole  ? rope::attn_rope_bwd<rope::kWhole>
                  : form == rope::kNext ? rope::attn_rope_bwd<rope::kNext>
                                        : rope::attn_rope_bwd<rope::kApart>;
  g_launched.store(true);
  if (!launch(fn, grid.blocks, rope::kThreads, rope::kBwdSmem, cs, false, p)) return ATTN_ERR_LAUNCH;
  const rope::JoinParams j = {p.part, dq_weight, dk_weight, static_cast<int>(grid.blocks)};
  return launch(rope::attn_rope_join, 2 * attn::kD / rope::kJoinCols, rope::kJoinThreads, 0, cs, true, j)
             ? ATTN_OK
             : ATTN_ERR_LAUNCH;
}

}  // extern "C"
