// rows.h - (B, S, H, 128) tensors wherever their rows of 128 lie: checks of element strides
// on the host. No CUDA, so that they are tested on the CPU too.
#pragma once
#include <cstdint>

namespace attn_host {

struct RowSet {
  const void* p;
  int64_t batch, token, head;  // element strides
  int64_t B, S, H;
  int64_t elem = 2;            // bytes an element
};

constexpr int64_t kRowElems = 128;

// Strides that the kernels' 64-bit offsets hold: not negative, below 2^40, and rows on
// 16-byte boundaries.
inline bool strides_in_range(const RowSet& r) {
  for (int64_t s : {r.batch, r.token, r.head})
    if (s < 0 || s >= (int64_t(1) << 40)) return false;
  return true;
}
inline bool strides_aligned(const RowSet& r) { return ((r.batch | r.token | r.head) * r.elem) % 16 == 0; }

// Elements from the first row's start to the last row's end. Sizes are at most 2^31 - 1 and
// strides below 2^40, so a tensor within 2^62 elements does not wrap.
inline int64_t extent(const RowSet& r) {
  return (r.B - 1) * r.batch + (r.S - 1) * r.token + (r.H - 1) * r.head + kRowElems;
}
inline bool extent_in_range(const RowSet& r) {
  const int64_t most = int64_t(1) << 50;
  int64_t sum = kRowElems;
  const int64_t n[3] = {r.B, r.S, r.H}, s[3] = {r.batch, r.token, r.head};
  for (int i = 0; i < 3; ++i) {
    if (s[i] && n[i] - 1 > most / s[i]) return false;
    sum += (n[i] - 1) * s[i];
    if (sum > most) return false;
  }
  return true;
}

// No two rows of the tensor share an element: from the smallest stride up, each is at least
// what the dimensions below it span. (Sufficient; a tensor to write needs it.)
inline bool rows_distinct(const RowSet& r) {
  int64_t n[3] = {r.B, r.S, r.H}, s[3] = {r.batch, r.token, r.head};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (s[j] < s[i]) {
        const int64_t a = s[i], b = n[i];
        s[i] = s[j], n[i] = n[j];
        s[j] = a, n[j] = b;
      }
  int64_t span = kRowElems;
  for (int i = 0; i < 3; ++i) {
    if (n[i] == 1) continue;
    if (s[i] < span) return false;
    span = (n[i] - 1) * s[i] + span;
  }
  return true;
}

inline bool spans_meet(const void* a, uint64_t na, const void* b, uint64_t nb) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + nb && b0 < a0 + na;
}

// Blocks of `wa` bytes every `stride` from a, and of `wb` bytes from b: whether some may meet.
// Exact for endless runs of blocks with wa, wb <= stride (the columns of one wider row).
inline bool columns_meet(const void* a, int64_t wa, const void* b, int64_t wb, int64_t stride) {
  const int64_t off = static_cast<int64_t>(
      (reinterpret_cast<uintptr_t>(b) % stride + stride - reinterpret_cast<uintptr_t>(a) % stride) % stride);
  return off < wa || off + wb > stride;
}

// Whether two tensors may share an element. Those whose spans meet are told apart where they
// are columns of the same tokens (views of one projection's output): equal batch and token
// strides, each token's heads within a token's stride.
inline bool rows_meet(const RowSet& a, const RowSet& b) {
  if (!spans_meet(a.p, extent(a) * a.elem, b.p, extent(b) * b.elem)) return false;
  const int64_t wa = (a.H - 1) * a.head + kRowElems, wb = (b.H - 1) * b.head + kRowElems;
  const bool one_grid = a.elem == b.elem && a.B == b.B && a.S == b.S && a.token == b.token && wa <= a.token &&
                        wb <= b.token && (a.B == 1 || (a.batch == b.batch && a.batch % a.token == 0));
  return !one_grid || columns_meet(a.p, wa * a.elem, b.p, wb * b.elem, a.token * a.elem);
}

inline bool same_rows(const RowSet& a, const RowSet& b) {
  return a.p == b.p && a.B == b.B && a.S == b.S && a.H == b.H && (a.B == 1 || a.batch == b.batch) &&
         (a.S == 1 || a.token == b.token) && (a.H == 1 || a.head == b.head);
}

// Pages of a cache: n blocks of rows * 128 elements, `stride` elements apart.
struct PageSet {
  const void* p;
  int64_t n, stride, rows;
  int64_t bytes() const { return ((n - 1) * stride + rows * kRowElems) * 2; }
};

// Whether two page sets of the same form (keys and values) may share an element: two tensors,
// or the two halves of every page of one.
inline bool pages_meet(const PageSet& a, const PageSet& b) {
  if (!spans_meet(a.p, a.bytes(), b.p, b.bytes())) return false;
  return a.n == 1 || columns_meet(a.p, a.rows * kRowElems * 2, b.p, b.rows * kRowElems * 2, a.stride * 2);
}

// What the kernels ask of a cache: pages that do not overlap, on 16-byte boundaries (rows on
// 256-byte steps from the first), all rows numbered within 31 bits.
inline bool pages_in_range(int64_t n_pages, int64_t page_size, int64_t page_stride, int64_t Hkv) {
  const int64_t lim = (int64_t(1) << 31) - 1;
  if (page_size > lim / Hkv || page_stride / kRowElems > lim / n_pages) return false;
  return page_size <= lim / n_pages;
}

// key / page_size for 0 <= key < 2^31 as a multiplication (Granlund and Montgomery, "Division by
// invariant integers using multiplication", 1994): with 2^(l-1) < page_size <= 2^l and mul =
// ceil(2^(31+l) / page_size), which is below 2^32, it is key * mul / 2^(31+l), rounded down. The kernels
// take the upper 32 bits of the product and shift them by l - 1; a page size of 1 (l = 0) has shift -1.
struct PageDivisor {
  uint32_t mul;
  int shift;
};
inline PageDivisor page_divisor(int64_t page_size) {
  int l = 0;
  while ((int64_t(1) << l) < page_size) ++l;
  const uint64_t n = uint64_t(1) << (31 + l), q = n / uint64_t(page_size) + (n % uint64_t(page_size) != 0);
  return {static_cast<uint32_t>(q), l - 1};
}
inline int64_t page_of(int64_t key, PageDivisor d) {
  return d.shift < 0 ? key : static_cast<int64_t>((uint64_t(key) * d.mul) >> 32 >> d.shift);
}

}  // namespace attn_host
