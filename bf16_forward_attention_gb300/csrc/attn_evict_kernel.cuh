// attn_evict_kernel.cuh - a paged cache kept to a budget: of each (sequence, kv head), the keys of
// greatest accumulated attention weight and the latest ones, moved together in order.
//
// Three steps on the stream: attn_evict_select finds, for each (sequence, kv head), which keys
// stay (their places in ascending order, with their masses), and counts how often each page is
// listed; attn_evict_move moves them to the first places. Kept keys move towards the front, so a
// round of moves reads everything it moves before it writes (a barrier of the cluster between
// the two), and later rounds read places that no earlier one wrote: place d takes key src[d] >= d,
// and a later round's keys lie behind all of this round's.
#pragma once
#include "few_rows.cuh"

namespace attn {
namespace evict {

struct Params {
  uint16_t* k;             // pages
  uint16_t* v;
  const int* table;        // (B, max_pages)
  const int* seqlens;
  const float* mass;       // (B, Hkv, cap)
  float* mass_out;         // may be mass
  int* seqlens_out;        // may be seqlens
  int* listed;             // [page]: how often the sequences list it; zeros at the start
  int2* head;              // [b * Hkv + kvh]: length (or -1: leave the sequence), first place that moves
  int* src;                // [b * Hkv + kvh][keep]: the kept keys of a sequence over its budget, ascending
  float* src_mass;         // their masses
  int page_rows;           // rows of 128 from a page to the next
  int B, Hkv, cap, layout, n_pages, page_size, page_shift, max_pages;
  uint32_t page_mul;       // with page_shift: see page_divisor
  int budget, recent, keep;  // keep: min(budget, cap)
};

// Masses in an order of unsigned integers: greater is greater, -0 is 0, and NaN is above all.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t u = __float_as_uint(x);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
  if ((u & 0x7FFFFFFFu) == 0) return 0x80000000u;
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

// A warp's stretch of the masses, lo .. hi - 1, 32 at a time: the first kHeld of a lane stay in its
// registers from pass to pass, the others are read again, kBatch on their way at once.
constexpr int kHeld = 32, kBatch = 8;
struct Stretch {
  const float* mass;
  int lo, hi, lane;
  float held[kHeld];

  __device__ __forceinline__ void load() {
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      const int i = lo + 32 * j + lane;
      held[j] = i < hi ? __ldg(mass + i) : 0.f;
    }
  }
  // fn(whether there is one, place, mass) for 32 places at a time, in order.
  template <typename Fn>
  __device__ __forceinline__ void each(Fn&& fn) const {
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      if (lo + 32 * j >= hi) break;  // the same for all lanes
      const int i = lo + 32 * j + lane;
      fn(i < hi, i, held[j]);
    }
    for (int base = lo + 32 * kHeld; base < hi; base += 32 * kBatch) {
      float x[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int i = base + 32 * j + lane;
        x[j] = i < hi ? __ldg(mass + i) : 0.f;
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (base + 32 * j >= hi) break;
        const int i = base + 32 * j + lane;
        fn(i < hi, i, x[j]);
      }
    }
  }
};

// ---------------------------------------------------------------- select
constexpr int kSelectWarps = 16;
constexpr int kSelectThreads = 32 * kSelectWarps;
constexpr int kBins = 2048;

// One block per (sequence, kv head). The m-th greatest of the masses of the keys that are not
// among the latest, by its digits of 11, 11 and 10 bits from the top: a histogram of a digit among the
// masses that share the digits above it. Then every warp counts, in its stretch of the keys,
// those above that value and those equal to it, and writes its kept keys behind the others';
// of the equal ones the first stay. A block's first 16384 masses are read once (read in each of
// the five passes, 256 blocks of up to 16384 keys took 27 us for 24).
__global__ void __launch_bounds__(kSelectThreads, 2) attn_evict_select(const Params p) {
  __shared__ __align__(16) int bins[kBins];
  __shared__ int warp_n[2][kSelectWarps];
  // The sum of the warps' entries before this one's.
  auto before_warp = [&](const int (&n)[kSelectWarps], int warp, int lane) {
    return static_cast<int>(__reduce_add_sync(0xFFFFFFFFu, lane < warp ? static_cast<unsigned>(n[lane & (kSelectWarps - 1)]) : 0u));
  };
  __shared__ int found, rest, first_move;
  const int b = blockIdx.x / p.Hkv, kvh = blockIdx.x - b * p.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = __ldg(p.seqlens + b);
  const int pages = len < 0 || len > p.cap ? 0 : (len + p.page_size - 1) / p.page_size;
  bool bad = false;
  for (int i = threadIdx.x; i < pages; i += kSelectThreads) {
    const int id = __ldg(p.table + static_cast<size_t>(b) * p.max_pages + i);
    if (id < 0 || id >= p.n_pages)
      bad = true;
    else if (kvh == 0)
      atomicAdd(p.listed + id, 1);
  }
  if (threadIdx.x == 0) first_move = p.keep;
  bad = __syncthreads_or(bad);
  if (bad || len < 0 || len > p.cap) {
    if (threadIdx.x == 0) {
      p.head[blockIdx.x] = make_int2(-1, 0);
      if (kvh == 0) atomicOr(&g_attn_status, bad ? 8u : 2u);
    }
    return;
  }
  if (len <= p.budget) {
    if (threadIdx.x == 0) p.head[blockIdx.x] = make_int2(len, p.keep);
    return;
  }
  const float* mass = p.mass + static_cast<size_t>(blockIdx.x) * p.cap;
  const int old = len - p.recent;   // more than m
  int m = p.budget - p.recent;      // how many of them stay
  const int each = ((old + kSelectWarps - 1) / kSelectWarps + 31) & ~31;  // of a warp; old is at least 1
  Stretch stretch = {mass, min(old, warp * each), min(old, (warp + 1) * each), lane, {}};
  stretch.load();
  uint32_t above = 0;               // the value's digits so far
  int shift = 32;
#pragma unroll 1
  for (int pass = 0; pass < 3 && m > 0; ++pass) {
    const int width = pass < 2 ? 11 : 10;
    const uint32_t high = pass == 0 ? 0u : 0xFFFFFFFFu << shift;
    shift -= width;
    static_assert(kBins == 4 * kSelectThreads, "four bins a thread");
    reinterpret_cast<int4*>(bins)[threadIdx.x] = make_int4(0, 0, 0, 0);
    __syncthreads();
    stretch.each([&](bool valid, int, float value) {
      const uint32_t x = order_of(value);
      if (valid && (x & high) == above) atomicAdd(&bins[(x >> shift) & ((1 << width) - 1)], 1);
    });
    __syncthreads();
    // From the top bin down: the one in which the m-th lies. Thread t has bins 4 t .. 4 t + 3 from
    // the top.
    const int4 four = reinterpret_cast<const int4*>(bins)[kSelectThreads - 1 - threadIdx.x];
    const int mine[4] = {four.w, four.z, four.y, four.x}, sum = (four.x + four.y) + (four.z + four.w);
    int upto = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(0xFFFFFFFFu, upto, d);
      if (lane >= d) upto += x;
    }
    if (lane == 31) warp_n[0][warp] = upto;
    __syncthreads();
    int before = upto - sum + before_warp(warp_n[0], warp, lane);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (before < m && m <= before + mine[j]) {
        found = kBins - 1 - (4 * static_cast<int>(threadIdx.x) + j);
        rest = m - before;
      }
      before += mine[j];
    }
    __syncthreads();
    above |= static_cast<uint32_t>(found) << shift;
    m = rest;
    __syncthreads();
  }
  // Above `above` all stay, of those equal to it the first m. With none of the old to stay, none do.
  const bool none = p.budget == p.recent;
  int more = 0, equal = 0;
  if (!none) {
    stretch.each([&](bool valid, int, float value) {
      const uint32_t x = order_of(value);
      more += valid && x > above;
      equal += valid && x == above;
    });
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      more += __shfl_xor_sync(0xFFFFFFFFu, more, d);
      equal += __shfl_xor_sync(0xFFFFFFFFu, equal, d);
    }
  }
  if (lane == 0) {
    warp_n[0][warp] = more;
    warp_n[1][warp] = equal;
  }
  __syncthreads();
  int n_more = before_warp(warp_n[0], warp, lane), n_equal = before_warp(warp_n[1], warp, lane);  // before the key at hand
  int* src = p.src + static_cast<size_t>(blockIdx.x) * p.keep;
  float* src_mass = p.src_mass + static_cast<size_t>(blockIdx.x) * p.keep;
  auto put = [&](int d, int i, float value) {
    if (!dbg_ok(d >= 0 && d < p.keep && d <= i)) return;
    src[d] = i;
    src_mass[d] = value;
  };
  // Keys before the first that goes stay where they are; the next kept one takes its place.
  int first_gone = none ? 0 : p.keep;
  if (!none) {
    const uint32_t below = (1u << lane) - 1;
    stretch.each([&](bool valid, int i, float value) {
      const uint32_t x = order_of(value);
      const uint32_t is_more = __ballot_sync(0xFFFFFFFFu, valid && x > above);
      const uint32_t is_equal = __ballot_sync(0xFFFFFFFFu, valid && x == above);
      const int eq = n_equal + __popc(is_equal & below);  // equal ones before this one
      if (valid) {
        if (x > above || (x == above && eq < m))
          put(n_more + __popc(is_more & below) + min(eq, m), i, value);
        else
          first_gone = min(first_gone, i);
      }
      n_more += __popc(is_more);
      n_equal += __popc(is_equal);
    });
  }
  for (int i = threadIdx.x; i < p.recent; i += kSelectThreads) put(p.budget - p.recent + i, old + i, mass[old + i]);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) first_gone = min(first_gone, __shfl_xor_sync(0xFFFFFFFFu, first_gone, d));
  if (lane == 0) atomicMin(&first_move, first_gone);
  __syncthreads();
  if (threadIdx.x == 0) p.head[blockIdx.x] = make_int2(len, first_move);
}

// ---------------------------------------------------------------- move
constexpr int kCluster = 8;        // CTAs of a (sequence, kv head)
constexpr int kMoveThreads = 256;
constexpr int kMoveKeys = 4;       // keys a half-warp moves at once: 8 loads of 16 bytes a lane in flight
constexpr int kMoveRound = kMoveThreads / 16 * kMoveKeys;  // keys of a CTA's round

// The rounds of a (sequence, kv head): 512 keys over its cluster, read, a barrier, written.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kMoveThreads, 4) attn_evict_move(const Params p) {
  const int rank = static_cast<int>(ptx::cluster_ctarank());
  const int item = blockIdx.x / kCluster, b = item / p.Hkv, kvh = item - b * p.Hkv;
  ptx::grid_dependency_wait();
  const int2 head = p.head[item];
  const int len = head.x;
  if (len < 0) return;  // the whole cluster
  const int* pages = p.table + static_cast<size_t>(b) * p.max_pages;
  const bool over = len > p.budget;
  if (over) {
    // A page that is listed twice would be written by two sequences, or read after it was written.
    bool twice = false;
    const int n = (len + p.page_size - 1) / p.page_size;
    for (int i = threadIdx.x; i < n; i += kMoveThreads) twice = twice || p.listed[__ldg(pages + i)] != 1;
    if (__syncthreads_or(twice)) {  // every CTA of the cluster, and every head, finds the same
      if (threadIdx.x == 0 && rank == 0 && kvh == 0) atomicOr(&g_attn_status, 8u);
      return;
    }
  }
  const int left = over ? p.budget : len;
  const size_t row = static_cast<size_t>(item) * p.cap, list = static_cast<size_t>(item) * p.keep;
  for (int j = rank * kMoveThreads + threadIdx.x; j < p.cap; j += kCluster * kMoveThreads)
    p.mass_out[row + j] = j >= left ? 0.f : over ? p.src_mass[list + j] : p.mass[row + j];
  if (threadIdx.x == 0 && rank == 0 && kvh == 0) p.seqlens_out[b] = left;
  if (!over) return;
  const int half = threadIdx.x >> 4, chunk = threadIdx.x & 15;
  auto row_of = [&](int key) {  // of 128, in the pages
    const int page = few::page_of(key, p.page_mul, p.page_shift), i = key - page * p.page_size;
    return __ldg(pages + page) * p.page_rows + (p.layout == 0 ? kvh * p.page_size + i : i * p.Hkv + kvh);
  };
  auto at = [&](uint16_t* t, int row) { return reinterpret_cast<uint4*>(t + static_cast<size_t>(row) * kD) + chunk; };
  // Rows that a round reads and writes (-1: none), looked up while the round before is under way.
  int from[kMoveKeys], to[kMoveKeys];
  auto look_up = [&](int base) {
    const int d0 = base + rank * kMoveRound + half * kMoveKeys;
#pragma unroll
    for (int i = 0; i < kMoveKeys; ++i) {
      const int key = d0 + i < left ? p.src[list + d0 + i] : -1;
      const bool moves = key >= 0 && dbg_ok(key > d0 + i && key < len);
      from[i] = moves ? row_of(key) : -1;
      to[i] = moves ? row_of(d0 + i) : -1;
    }
  };
  look_up(head.y);
  for (int base = head.y; base < left; base += kCluster * kMoveRound) {
    uint4 k[kMoveKeys], v[kMoveKeys];
    int dst[kMoveKeys];
#pragma unroll
    for (int i = 0; i < kMoveKeys; ++i) {
      dst[i] = to[i];
      if (from[i] >= 0) {
        k[i] = __ldcg(at(p.k, from[i]));
        v[i] = __ldcg(at(p.v, from[i]));
      }
    }
    look_up(base + kCluster * kMoveRound);
    __syncwarp();
    ptx::cluster_sync();
#pragma unroll
    for (int i = 0; i < kMoveKeys; ++i) {
      if (dst[i] >= 0) {
        *at(p.k, dst[i]) = k[i];
        *at(p.v, dst[i]) = v[i];
      }
    }
    __syncwarp();
  }
}

}  // namespace evict
}  // namespace attn
