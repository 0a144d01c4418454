// attn_bwd_kernel.cuh - backward pass of bf16 attention for sm_103a (GB300).
//
// With s_ij = scale q_i.k_j, lse_i = ln sum_j exp(s_ij) (left by the forward pass)
// and the output's gradient dO, over the pairs that are not hidden:
//   P_ij  = exp(s_ij - lse_i)           recomputed, never stored in global memory
//   D_i   = sum_c dO_ic O_ic            (= sum_j P_ij dP_ij)
//   dP    = dO V^T        dS = P o (dP - D)
//   dV    = P^T dO        dK = scale dS^T Q        dQ = scale dS K
// dK and dV of a key/value head sum over the query heads that share it.
//
// Why two kernels. dK and dV sum over query rows, dQ over keys. One kernel that
// forms P and dS once (5 products per tile pair) has to add either dQ or dK/dV
// across CTAs: with atomics, whose order changes the bits from run to run, or
// with CTAs that wait on one another. Here each result has one owner and a
// fixed order of summation: attn_bwd_dkv owns 128 keys and streams query tiles
// (4 products), attn_bwd_dq owns 128 queries and streams key tiles (3 products),
// S and dP being formed twice: 7 products of 128 x 128 x 128 per tile pair.
// In exchange P and dS never leave tensor memory (they are the A operands of the
// second products, in the lanes where the softmax threads write them), nothing is
// accumulated in global memory, and no atomic touches a result.
//
// Precision. S, dP and all sums are fp32. P and dS are rounded once to bf16 as
// operands of the second products, like their partners dO, Q and K; the rounding
// errors (at most 2^-8 relative, independent from pair to pair) reach a gradient with
// about the weight of its own rounding to bf16, so a second term as in the forward
// kernel's P (which has to hold every output to one unit in the last place) would
// cost 3 more products for less than a factor of 2 in the final error.
// The tensor pipe's fp32 accumulation truncates, a bias that grows with the number of
// products in one accumulator: dV over 8192 tiles (131072 queries of 8 heads, dO of mean
// 1) came out 0.63% small, more than its rounding to bf16. So an accumulator takes
// kAccTiles streamed tiles at most (0.02% there); the softmax threads then add it, rounded to
// nearest, to the item's fp32 terms in the workspace, and the next one starts anew (that
// call: 18.5 -> 19.1 ms; shorter items are as they were).
//
// Both kernels: 384 threads. Warp 0: TMA producer. Warp 1: TMEM allocation and
// the tcgen05.mma issue (one elected lane, in warp-uniform code). Warps 2-3: check of the
// tiles where some pairs are hidden. Warps 4-7 and 8-11: softmax, each thread one TMEM
// lane (a key in dkv, a query in dq) and one 64-column half.
// A CTA works on one item (an owned tile, or a part of its streamed range) after another:
// it takes over CTAs of its grid that have not been launched yet (cluster launch
// control), in launch order, so the schedule is the hardware's dynamic one, longest
// items first, while barriers, tensor memory and the rings live on, the next item's loads
// start when the last products of this one have read their tiles, and a result is stored
// while the next item's first products run. (One item per CTA cost 11,000 cycles around
// each item's loop.) Every wait is bounded, as in the forward kernel.
#pragma once
#include "attn_fwd_kernel.cuh"

namespace attn {
namespace bwd {

constexpr int kTile = 128;             // queries and keys per tile
constexpr int kStatFloats = 2 * kTile; // per query tile: 128 of -lse log2(e), 128 of -D
constexpr int kAccTiles = 256;         // streamed tiles summed in one tensor-memory accumulator
static_assert((kAccTiles & (kAccTiles - 1)) == 0, "used as a mask");

// Accumulators that n streamed tiles take. Kernels are instantiated for calls whose items may
// take several (kLong) and for the others: the loop and the reads of the terms so far cost
// a call of a few tiles 3 to 7% (256 tokens: 12.9 -> 13.9 us).
template <bool kLong>
__device__ __forceinline__ int accumulators(int n) {
  return kLong ? (n + kAccTiles - 1) / kAccTiles : n > 0;
}

// Division of n in [0, 2^31) by a number fixed for a launch, as a product (Granlund and
// Montgomery, "Division by invariant integers using multiplication"): with 2^(s+1) >= d and
// mul = ceil(2^(32+s) / d), n * mul exceeds n 2^(32+s) / d by less than 2^(32+s) / d. An item's
// place takes five divisions, some 500 cycles otherwise.
struct Div {
  uint32_t mul;
  int shift, d;
  __host__ static Div by(int64_t d) {
    Div r;
    r.d = static_cast<int>(d);
    r.shift = 0;
    while ((int64_t(2) << r.shift) < d) ++r.shift;
    r.mul = static_cast<uint32_t>(((uint64_t(1) << (32 + r.shift)) + d - 1) / d);  // (d = 1: not used)
    return r;
  }
  __device__ __forceinline__ int of(int n) const {
    return d == 1 ? n : static_cast<int>(__umulhi(static_cast<uint32_t>(n), mul) >> shift);
  }
};

struct BwdParams {
  int Sq, Sk;              // per batch entry, or packed totals
  int Hq, Hkv, group;      // group = Hq / Hkv
  int BH;                  // heads of the grid: B * Hq (dq) or B * Hkv (dkv)
  int n_tiles;             // tiles of the owned axis per head (grid)
  int n_splits;            // items per owned tile, each over a part of the streamed tiles
  // An item's place: heads are scheduled together in n_groups groups (causal: longest
  // first), of heads.d heads each, the last one of last.d.
  int n_groups;
  Div splits, span, heads, last, owners;  // span = n_tiles * heads.d, owners = heads of the owned axis
  int layout, mode;
  float c, scale;          // c = scale * log2(e)
  unsigned long long timeout_ns;
  int withhold;            // self-test: the first S is waited for once more than it is announced
  const int* cu_q;         // packed batch: B + 1 offsets each (else null)
  const int* cu_k;
  int max_sq, max_sk;
  int q_slots, k_slots;    // tile slots per head (see tile_slot)
  const float* lse;
  float* stats;            // [head][slot][2][128]: written by dq, read by dkv
  // Tiles of fp32 terms, [split][result][head * slots]: of results shared by n_splits > 1
  // items, and of items of more than kAccTiles streamed tiles.
  float* part;
  uint16_t *dq, *dk, *dv;  // results
};

// Tile slots: a dense head has ceil(S / 128) tiles. A packed batch has no host copy
// of its offsets, so sequence b's tiles start at slot off/128 + b of its head:
// since floor(x + y) >= floor(x) + floor(y), the next sequence's start is never
// below this one's end, and total/128 + B + 1 slots hold them all.
template <bool kVarlen>
__device__ __forceinline__ int tile_slot(int base, int b) {
  return kVarlen ? (base >> 7) + b : 0;
}

// One CTA's sequence, head and range.
struct Seq {
  int head;          // head of the owned axis (query head or key/value head)
  int batch;         // TMA batch coordinate (0 for a packed batch)
  int q_base, k_base, sq, sk;
  int slot_q, slot_k;  // slot of the sequence's first query / key tile, head included
  int tile, split;
  bool bad;
};

template <bool kCausal, bool kVarlen, bool kOwnQ>
__device__ __forceinline__ Seq seq_of(const BwdParams& p, int block) {
  Seq s;
  const int item = p.splits.of(block);
  s.split = block - item * p.n_splits;
  const int g = p.span.of(item), r = item - g * p.span.d;
  const bool last = g == p.n_groups - 1;
  const int t = last ? p.last.of(r) : p.heads.of(r);
  const int bh = g * p.heads.d + r - t * (last ? p.last.d : p.heads.d);
  // Longest ranges first under the causal mask: late queries see most keys, early
  // keys are seen by most queries.
  s.tile = (kOwnQ && kCausal) ? p.n_tiles - 1 - t : t;
  const int b = p.owners.of(bh);
  s.head = bh - b * p.owners.d;
  s.bad = false;
  if (kVarlen) {
    s.q_base = __ldg(p.cu_q + b);
    s.sq = packed_len(s.q_base, __ldg(p.cu_q + b + 1), p.max_sq, p.Sq);
    s.k_base = __ldg(p.cu_k + b);
    s.sk = packed_len(s.k_base, __ldg(p.cu_k + b + 1), p.max_sk, p.Sk);
    s.bad = s.sq < 0 || s.sk < 0;
    s.batch = 0;
    s.slot_q = tile_slot<true>(s.q_base, b);  // the head's offset is added by the user
    s.slot_k = tile_slot<true>(s.k_base, b);
  } else {
    s.q_base = s.k_base = 0;
    s.sq = p.Sq;
    s.sk = p.Sk;
    s.batch = b;
    s.slot_q = b * p.Hq * p.q_slots;
    s.slot_k = b * p.Hkv * p.k_slots;
  }
  return s;
}

// The items of a CTA, in order, for its warps: item 0 is the CTA's own number, and answer
// `it` names item it + 1. The producer asks when it has issued an item's last loads, a few
// tiles before its end: an item claimed earlier would wait for this CTA while others run
// out of work (asked one item earlier, a packed batch took 986 us instead of 900, and
// where there are many equal items nothing was won). Per slot an answer (16 bytes), a barrier
// for it and one for its readers.
constexpr int kItemSlots = 2;
struct Items {
  uint32_t resp, full, empty;  // shared-memory addresses of slot 0
  volatile int* abort_flag;
  unsigned long long timeout_ns;

  // By the producer's lane.
  __device__ __forceinline__ void ask(int it) const {
    const uint32_t slot = it % kItemSlots;
    if (!wait_bounded(empty + 8 * slot, ((it / kItemSlots) & 1) ^ 1, abort_flag, timeout_ns, true)) return;
    ptx::mbar_arrive_expect_tx(full + 8 * slot, 16);
    ptx::clc_try_cancel(resp + 16 * slot, full + 8 * slot);
  }
  // By one lane of a role: the item after item `it`, -1 at the end.
  __device__ __forceinline__ int next_lane(int it) const {
    const uint32_t slot = it % kItemSlots;
    if (!wait_bounded(full + 8 * slot, (it / kItemSlots) & 1, abort_flag, timeout_ns, true)) return -1;
    const int item = ptx::clc_answer(resp + 16 * slot);
    ptx::fence_proxy_async_smem();  // the read, before the slot's next answer
    ptx::mbar_arrive(empty + 8 * slot);
    return item;
  }
  // By a whole warp.
  __device__ __forceinline__ int next_warp(int it, int lane) const {
    const uint32_t slot = it % kItemSlots;
    if (!warp_wait(full + 8 * slot, (it / kItemSlots) & 1, abort_flag, timeout_ns)) return -1;
    const int item = ptx::clc_answer(resp + 16 * slot);
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(empty + 8 * slot);
    return __shfl_sync(0xFFFFFFFFu, item, 0);
  }
  // The answers asked for and not taken have landed (before the CTA exits).
  __device__ __forceinline__ void drain(int asked) const {
    for (int it = asked > kItemSlots ? asked - kItemSlots : 0; it < asked; ++it)
      wait_bounded(full + 8 * (it % kItemSlots), (it / kItemSlots) & 1, abort_flag, timeout_ns, false);
  }
};
// Readers of an answer: producer, MMA warp, softmax warps, and the check's.
__host__ __device__ constexpr int item_readers(bool check) { return 10 + (check ? 2 : 0); }

// The next item for warps 2 and 3, which meet at named barriers: -1 for both if it is for one.
__device__ __forceinline__ int next_together(const Items& items, int it, int lane) {
  const int item = items.next_warp(it, lane);
  return ptx::named_barrier_or(1, 64, item < 0) ? -1 : item;
}

// Part `split` of n streamed tiles: [first, first + count).
__device__ __forceinline__ void part_of(int n, int splits, int split, int& first, int& count) {
  const int base = n / splits, rem = n % splits;
  first = split * base + min(split, rem);
  count = base + (split < rem ? 1 : 0);
}

// 64 columns of a TMEM row as 32 packed pairs of fp32.
using Half = uint64_t[32];

// Runs half(ch, r) on the 32-column halves of a 64-column TMEM row: the second is loaded
// while the first is worked on.
template <typename F>
__device__ __forceinline__ void by_halves(uint32_t taddr, F half) {
  uint32_t a[32], b[32];
  ptx::tmem_ld32_nowait(taddr, a);
  ptx::tmem_wait_ld32(a);
  ptx::tmem_ld32_nowait(taddr + 32, b);
  half(0, a);
  ptx::tmem_wait_ld32(b);
  half(1, b);
}

// acc += A[tmem: 128 x 128 bf16] * B[smem, MN-major]: 8 MMAs of K = 16. A's columns
// 0..63 sit packed at tmem_a, columns 64..127 at tmem_a + 64 (each softmax
// warpgroup writes its half over the first half of the columns that it read).
template <int... kK>
__device__ __forceinline__ void issue_second_seq(uint32_t tmem_d, uint32_t tmem_a, uint32_t b_lo,
                                                 uint32_t accumulate,
                                                 std::integer_sequence<int, kK...>) {
  constexpr uint32_t idesc = idesc_bf16(kTile, kD, 1);
  (ptx::mma_ts_warp<(kK < 4 ? 8 * kK : 64 + 8 * (kK - 4)), (kK << 7)>(
       tmem_d, tmem_a, b_lo, kDescHi, idesc, kK == 0 ? accumulate : 1u),
   ...);
}
__device__ __forceinline__ void issue_second(uint32_t tmem_d, uint32_t tmem_a, uint32_t b_lo,
                                             uint32_t accumulate) {
  issue_second_seq(tmem_d, tmem_a, b_lo, accumulate, std::make_integer_sequence<int, 8>{});
}
// The same in two parts: the columns that each warpgroup writes first, then the others.
__device__ __forceinline__ void issue_second_part(bool first, uint32_t tmem_d, uint32_t tmem_a, uint32_t b_lo,
                                                  uint32_t accumulate) {
  if (first)
    issue_second_seq(tmem_d, tmem_a, b_lo, accumulate, std::integer_sequence<int, 0, 1, 4, 5>{});
  else
    issue_second_seq(tmem_d, tmem_a, b_lo, 1, std::integer_sequence<int, 2, 3, 6, 7>{});
}

// Byte offset of 16-byte chunk c (0..15) of row r in a 128 x 128 bf16 tile stored as
// two 64-column halves in the 128-byte swizzle.
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  return static_cast<uint32_t>((c >> 3) * kHalfBytes + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

__device__ __forceinline__ void zero_row(uint32_t tile, int r) {
  for (int c = 0; c < 16; ++c) ptx::st_shared_v4(tile + chunk_at(r, c), 0, 0, 0, 0);
}

// Sets the non-finite elements of a row to 0; with_col(col) for each of them.
template <typename F>
__device__ __forceinline__ void clean_row(uint32_t tile, int r, F with_col) {
  for (int c = 0; c < 16; ++c) {
    const uint4 x = ptx::ld_shared_v4(tile + chunk_at(r, c));
    uint32_t w[4] = {x.x, x.y, x.z, x.w};
    bool dirty = false;
    for (int e = 0; e < 8; ++e) {
      const uint32_t h = (w[e >> 1] >> (16 * (e & 1))) & 0xFFFFu;
      if ((h & 0x7F80u) != 0x7F80u) continue;
      with_col(8 * c + e);
      w[e >> 1] &= ~(0xFFFFu << (16 * (e & 1)));
      dirty = true;
    }
    if (dirty) ptx::st_shared_v4(tile + chunk_at(r, c), w[0], w[1], w[2], w[3]);
  }
}

// Record of an item's non-finite elements found in masked tiles: per result column the
// last (or first) row that has one, and whether there is any.
constexpr int kPoisonWords = kD + 4, kPoisonBytes = kPoisonWords * 4;

// A meeting of the eight softmax warps, on an mbarrier of eight arrivals: a named barrier would
// hold the others for good when one has left the item's loop after a wait that ran out.
struct Meeting {
  uint32_t bar;
  volatile int* abort_flag;
  unsigned long long timeout_ns;
  int met;
  __device__ __forceinline__ bool meet(int lane) {
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(bar);
    return warp_wait(bar, met++ & 1, abort_flag, timeout_ns);
  }
};

// By the softmax warps, which all found the record set: once every one has read it.
__device__ __forceinline__ bool clear_poison(int* rec, int none, Meeting& all, int lane) {
  if (!all.meet(lane)) return false;
  const int t = static_cast<int>(threadIdx.x) - 32 * kSoftmaxWarp0;
  if (t < kD) rec[t] = none;
  if (t == kD) rec[kD] = 0;
  return all.meet(lane);
}

// TMA load of one 128 x 128 tile (two 64-column boxes).
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, uint32_t bar, int layout,
                                          int row, int head, int batch, uint64_t policy) {
  int c1, c2;
  tma_coords(layout, row, head, c1, c2);
  for (int hf = 0; hf < 2; ++hf)
    ptx::tma_load_4d_hint(dst + hf * kHalfBytes, map, bar, 64 * hf, c1, c2, batch, policy);
}

// Element offset of (head, row) in a tensor of H heads and S rows per batch entry.
__device__ __forceinline__ size_t row_at(int layout, int batch, int H, int S, int head, int row) {
  return (layout == 0 ? (static_cast<size_t>(batch) * H + head) * S + row
                      : (static_cast<size_t>(batch) * S + row) * H + head) * kD;
}

// Two neighbouring fp32 of a TMEM row.
__device__ __forceinline__ uint64_t pair_of(const uint32_t (&r)[32], int x) {
  return ptx::f2_pack(__uint_as_float(r[x]), __uint_as_float(r[x + 1]));
}

// kCols finished columns of a warp's 32 rows of a result in TMEM -> bf16 in global memory.
// A thread holds one row (lane 4 hi + lo: row 4 hi + lo); stored as it is, a warp's
// 16-byte store would touch 32 lines (3,300 cycles an item in dq). So 64 columns at a
// time, an 8 x 8 transposition across the lanes of one lo (hi against the 16-byte chunk,
// three exchanges) leaves chunk hi of row 4 k + lo in register k, and each store writes
// 128 bytes of four rows. `out`: row 0 of the warp, pitch: elements from row to row, rows:
// how many are stored. `poison(col)`: the thread's row is NaN there; any: there is such
// a column. zero: no product was formed, the result is 0. sum: the thread's terms so far
// (the tile's, as store_part leaves them, at the thread's row and first column), or null.
template <int kCols, typename F>
__device__ __forceinline__ void store_rows(uint32_t tacc, bool zero, float factor, int mode, uint16_t* out,
                                           size_t pitch, int rows, int lane, const float4* sum, bool any,
                                           F poison) {
  const uint64_t f2 = ptx::f2_pack(factor, factor);
  const uint32_t bias = mode == 1 ? 0x8000u : 0u;
  const int hi = lane >> 2, lo = lane & 3;
#pragma unroll
  for (int part = 0; part < kCols / 64; ++part) {
    uint32_t w[8][4];
#pragma unroll
    for (int ch = 0; ch < 2; ++ch) {
      uint32_t r[32];
      if (!zero) {
        ptx::tmem_ld32(tacc + 64 * part + 32 * ch, r);
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) r[i] = 0;
      }
      if (sum) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 x = sum[(16 * part + 8 * ch + i) * kTile];
          r[4 * i] = __float_as_uint(__uint_as_float(r[4 * i]) + x.x);
          r[4 * i + 1] = __float_as_uint(__uint_as_float(r[4 * i + 1]) + x.y);
          r[4 * i + 2] = __float_as_uint(__uint_as_float(r[4 * i + 2]) + x.z);
          r[4 * i + 3] = __float_as_uint(__uint_as_float(r[4 * i + 3]) + x.w);
        }
      }
      if (any) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (poison(64 * part + 32 * ch + i)) r[i] = 0x7FC00000u;
      }
      if (mode == 0) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float x0, x1;
          ptx::f2_unpack(ptx::f2_mul(pair_of(r, 2 * i), f2), x0, x1);
          w[4 * ch + i / 4][i % 4] = round_pair_bf16_rtne(x0, x1);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float x0, x1;
          ptx::f2_unpack(ptx::f2_mul(pair_of(r, 2 * i), f2), x0, x1);
          w[4 * ch + i / 4][i % 4] = round_pair_bf16(x0, x1, bias);
        }
      }
    }
#pragma unroll
    for (int bit = 1; bit < 8; bit *= 2) {
      const bool up = hi & bit;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        if (c & bit) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t x = __shfl_xor_sync(0xFFFFFFFFu, up ? w[c][e] : w[c | bit][e], 4 * bit);
          if (up)
            w[c][e] = x;
          else
            w[c | bit][e] = x;
        }
      }
    }
    uint16_t* dst = out + lo * pitch + 64 * part + 8 * hi;
    if (rows >= 32) {
#pragma unroll
      for (int k = 0; k < 8; ++k, dst += 4 * pitch)
        *reinterpret_cast<uint4*>(dst) = make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k, dst += 4 * pitch)
        if (4 * k + lo < rows) *reinterpret_cast<uint4*>(dst) = make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
    }
  }
}

// kCols columns of a row as fp32 into the workspace (one of n_splits terms of a sum, or an
// item's sum so far), or added to what the thread left there. A tile's terms lie by chunks of
// four columns, [chunk][row][4], so that a warp's store is 512 consecutive bytes. `part`: the
// tile's terms at the thread's row and first column.
template <int kCols, typename F>
__device__ __forceinline__ void store_part(uint32_t tacc, bool zero, float4* part, bool add, F poison) {
  const float nan = __int_as_float(0x7FC00000);
#pragma unroll 1
  for (int ch = 0; ch < kCols / 16; ++ch) {
    uint32_t r[16];
    if (!zero) {
      ptx::tmem_ld16(tacc + 16 * ch, r);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) r[i] = 0;
    }
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = poison(16 * ch + i + e) ? nan : __uint_as_float(r[i + e]);
      float4* at = part + (4 * ch + i / 4) * kTile;
      if (add) {
        const float4 y = *at;
        x[0] += y.x; x[1] += y.y; x[2] += y.z; x[3] += y.w;
      }
      *at = make_float4(x[0], x[1], x[2], x[3]);
    }
  }
}

// The softmax threads' turns, over 64 columns each. kMask is a template argument:
// as a run-time test inside, its compares ran in every tile (half of the
// instructions of the unmasked loop).

// dkv: P from S (a lane's key against 64 queries, whose -lse log2(e) are in shared
// memory); kept in pr, and written over S as bf16.
template <bool kMask>
__device__ __forceinline__ void dkv_p(uint32_t tS, const ulonglong2* stat, uint64_t c2, int lo, int hi,
                                      Half& pr, uint32_t half_bar, int lane) {
  by_halves(tS, [&](int ch, const uint32_t (&r)[32]) {
    uint32_t w[16];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const ulonglong2 nl = stat[8 * ch + e];  // four columns
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int x = 4 * e + 2 * u;
        float t0, t1;
        ptx::f2_unpack(ptx::f2_fma(pair_of(r, x), c2, u ? nl.y : nl.x), t0, t1);
        float p0 = ptx::ex2(t0), p1 = ptx::ex2(t1);
        if (kMask) {
          const int col = 32 * ch + x;
          if (col < lo || col >= hi) p0 = 0.f;
          if (col + 1 < lo || col + 1 >= hi) p1 = 0.f;
        }
        pr[16 * ch + 2 * e + u] = ptx::f2_pack(p0, p1);
        w[2 * e + u] = ptx::pack_bf16x2(p0, p1);
      }
    }
    ptx::tmem_st16(tS + 16 * ch, w);
    if (ch == 0) {
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(half_bar);
    }
  });
}

// dkv: dS from dP and P, written over dP as bf16.
template <bool kMask>
__device__ __forceinline__ void dkv_ds(uint32_t tP, const ulonglong2* stat, int lo, int hi, const Half& pr) {
  by_halves(tP, [&](int ch, const uint32_t (&r)[32]) {
    uint32_t w[16];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const ulonglong2 nd = stat[32 + 8 * ch + e];  // four columns of -D
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int x = 4 * e + 2 * u;
        float s0, s1;
        ptx::f2_unpack(
            ptx::f2_mul(pr[16 * ch + 2 * e + u], ptx::f2_add(pair_of(r, x), u ? nd.y : nd.x)), s0, s1);
        if (kMask) {
          const int col = 32 * ch + x;
          if (col < lo || col >= hi) s0 = 0.f;
          if (col + 1 < lo || col + 1 >= hi) s1 = 0.f;
        }
        w[2 * e + u] = ptx::pack_bf16x2(s0, s1);
      }
    }
    ptx::tmem_st16(tP + 16 * ch, w);
  });
}

// dq: dS from dP and P (a lane's query against 64 keys), written over S as bf16.
template <bool kMask>
__device__ __forceinline__ void dq_ds(uint32_t tP, uint32_t tS, uint64_t nd2, int hi, const Half& pr) {
  by_halves(tP, [&](int ch, const uint32_t (&r)[32]) {
    uint32_t w[16];
#pragma unroll
    for (int x = 0; x < 16; ++x) {
      float s0, s1;
      ptx::f2_unpack(ptx::f2_mul(pr[16 * ch + x], ptx::f2_add(pair_of(r, 2 * x), nd2)), s0, s1);
      if (kMask) {
        if (32 * ch + 2 * x >= hi) s0 = 0.f;
        if (32 * ch + 2 * x + 1 >= hi) s1 = 0.f;
      }
      w[x] = ptx::pack_bf16x2(s0, s1);
    }
    ptx::tmem_st16(tS + 16 * ch, w);
  });
}

// ---------------------------------------------------------------- dK and dV
//
// One CTA: 128 keys of one key/value head, streaming the query tiles (of every query
// head of the group) that see any of them. Transposed scores put a key in each
// TMEM lane: S^T = K Q^T, dP^T = V dO^T (both operands in shared memory,
// K-major), then dV += P^T dO and dK += dS^T Q with P^T, dS^T from TMEM and
// dO, Q as the same shared tiles read MN-major.
// Tensor memory: S/P [0,128), dP/dS [128,256), dK [256,384), dV [384,512).
// It is full, so S and dP have one buffer each and the two halves of the softmax
// take turns with the tensor pipe: while dV_i and S_{i+1} run, the threads form
// dS_i from dP_i; while dK_i and dP_{i+1} run, they form P_{i+1} from S_{i+1}.
// Each turn has 1024 tensor cycles to cover 64 exponentials per thread, or 64
// subtract-multiplies. P is handed over in two halves, so that dV starts on the first.
// Bound by the tensor cores: of four products' 2048 cycles it takes 2,320 a tile pair (8192
// x 8192, 32 heads: 1.2 ms); there the power cap sets the clock, and without the
// exponentials, the statistics or the loads it takes as long. 64-query tiles would let S
// and dP have two buffers, but an N = 64 product runs at two thirds of the rate.
// Shared memory is full as well: K, V, three stages of Q and two of dO. Q_i is read last
// (dK_i) shortly before S_{i+2} wants Q_{i+2}: with two stages its refill had 1024 cycles, and
// takes some 1600 when every SM streams; dO has slack.
constexpr int kDkvQStages = 3, kDkvOStages = 2;
enum : int {
  kDkvKV = 0,
  kDkvKVFree,   // the item's last S and dP products have read K and V
  kDkvQFull,
  kDkvQEmpty = kDkvQFull + kDkvQStages,
  kDkvOFull = kDkvQEmpty + kDkvQStages,  // dO and the row statistics
  kDkvOEmpty = kDkvOFull + kDkvOStages,
  kDkvSFull = kDkvOEmpty + kDkvOStages,
  kDkvPHalf,    // each warpgroup's first 32 columns of P
  kDkvPFull,
  kDkvDpFull,
  kDkvDsFull,
  kDkvAcc,      // dK and dV of an item, or of kAccTiles of its tiles
  kDkvAccFree,  // the epilogue has read them
  kDkvLanded,
  kDkvChecked,
  kDkvDrain,
  kDkvMeet,     // the softmax warps among themselves
  kDkvItemFull,
  kDkvItemEmpty = kDkvItemFull + kItemSlots,
  kDkvBars = kDkvItemEmpty + kItemSlots
};
constexpr int kDkvOffK = 0, kDkvOffV = kTileBytes, kDkvOffQ = 2 * kTileBytes,
              kDkvOffO = kDkvOffQ + kDkvQStages * kTileBytes,
              kDkvOffStats = kDkvOffO + kDkvOStages * kTileBytes,
              kDkvOffItems = kDkvOffStats + kDkvOStages * kStatFloats * 4,
              kDkvOffPoison = kDkvOffItems + 16 * kItemSlots, kDkvOffBar = kDkvOffPoison + kPoisonBytes,
              kDkvOffSlot = kDkvOffBar + kDkvBars * 8, kDkvSmem = kDkvOffSlot + 8;
static_assert(kDkvSmem <= 232448, "shared memory budget (dkv)");

// An item: an owned key tile and the part of its streamed tiles: query tiles from first_qt
// on, for each query head of the group, n of them from number t0 on (skip: nothing
// to do, not even a zero to store).
struct DkvItem {
  Seq s;
  int first_qt, per, t0, n;
  int off, k0;  // key j is visible to query i iff j <= i + off (causal); the tile's first key
  bool skip;
};

template <bool kCausal, bool kVarlen>
__device__ __forceinline__ DkvItem dkv_item(const BwdParams& p, int item) {
  DkvItem r;
  r.s = seq_of<kCausal, kVarlen, false>(p, item);
  const Seq& s = r.s;
  r.off = s.sk - s.sq;
  r.k0 = s.tile * kTile;
  r.skip = kVarlen && (s.bad || r.k0 >= s.sk);
  const int nqt = (s.sq + kTile - 1) / kTile;
  r.first_qt = kCausal ? min(max(0, r.k0 - r.off) / kTile, nqt) : 0;
  r.per = nqt - r.first_qt;
  part_of(r.per * p.group, p.n_splits, s.split, r.t0, r.n);
  if (r.skip) r.n = 0;
  return r;
}

// A tile some of whose pairs are hidden: crossed by the diagonal, or past the end.
template <bool kCausal>
__device__ __forceinline__ bool dkv_masked(int q0, int sq, int off, int k0) {
  return q0 + kTile > sq || (kCausal && q0 + off < k0 + kTile - 1);
}

// First query of the item's streamed tiles, one after another (no division per tile).
struct QueryTiles {
  int q0, first, last;
  __device__ __forceinline__ explicit QueryTiles(const DkvItem& w) {
    first = w.first_qt * kTile;
    last = (w.first_qt + w.per - 1) * kTile;
    q0 = w.n > 0 ? (w.first_qt + w.t0 % w.per) * kTile : 0;
  }
  __device__ __forceinline__ void step() { q0 = q0 == last ? first : q0 + kTile; }
};

template <bool kCausal, bool kVarlen, bool kLong>
__global__ void __launch_bounds__(kThreads, 1)
    attn_bwd_dkv(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                 const BwdParams p) {
  extern __shared__ uint8_t smem_raw[];
  // Dynamic shared memory starts on a 1024-byte boundary here (the tiles' swizzle wants it,
  // and there is no room to align it).
  const uint32_t sbase = ptx::smem_u32(smem_raw);
  uint8_t* smem = smem_raw;
  if (sbase & 1023u) {
    if (threadIdx.x == 0) atomicOr(&g_attn_status, 4u);
    ptx::grid_dependency_wait();
    return;
  }
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kDkvOffSlot);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kDkvOffSlot + 4);
  int* poison = reinterpret_cast<int*>(smem + kDkvOffPoison);
  auto bar = [&](int i) -> uint32_t { return sbase + kDkvOffBar + 8u * static_cast<uint32_t>(i); };
  // (Through a shuffle, so that the compiler knows it to be the same on every lane.)
  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  constexpr bool kCheck = kCausal || kVarlen;
  const Items items{sbase + kDkvOffItems, bar(kDkvItemFull), bar(kDkvItemEmpty), abort_flag, p.timeout_ns};

  if (threadIdx.x == 0) {
    for (int i = 0; i < kDkvBars; ++i)
      ptx::mbar_init(bar(i), (i == kDkvPHalf || i == kDkvPFull || i == kDkvDsFull || i == kDkvAccFree || i == kDkvMeet)
                                 ? 8
                             : i >= kDkvItemEmpty ? item_readers(kCheck)
                             : i == kDkvSFull     ? 1 + p.withhold
                                                  : 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
  }
  for (int i = threadIdx.x; i < kPoisonWords; i += kThreads) poison[i] = i < kD ? -1 : 0;
  if (warp == 0 && lane == 0) {
    ptx::prefetch_tmap(&tm_q);
    ptx::prefetch_tmap(&tm_k);
    ptx::prefetch_tmap(&tm_v);
    ptx::prefetch_tmap(&tm_do);
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  ptx::launch_dependents();
  const uint32_t tS = tmem, tP = tmem + 128, tK = tmem + 256, tV = tmem + 384;

  // In every role: `used` counts the items with streamed tiles so far (the phases of the
  // per-item barriers), `tile` their streamed tiles (the phases of the per-tile ones;
  // tile t goes to stage t % kDkvQStages of Q's ring, t % kDkvOStages of dO's).
  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    if (lane == 0) {
      const uint64_t pol_once = ptx::l2_policy_evict_first();
      const uint64_t pol_reuse = ptx::l2_policy_evict_last();
      int used = 0, q_issued = 0, o_issued = 0, asked = 0;
      bool ok = true;
      for (int item = static_cast<int>(blockIdx.x), it = 0; ok && item >= 0; ++it) {
        const DkvItem w = dkv_item<kCausal, kVarlen>(p, item);
        const Seq& s = w.s;
        if (kVarlen && s.bad) atomicOr(&g_attn_status, 2u);
        if (w.n > 0) {
          if (used > 0 && !(ok = wait_bounded(bar(kDkvKVFree), (used - 1) & 1, abort_flag, p.timeout_ns, true)))
            break;
          dbg_ok(s.k_base + w.k0 < p.Sk);
          ptx::mbar_arrive_expect_tx(bar(kDkvKV), 2 * kTileBytes);
          load_tile(sbase + kDkvOffK, &tm_k, bar(kDkvKV), p.layout, s.k_base + w.k0, s.head, s.batch, pol_once);
          load_tile(sbase + kDkvOffV, &tm_v, bar(kDkvKV), p.layout, s.k_base + w.k0, s.head, s.batch, pol_once);
          QueryTiles qt(w);
          int h = s.head * p.group + w.t0 / w.per;
          auto load_stats = [&](int os, int head, int q0) {
            const float* src = p.stats + (static_cast<size_t>(s.slot_q) + static_cast<size_t>(head) * p.q_slots +
                                          q0 / kTile) * kStatFloats;
            ptx::bulk_load(sbase + kDkvOffStats + os * kStatFloats * 4, src, kStatFloats * 4,
                           bar(kDkvOFull + os));
          };
          // The row statistics are the only thing here that the kernel before this one writes:
          // the CTA's first tiles load while it ends.
          const int early = used == 0 ? min(w.n, kDkvOStages) : 0;
          QueryTiles late = qt;
          int late_h = h;
          ++used;
          for (int i = 0; i < w.n; ++i) {
            const int qs = q_issued % kDkvQStages, os = o_issued % kDkvOStages;
            dbg_ok(s.q_base + qt.q0 < p.Sq && h < p.Hq);
            if (!(ok = wait_bounded(bar(kDkvQEmpty + qs), ((q_issued / kDkvQStages) & 1) ^ 1, abort_flag,
                                    p.timeout_ns, true)))
              break;
            ptx::mbar_arrive_expect_tx(bar(kDkvQFull + qs), kTileBytes);
            load_tile(sbase + kDkvOffQ + qs * kTileBytes, &tm_q, bar(kDkvQFull + qs), p.layout,
                      s.q_base + qt.q0, h, s.batch, pol_reuse);
            ++q_issued;
            if (!(ok = wait_bounded(bar(kDkvOEmpty + os), ((o_issued / kDkvOStages) & 1) ^ 1, abort_flag,
                                    p.timeout_ns, true)))
              break;
            ptx::mbar_arrive_expect_tx(bar(kDkvOFull + os), kTileBytes + kStatFloats * 4);
            load_tile(sbase + kDkvOffO + os * kTileBytes, &tm_do, bar(kDkvOFull + os), p.layout,
                      s.q_base + qt.q0, h, s.batch, pol_reuse);
            if (i >= early) load_stats(os, h, qt.q0);
            ++o_issued;
            if (i + 1 == early) {
              ptx::grid_dependency_wait();
              ptx::fence_proxy_async_global();
              for (int e = 0; e < early; ++e) {
                load_stats(e, late_h, late.q0);
                if (late.q0 == late.last) ++late_h;
                late.step();
              }
            }
            if (qt.q0 == qt.last) ++h;
            qt.step();
          }
          if (!ok) break;
        }
        items.ask(it);
        asked = it + 1;
        item = items.next_lane(it);
      }
      // Every copy this thread started lands before the CTA can exit, and so does every
      // answer asked for.
      if (used > 0) wait_bounded(bar(kDkvKV), (used - 1) & 1, abort_flag, p.timeout_ns, false);
      for (int st = 0; st < kDkvQStages && st < q_issued; ++st)
        wait_bounded(bar(kDkvQFull + st), ((q_issued - 1 - st) / kDkvQStages) & 1, abort_flag, p.timeout_ns,
                     false);
      for (int st = 0; st < kDkvOStages && st < o_issued; ++st)
        wait_bounded(bar(kDkvOFull + st), ((o_issued - 1 - st) / kDkvOStages) & 1, abort_flag, p.timeout_ns,
                     false);
      items.drain(asked);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer (whole warp)
    const uint32_t k_desc = desc_lo(sbase + kDkvOffK, 16), v_desc = desc_lo(sbase + kDkvOffV, 16);
    auto q_tile = [&](int t) -> uint32_t { return sbase + kDkvOffQ + (t % kDkvQStages) * kTileBytes; };
    auto o_tile = [&](int t) -> uint32_t { return sbase + kDkvOffO + (t % kDkvOStages) * kTileBytes; };
    auto wait = [&](int b, uint32_t par) -> bool {
      const bool r = warp_wait(bar(b), par & 1, abort_flag, p.timeout_ns);
      ptx::tc_fence_after();
      return r;
    };
    int used = 0, tile = 0, checks = 0, accs = 0;
    bool ok = true;
    for (int item = static_cast<int>(blockIdx.x), it = 0; ok && item >= 0; ++it) {
      const DkvItem w = dkv_item<kCausal, kVarlen>(p, item);
      if (w.n > 0) {
        QueryTiles qt(w);  // of the next S
        bool masked_s = false, masked = false;  // the tile of the last S, and of the last dP
        auto do_s = [&](int t) -> bool {
          if (!wait(kDkvQFull + t % kDkvQStages, t / kDkvQStages)) return false;
          masked_s = kCheck && dkv_masked<kCausal>(qt.q0, w.s.sq, w.off, w.k0);
          qt.step();
          issue_s(tS, k_desc, desc_lo(q_tile(t), 16));
          ptx::mma_commit_warp(bar(kDkvSFull));
          return true;
        };
        auto do_dp = [&](int t) -> bool {
          if (!wait(kDkvOFull + t % kDkvOStages, t / kDkvOStages)) return false;
          masked = masked_s;
          if (masked && lane == 0) ptx::mbar_arrive(bar(kDkvLanded));
          issue_s(tP, v_desc, desc_lo(o_tile(t), 16));
          ptx::mma_commit_warp(bar(kDkvDpFull));
          return true;
        };
        ok = wait(kDkvKV, used) && do_s(tile) && do_dp(tile);
        if (ok && w.n == 1) ptx::mma_commit_warp(bar(kDkvKVFree));
        for (int i = 0; ok && i < w.n; ++i) {
          const int t = tile + i;
          const bool more = i + 1 < w.n;
          if (!(ok = wait(kDkvPHalf, t))) break;
          // dV (and dK) start anew with the item, and after every kAccTiles tiles.
          const int summed = kLong ? i & (kAccTiles - 1) : i;
          if (summed == 0 && accs > 0 && !(ok = wait(kDkvAccFree, accs - 1))) break;
          if (masked) {  // the second products read checked rows
            if (!(ok = wait(kDkvChecked, checks))) break;
            ++checks;
          }
          issue_second_part(true, tV, tS, desc_lo(o_tile(t), kHalfBytes), summed > 0);
          if (!(ok = wait(kDkvPFull, t))) break;
          issue_second_part(false, tV, tS, desc_lo(o_tile(t), kHalfBytes), 1);
          if (more && !(ok = do_s(t + 1))) break;
          if (!(ok = wait(kDkvDsFull, t))) break;
          issue_second(tK, tP, desc_lo(q_tile(t), kHalfBytes), summed > 0);
          ptx::mma_commit_warp(bar(kDkvQEmpty + t % kDkvQStages));
          // (dO's last product is dV, but the statistics beside it are read until dS.)
          ptx::mma_commit_warp(bar(kDkvOEmpty + t % kDkvOStages));
          if (kLong && more && summed == kAccTiles - 1) {
            ptx::mma_commit_warp(bar(kDkvAcc));
            ++accs;
          }
          if (more && !(ok = do_dp(t + 1))) break;
          if (i + 2 == w.n) ptx::mma_commit_warp(bar(kDkvKVFree));  // the last dP was issued
        }
        if (ok) ptx::mma_commit_warp(bar(kDkvAcc));
        ++accs;
        tile += w.n;
        ++used;
      }
      if (ok) item = items.next_warp(it, lane);
    }
    ptx::mma_commit_warp(bar(kDkvDrain));
    wait_bounded(bar(kDkvDrain), 0, abort_flag, p.timeout_ns, false);  // every MMA is done
    __syncwarp();
  } else if (warp < kSoftmaxWarp0) {
    // ------------------------------------------------ check of the masked tiles (warps 2-3)
    // A hidden pair has P = dS = 0, and 0 * NaN in the second products would carry a
    // non-finite element of its Q or dO row to keys that do not see it. Rows that
    // take no part (past the sequence's end, or seeing no key) are set to 0. A row
    // with a non-finite element has a NaN among its statistics; its non-finite
    // elements are set to 0 as well. The keys that do see it still get NaN: in
    // every column of dK (and of dV, when it is Q) through the statistics, and in
    // the column of a non-finite dO element through `poison`, the last row that has
    // one there. An item's epilogue clears it; only then are the next item's put in.
    // S and dP need no checked rows (a hidden pair's are not used), so the check runs beside
    // them, and only a row to be changed waits until they have read it. (Before S, the check
    // held up every masked tile: 16
    // causal sequences of 1900 tokens 620 us instead of 604.)
    if constexpr (kCheck) {
      const int tid = static_cast<int>(threadIdx.x) - 64;
      int accs = 0, tile = 0, m = 0;  // accs: accumulators of the items before this one
      bool ok = true;
      for (int item = static_cast<int>(blockIdx.x), it = 0; ok && item >= 0; ++it) {
        const DkvItem w = dkv_item<kCausal, kVarlen>(p, item);
        const Seq& s = w.s;
        QueryTiles qt(w);
        for (int i = 0; i < w.n; ++i, qt.step()) {
          const int q0 = qt.q0;
          if (!dkv_masked<kCausal>(q0, s.sq, w.off, w.k0)) continue;
          ok = wait_bounded(bar(kDkvLanded), m & 1, abort_flag, p.timeout_ns, true);
          ok = !ptx::named_barrier_or(1, 64, !ok);
          if (!ok) break;
          ++m;
          const int os = (tile + i) % kDkvOStages;
          const uint32_t q_t = sbase + kDkvOffQ + ((tile + i) % kDkvQStages) * kTileBytes;
          const uint32_t o_t = sbase + kDkvOffO + os * kTileBytes;
          const float* stat = reinterpret_cast<const float*>(smem + kDkvOffStats) + os * kStatFloats;
          bool dirty = false;
          auto products_done = [&] {
            wait_bounded(bar(kDkvDpFull), (tile + i) & 1, abort_flag, p.timeout_ns, true);
          };
          for (int r = tid; r < kTile; r += 64) {
            const float nl = stat[r], nd = stat[kTile + r];
            const bool past = q0 + r >= s.sq;  // (zero already in a dense tensor's tile)
            if (past && !kVarlen) continue;
            if (past || nl == -__int_as_float(0x7F800000)) {
              products_done();
              zero_row(q_t, r);
              zero_row(o_t, r);
              dirty = true;
            } else if (isnan(nl) || isnan(nd)) {
              products_done();
              // (Past the item's first kAccTiles the last one's epilogue is long over.)
              if (accs > 0 && (!kLong || i < kAccTiles))
                wait_bounded(bar(kDkvAccFree), (accs - 1) & 1, abort_flag, p.timeout_ns, true);
              clean_row(q_t, r, [](int) {});
              clean_row(o_t, r, [&](int col) {
                atomicMax(&poison[col], q0 + r);
                *static_cast<volatile int*>(poison + kD) = 1;
              });
              dirty = true;
            }
          }
          if (dirty) ptx::fence_proxy_async_smem();
          __syncwarp();
          ptx::named_barrier_sync(1, 64);
          if (tid == 0) ptx::mbar_arrive(bar(kDkvChecked));
        }
        tile += w.n;
        accs += accumulators<kLong>(w.n);
        if (ok) item = next_together(items, it, lane);
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax
    const int g = (warp - kSoftmaxWarp0) >> 2;  // 64-query half of the tile
    const int wq = warp & 3;
    const int row = wq * 32 + lane;             // key within the tile
    const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tSh = tS + lane_base + 64 * g, tPh = tP + lane_base + 64 * g;
    const uint64_t c2 = ptx::f2_pack(p.c, p.c);
    Meeting all{bar(kDkvMeet), abort_flag, p.timeout_ns, 0};
    int accs = 0, tile = 0;
    bool ok = true;
    int item = static_cast<int>(blockIdx.x);
    DkvItem w = dkv_item<kCausal, kVarlen>(p, item);
    for (int it = 0; ok && item >= 0; ++it) {
      const int first_row = w.k0 + row - w.off;  // the first query that sees this key (causal)
      const int n = w.n, sq = w.s.sq, off = w.off, k0 = w.k0;
      QueryTiles qt(w);
      int i = 0;
      do {
        const int end = kLong ? min(n, i + kAccTiles) : n;
        for (; i < end; ++i, ++tile, qt.step()) {
          const bool mk = dkv_masked<kCausal>(qt.q0, sq, off, k0);
          // The columns of this half that this key is visible to: [lo, hi).
          const int lo = kCausal ? first_row - qt.q0 - 64 * g : 0;
          const int hi = sq - qt.q0 - 64 * g;
          const ulonglong2* stat = reinterpret_cast<const ulonglong2*>(
              smem + kDkvOffStats + (tile % kDkvOStages) * kStatFloats * 4 + 256 * g);
          Half pr;
          if (!(ok = warp_wait(bar(kDkvSFull), tile & 1, abort_flag, p.timeout_ns))) break;
          // (dO's barrier, for the statistics that land with it.)
          if (!(ok = warp_wait(bar(kDkvOFull + tile % kDkvOStages), (tile / kDkvOStages) & 1, abort_flag,
                               p.timeout_ns)))
            break;
          ptx::tc_fence_after();
          if (mk)
            dkv_p<true>(tSh, stat, c2, lo, hi, pr, bar(kDkvPHalf), lane);
          else
            dkv_p<false>(tSh, stat, c2, lo, hi, pr, bar(kDkvPHalf), lane);
          ptx::tmem_wait_st();
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar(kDkvPFull));

          if (!(ok = warp_wait(bar(kDkvDpFull), tile & 1, abort_flag, p.timeout_ns))) break;
          ptx::tc_fence_after();
          if (mk)
            dkv_ds<true>(tPh, stat, lo, hi, pr);
          else
            dkv_ds<false>(tPh, stat, lo, hi, pr);
          ptx::tmem_wait_st();
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar(kDkvDsFull));
        }
        if (!ok) break;
        // ---- epilogue: warpgroup 0 stores dK, warpgroup 1 dV, or adds them to the item's
        // terms. (The next item is taken up before the wait.)
        const bool zero = n == 0, last = !kLong || i == n;
        const DkvItem v = w;
        if (last) {
          item = items.next_warp(it, lane);
          if (item >= 0) w = dkv_item<kCausal, kVarlen>(p, item);
        }
        if (!zero && !(ok = warp_wait(bar(kDkvAcc), accs & 1, abort_flag, p.timeout_ns))) break;
        ptx::tc_fence_after();
        if (!v.skip) {
          const Seq& s = v.s;
          const uint32_t tacc = (g == 0 ? tK : tV) + lane_base;
          const bool any = kCheck && !zero && last && *static_cast<volatile int*>(poison + kD);
          // The last query row whose non-finite dO element a key may see (see above).
          const int seen = kCausal ? max(0, v.k0 + row - v.off) : 0;
          auto is_nan = [&](int col) -> bool { return any && g == 1 && poison[col] >= seen; };
          auto terms = [&]() -> float4* {
            const size_t slots = static_cast<size_t>(p.k_slots) * (kVarlen ? p.Hkv : p.BH);
            const size_t slot = static_cast<size_t>(s.slot_k) + static_cast<size_t>(s.head) * p.k_slots + s.tile;
            return reinterpret_cast<float4*>(
                       p.part + ((static_cast<size_t>(s.split) * 2 + g) * slots + slot) * kTile * kD) + row;
          };
          if (last && p.n_splits == 1) {
            const int first = v.k0 + 32 * wq;  // of the warp's rows
            const int rows = dbg_ok(s.k_base + s.sk <= p.Sk) ? s.sk - first : 0;
            uint16_t* dst = (g == 0 ? p.dk : p.dv) +
                            row_at(p.layout, s.batch, p.Hkv, p.Sk, s.head, s.k_base + (rows > 0 ? first : 0));
            store_rows<kD>(tacc, zero, g == 0 ? p.scale : 1.f, p.mode, dst,
                           static_cast<size_t>(p.layout == 0 ? 1 : p.Hkv) * kD, rows, lane,
                           kLong && n > kAccTiles ? terms() : nullptr, any && g == 1, is_nan);
          } else {
            store_part<kD>(tacc, zero, terms(), kLong && i > kAccTiles, is_nan);
          }
          if (any && !(ok = clear_poison(poison, -1, all, lane))) break;
        }
        if (!zero) {
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar(kDkvAccFree));
          ++accs;
        }
      } while (kLong && i < n);
      if (!ok) break;
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
  // A CTA leaves only after the kernel before it on the stream has finished, so
  // that this grid's end is the end of both.
  ptx::grid_dependency_wait();
}

// ---------------------------------------------------------------- dQ
//
// One CTA: 128 queries of one head, streaming the key tiles they see. S = Q K^T and
// dP = dO V^T from shared memory, dS over S's columns, dQ += dS K with K read
// MN-major from the tile that S used. Tensor memory: S/dS two buffers [0,256), dP
// [256,384), dQ [384,512). With two S buffers the tensor pipe forms S_{j+1} and
// dP_{j+1} around dQ_j, and a turn of the softmax (exponentials of S_{j+1}, then
// dS once dP_{j+1} is there) has 1536 tensor cycles. Bound by the tensor cores: 1,840 cycles a
// tile pair (8192 x 8192, 32 heads: 0.87 ms). It streams 64 KiB in those, 36 bytes a clock (9.9
// TB/s from L2, 27% of what that path can carry), and a copy without the loads takes as long;
// sharing them by TMA multicast between two CTAs of a cluster was slower (2.39 against 2.28 ms
// for the whole pass: both wait for the slower one at every tile).
//
// It also leaves the row statistics that dkv reads: per query row -lse log2(e) and -D,
// D = sum_c dO_ic O_ic, formed from the dO tile it has and the O tile, which passes
// through K's ring. (A kernel of its own for them
// read dO once more and cost 25 us of 2.35 ms on 8K self-attention, 47 of 1039 us on a
// packed batch, and a launch.) Rows past the end, and rows that see no key, get -Inf
// and 0 (P = 0). A non-finite D becomes NaN: it marks a row whose dO or O has a
// non-finite element. A row whose keys all have the logit -Inf is NaN, as its output is.
constexpr int kDqKStages = 3, kDqVStages = 2;  // K_j is in use while K_{j+2} loads
constexpr int kDqChecks = 4;  // masked tiles between landing and being checked: at most 2
enum : int {
  kDqQ = 0,
  kDqQFree,     // the item's last S and dP products, and the statistics, have read Q and dO
  kDqKFull,
  kDqKEmpty = kDqKFull + kDqKStages,
  kDqVFull = kDqKEmpty + kDqKStages,
  kDqVEmpty = kDqVFull + kDqVStages,
  kDqSFull = kDqVEmpty + kDqVStages,
  kDqDpFull = kDqSFull + 2,
  kDqDsFull,
  kDqAcc,       // dQ of an item, or of kAccTiles of its tiles
  kDqAccFree,   // the epilogue has read it
  kDqLanded,
  kDqChecked = kDqLanded + kDqChecks,
  kDqDrain = kDqChecked + kDqChecks,
  kDqMeet,      // the softmax warps among themselves
  kDqItemFull,
  kDqItemEmpty = kDqItemFull + kItemSlots,
  kDqBars = kDqItemEmpty + kItemSlots
};
constexpr int kDqOffQ = 0, kDqOffO = kTileBytes, kDqOffK = 2 * kTileBytes,
              kDqOffV = kDqOffK + kDqKStages * kTileBytes,
              kDqOffItems = kDqOffV + kDqVStages * kTileBytes, kDqOffPoison = kDqOffItems + 16 * kItemSlots,
              kDqOffDots = kDqOffPoison + kPoisonBytes, kDqOffBar = kDqOffDots + 2 * kTile * 4,
              kDqOffSlot = kDqOffBar + kDqBars * 8, kDqSmem = kDqOffSlot + 8 + 1024;
static_assert(kDqSmem <= 232448, "shared memory budget (dq)");

// An item: an owned query tile and the part [t0, t0 + n) of the key tiles any of its rows
// sees; from first_masked on some row does not see every key (the causal diagonal, or
// the ragged last tile). skip: nothing to do, not even a zero to store.
struct DqItem {
  Seq s;
  int off, q0, t0, n, first_masked;
  bool skip;
};

template <bool kCausal, bool kVarlen>
__device__ __forceinline__ DqItem dq_item(const BwdParams& p, int item) {
  DqItem r;
  r.s = seq_of<kCausal, kVarlen, true>(p, item);
  const Seq& s = r.s;
  r.off = s.sk - s.sq;
  r.q0 = s.tile * kTile;
  r.skip = kVarlen && (s.bad || r.q0 >= s.sq);
  int n_kv = (s.sk + kTile - 1) / kTile;
  r.first_masked = s.sk / kTile;
  if (kCausal) {
    const int last = min(s.sq, r.q0 + kTile) + r.off;  // keys the last row sees
    n_kv = min(n_kv, last <= 0 ? 0 : (last + kTile - 1) / kTile);
    r.first_masked = min(r.first_masked, max(0, r.q0 + r.off + 1) / kTile);
  }
  part_of(n_kv, p.n_splits, s.split, r.t0, r.n);
  if (r.skip) r.n = 0;
  return r;
}

// The ring of K takes, per item, O, K_0, K_1, ... (O's stage is free again by the time K_2
// is wanted): fill of K_j, counted from the item's first.
__device__ __forceinline__ int k_fill(int j) { return j + 1; }

template <bool kCausal, bool kVarlen, bool kLong>
__global__ void __launch_bounds__(kThreads, 1)
    attn_bwd_dq(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                const __grid_constant__ CUtensorMap tm_out, const BwdParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kDqOffSlot);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kDqOffSlot + 4);
  int* poison = reinterpret_cast<int*>(smem + kDqOffPoison);
  auto bar = [&](int i) -> uint32_t { return sbase + kDqOffBar + 8u * static_cast<uint32_t>(i); };
  // (Through a shuffle, so that the compiler knows it to be the same on every lane.)
  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  constexpr bool kCheck = kCausal || kVarlen;
  constexpr int kNever = 0x7FFFFFFF;
  const Items items{sbase + kDqOffItems, bar(kDqItemFull), bar(kDqItemEmpty), abort_flag, p.timeout_ns};

  if (threadIdx.x == 0) {
    for (int i = 0; i < kDqBars; ++i)
      ptx::mbar_init(bar(i), (i == kDqDsFull || i == kDqAccFree || i == kDqMeet) ? 8
                             : i >= kDqItemEmpty                                 ? item_readers(kCheck)
                             : i == kDqQFree                                     ? 2
                             : i == kDqSFull                                     ? 1 + p.withhold
                                                                                 : 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
  }
  for (int i = threadIdx.x; i < kPoisonWords; i += kThreads) poison[i] = i < kD ? kNever : 0;
  if (warp == 0 && lane == 0) {
    ptx::prefetch_tmap(&tm_q);
    ptx::prefetch_tmap(&tm_k);
    ptx::prefetch_tmap(&tm_v);
    ptx::prefetch_tmap(&tm_do);
    ptx::prefetch_tmap(&tm_out);
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  ptx::launch_dependents();  // the next kernel waits for this grid before it reads its results
  const uint32_t tP = tmem + 256, tQ = tmem + 384;

  // In every role: `used` counts the items with key tiles so far (the phases of the
  // per-item barriers), `tile` their key tiles (S buffer tile & 1), k_base the fills of
  // K's ring before the item.
  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    if (lane == 0) {
      const uint64_t pol_once = ptx::l2_policy_evict_first();
      const uint64_t pol_reuse = ptx::l2_policy_evict_last();
      int used = 0, k_issued = 0, v_issued = 0, asked = 0;
      bool ok = true;
      auto k_slot = [&]() -> bool {
        return wait_bounded(bar(kDqKEmpty + k_issued % kDqKStages), ((k_issued / kDqKStages) & 1) ^ 1,
                            abort_flag, p.timeout_ns, true);
      };
      for (int item = static_cast<int>(blockIdx.x), it = 0; ok && item >= 0; ++it) {
        const DqItem w = dq_item<kCausal, kVarlen>(p, item);
        const Seq& s = w.s;
        if (kVarlen && s.bad) atomicOr(&g_attn_status, 2u);
        if (w.n > 0) {
          const int kv_head = s.head / p.group;
          if (used > 0 && !(ok = wait_bounded(bar(kDqQFree), (used - 1) & 1, abort_flag, p.timeout_ns, true)))
            break;
          dbg_ok(s.q_base + w.q0 < p.Sq);
          ptx::mbar_arrive_expect_tx(bar(kDqQ), 2 * kTileBytes);
          load_tile(sbase + kDqOffQ, &tm_q, bar(kDqQ), p.layout, s.q_base + w.q0, s.head, s.batch, pol_once);
          load_tile(sbase + kDqOffO, &tm_do, bar(kDqQ), p.layout, s.q_base + w.q0, s.head, s.batch, pol_once);
          ++used;
          if (!(ok = k_slot())) break;
          const int os = k_issued % kDqKStages;
          ptx::mbar_arrive_expect_tx(bar(kDqKFull + os), kTileBytes);
          load_tile(sbase + kDqOffK + os * kTileBytes, &tm_out, bar(kDqKFull + os), p.layout, s.q_base + w.q0,
                    s.head, s.batch, pol_once);
          ++k_issued;
          for (int j = 0; j < w.n; ++j) {
            const int row = s.k_base + (w.t0 + j) * kTile;
            dbg_ok(row < p.Sk);
            if (!(ok = k_slot())) break;
            const int ks = k_issued % kDqKStages, vs = v_issued % kDqVStages;
            ptx::mbar_arrive_expect_tx(bar(kDqKFull + ks), kTileBytes);
            load_tile(sbase + kDqOffK + ks * kTileBytes, &tm_k, bar(kDqKFull + ks), p.layout, row, kv_head,
                      s.batch, pol_reuse);
            ++k_issued;
            if (!(ok = wait_bounded(bar(kDqVEmpty + vs), ((v_issued / kDqVStages) & 1) ^ 1, abort_flag,
                                    p.timeout_ns, true)))
              break;
            ptx::mbar_arrive_expect_tx(bar(kDqVFull + vs), kTileBytes);
            load_tile(sbase + kDqOffV + vs * kTileBytes, &tm_v, bar(kDqVFull + vs), p.layout, row, kv_head,
                      s.batch, pol_reuse);
            ++v_issued;
          }
          if (!ok) break;
        }
        items.ask(it);
        asked = it + 1;
        item = items.next_lane(it);
      }
      // Every copy this thread started lands before the CTA can exit, and so does every
      // answer asked for.
      if (used > 0) wait_bounded(bar(kDqQ), (used - 1) & 1, abort_flag, p.timeout_ns, false);
      for (int st = 0; st < kDqKStages && st < k_issued; ++st)
        wait_bounded(bar(kDqKFull + st), ((k_issued - 1 - st) / kDqKStages) & 1, abort_flag, p.timeout_ns,
                     false);
      for (int st = 0; st < kDqVStages && st < v_issued; ++st)
        wait_bounded(bar(kDqVFull + st), ((v_issued - 1 - st) / kDqVStages) & 1, abort_flag, p.timeout_ns,
                     false);
      items.drain(asked);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer (whole warp)
    const uint32_t q_desc = desc_lo(sbase + kDqOffQ, 16), o_desc = desc_lo(sbase + kDqOffO, 16);
    auto wait = [&](int b, uint32_t par) -> bool {
      const bool r = warp_wait(bar(b), par & 1, abort_flag, p.timeout_ns);
      ptx::tc_fence_after();
      return r;
    };
    int used = 0, tile = 0, k_base = 0, landed = 0, checked = 0, accs = 0;
    bool ok = true;
    for (int item = static_cast<int>(blockIdx.x), it = 0; ok && item >= 0; ++it) {
      const DqItem w = dq_item<kCausal, kVarlen>(p, item);
      const int n = w.n;
      if (n > 0) {
        auto k_tile = [&](int j) -> uint32_t {
          return sbase + kDqOffK + ((k_base + k_fill(j)) % kDqKStages) * kTileBytes;
        };
        auto masked = [&](int j) -> bool { return kCheck && w.t0 + j >= w.first_masked; };
        auto do_s = [&](int j) -> bool {
          const int f = k_base + k_fill(j);
          if (!wait(kDqKFull + f % kDqKStages, f / kDqKStages)) return false;
          issue_s(tmem + 128 * ((tile + j) & 1), q_desc, desc_lo(k_tile(j), 16));
          ptx::mma_commit_warp(bar(kDqSFull + ((tile + j) & 1)));
          if (masked(j)) {
            if (lane == 0) ptx::mbar_arrive(bar(kDqLanded + landed % kDqChecks));
            ++landed;
          }
          return true;
        };
        auto do_dp = [&](int j) -> bool {
          const int f = tile + j;
          if (!wait(kDqVFull + f % kDqVStages, f / kDqVStages)) return false;
          issue_s(tP, o_desc, desc_lo(sbase + kDqOffV + (f % kDqVStages) * kTileBytes, 16));
          ptx::mma_commit_warp(bar(kDqDpFull));
          ptx::mma_commit_warp(bar(kDqVEmpty + f % kDqVStages));
          // The item's last S was issued before its last dP.
          if (j + 1 == n) ptx::mma_commit_warp(bar(kDqQFree));
          return true;
        };
        ok = wait(kDqQ, used) && do_s(0) && (n == 1 ? do_dp(0) : do_dp(0) && do_s(1));
        for (int j = 0; ok && j < n; ++j) {
          if (!(ok = wait(kDqDsFull, tile + j))) break;
          if (j + 1 < n && !(ok = do_dp(j + 1))) break;
          if (masked(j)) {
            if (!(ok = wait(kDqChecked + checked % kDqChecks, checked / kDqChecks))) break;
            ++checked;
          }
          // dQ starts anew with the item, and after every kAccTiles tiles.
          const int summed = kLong ? j & (kAccTiles - 1) : j;
          if (summed == 0 && accs > 0 && !(ok = wait(kDqAccFree, accs - 1))) break;
          issue_second(tQ, tmem + 128 * ((tile + j) & 1), desc_lo(k_tile(j), kHalfBytes), summed > 0);
          ptx::mma_commit_warp(bar(kDqKEmpty + (k_base + k_fill(j)) % kDqKStages));
          if (kLong && j + 1 < n && summed == kAccTiles - 1) {
            ptx::mma_commit_warp(bar(kDqAcc));
            ++accs;
          }
          if (j + 2 < n && !(ok = do_s(j + 2))) break;
        }
        if (ok) ptx::mma_commit_warp(bar(kDqAcc));
        ++accs;
        tile += n;
        k_base += n + 1;
        ++used;
      }
      if (ok) item = items.next_warp(it, lane);
    }
    ptx::mma_commit_warp(bar(kDqDrain));
    wait_bounded(bar(kDqDrain), 0, abort_flag, p.timeout_ns, false);  // every MMA is done
    __syncwarp();
  } else if (warp < kSoftmaxWarp0) {
    // ------------------------------------------------ check of the masked tiles (warps 2-3)
    // A hidden pair has dS = 0, and 0 * NaN in dS K would carry a non-finite element of
    // its key to a query that does not see it. Once S has been formed, the tile's
    // rows past the sequence's end and its non-finite elements are set to 0; the
    // queries that see such a key get NaN in that column through `poison`, the first key
    // that has one there. An item's epilogue clears it; only then are the next item's put
    // in.
    if constexpr (kCheck) {
      const int tid = static_cast<int>(threadIdx.x) - 64;
      int accs = 0, tile = 0, k_base = 0, m = 0;  // accs: accumulators of the items before this one
      bool ok = true;
      for (int item = static_cast<int>(blockIdx.x), it = 0; ok && item >= 0; ++it) {
        const DqItem w = dq_item<kCausal, kVarlen>(p, item);
        const Seq& s = w.s;
        for (int j = max(0, w.first_masked - w.t0); j < w.n; ++j, ++m) {
          ok = wait_bounded(bar(kDqLanded + m % kDqChecks), (m / kDqChecks) & 1, abort_flag, p.timeout_ns,
                            true) &&
               wait_bounded(bar(kDqSFull + ((tile + j) & 1)), ((tile + j) >> 1) & 1, abort_flag, p.timeout_ns,
                            true);
          ok = !ptx::named_barrier_or(1, 64, !ok);
          if (!ok) break;
          const uint32_t kt = sbase + kDqOffK + ((k_base + k_fill(j)) % kDqKStages) * kTileBytes;
          const int first = (w.t0 + j) * kTile;
          bool dirty = false;
          for (int r = tid; r < kTile; r += 64) {
            if (first + r >= s.sk) {
              if (kVarlen) {  // (a dense tile's rows past the end are zero already)
                zero_row(kt, r);
                dirty = true;
              }
              continue;
            }
            uint32_t acc = 0;
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const uint4 x = ptx::ld_shared_v4(kt + chunk_at(r, c));
              acc = ptx::bf16x2_nonfinite_acc(x.x, ptx::bf16x2_nonfinite_acc(x.y, acc));
              acc = ptx::bf16x2_nonfinite_acc(x.z, ptx::bf16x2_nonfinite_acc(x.w, acc));
            }
            if (acc != 0) {
              // (Past the item's first kAccTiles the last one's epilogue is long over.)
              if (accs > 0 && (!kLong || j < kAccTiles))
                wait_bounded(bar(kDqAccFree), (accs - 1) & 1, abort_flag, p.timeout_ns, true);
              clean_row(kt, r, [&](int col) {
                atomicMin(&poison[col], first + r);
                *static_cast<volatile int*>(poison + kD) = 1;
              });
              dirty = true;
            }
          }
          if (dirty) ptx::fence_proxy_async_smem();
          __syncwarp();
          ptx::named_barrier_sync(1, 64);
          if (tid == 0) ptx::mbar_arrive(bar(kDqChecked + m % kDqChecks));
        }
        if (w.n > 0) {
          tile += w.n;
          k_base += w.n + 1;
          accs += accumulators<kLong>(w.n);
        }
        if (ok) item = next_together(items, it, lane);
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax
    const int g = (warp - kSoftmaxWarp0) >> 2;  // 64-key half of the tile
    const int wq = warp & 3;
    const int row = wq * 32 + lane;             // query within the tile
    const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tPh = tP + lane_base + 64 * g;
    const uint64_t c2 = ptx::f2_pack(p.c, p.c);
    Meeting all{bar(kDqMeet), abort_flag, p.timeout_ns, 0};
    int used = 0, tile = 0, k_base = 0, accs = 0;
    bool ok = true;
    // The row's log-sum-exp is read when the item is known, long before it is used.
    auto read_lse = [&](const DqItem& w) -> float {
      if (w.n == 0 || w.q0 + row >= w.s.sq) return -__int_as_float(0x7F800000);
      return __ldg(p.lse + (kVarlen ? static_cast<size_t>(w.s.head) * p.Sq + w.s.q_base + w.q0 + row
                                    : (static_cast<size_t>(w.s.batch) * p.Hq + w.s.head) * p.Sq + w.q0 + row));
    };
    int item = static_cast<int>(blockIdx.x);
    DqItem w = dq_item<kCausal, kVarlen>(p, item);
    float lse = read_lse(w);
    for (int it = 0; ok && item >= 0; ++it) {
      const int n = w.n;
      // Keys this row sees, counted from the part's first.
      const int limit = (kCausal ? min(w.q0 + row + w.off + 1, w.s.sk) : w.s.sk) - w.t0 * kTile;
      const int first_masked = w.first_masked - w.t0;
      uint64_t nl2 = 0, nd2 = 0;
      if (n > 0) {
        const Seq& s = w.s;
        // The row's statistics: each warpgroup adds its 64 columns of dO O.
        float dot = 0.f;
        const int fo = k_base, os = fo % kDqKStages;
        ok = warp_wait(bar(kDqQ), used & 1, abort_flag, p.timeout_ns) &&
             warp_wait(bar(kDqKFull + os), (fo / kDqKStages) & 1, abort_flag, p.timeout_ns);
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint4 x = ptx::ld_shared_v4(sbase + kDqOffO + chunk_at(row, 8 * g + c));
          const uint4 y = ptx::ld_shared_v4(sbase + kDqOffK + os * kTileBytes + chunk_at(row, 8 * g + c));
          const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            dot = fmaf(__uint_as_float(xs[e] << 16), __uint_as_float(ys[e] << 16), dot);
            dot = fmaf(__uint_as_float(xs[e] & 0xFFFF0000u), __uint_as_float(ys[e] & 0xFFFF0000u), dot);
          }
        }
        ptx::fence_proxy_async_smem();  // these reads, before the stage is refilled
        float* dots = reinterpret_cast<float*>(smem + kDqOffDots);
        dots[g * kTile + row] = dot;
        if (!(ok = all.meet(lane))) break;
        dot = dots[row] + dots[kTile + row];
        if (threadIdx.x == 32 * kSoftmaxWarp0) {  // O and dO have been read
          ptx::mbar_arrive(bar(kDqKEmpty + os));
          ptx::mbar_arrive(bar(kDqQFree));
        }
        float nl = -__int_as_float(0x7F800000), nd = 0.f;
        if (lse != -__int_as_float(0x7F800000)) {
          nl = -lse * 1.4426950408889634f;
          nd = isfinite(dot) ? -dot : __int_as_float(0x7FC00000);
        } else if (w.q0 + row < s.sq && limit + w.t0 * kTile > 0) {
          nl = nd = __int_as_float(0x7FC00000);  // it sees keys, and every logit is -Inf
        }
        if (g == 0 && s.split == 0) {
          float* st = p.stats + (static_cast<size_t>(s.slot_q) + static_cast<size_t>(s.head) * p.q_slots +
                                 s.tile) * kStatFloats;
          st[row] = nl;
          st[kTile + row] = nd;
        }
        nl2 = ptx::f2_pack(nl, nl);
        nd2 = ptx::f2_pack(nd, nd);
      }
      int j = 0;
      do {
        const int end = kLong ? min(n, j + kAccTiles) : n;
        for (; j < end; ++j, ++tile) {
          const uint32_t tSh = tmem + 128 * (tile & 1) + lane_base + 64 * g;
          const int hi = limit - j * kTile - 64 * g;  // columns of this half the row sees
          Half pr;
          if (!(ok = warp_wait(bar(kDqSFull + (tile & 1)), (tile >> 1) & 1, abort_flag, p.timeout_ns))) break;
          ptx::tc_fence_after();
          by_halves(tSh, [&](int ch, const uint32_t (&r)[32]) {
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              float e0, e1;
              ptx::f2_unpack(ptx::f2_fma(pair_of(r, 2 * x), c2, nl2), e0, e1);
              pr[16 * ch + x] = ptx::f2_pack(ptx::ex2(e0), ptx::ex2(e1));
            }
          });
          if (!(ok = warp_wait(bar(kDqDpFull), tile & 1, abort_flag, p.timeout_ns))) break;
          ptx::tc_fence_after();
          if (j >= first_masked)
            dq_ds<true>(tPh, tSh, nd2, hi, pr);
          else
            dq_ds<false>(tPh, tSh, nd2, hi, pr);
          ptx::tmem_wait_st();
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar(kDqDsFull));
        }
        if (!ok) break;
        // ---- epilogue: each warpgroup stores 64 columns of the rows, or adds them to the item's
        // terms. (The next item is taken up before the wait.)
        const bool zero = n == 0, last = !kLong || j == n;
        const DqItem v = w;
        if (last) {
          item = items.next_warp(it, lane);
          if (item >= 0) {
            w = dq_item<kCausal, kVarlen>(p, item);
            lse = read_lse(w);
          }
        }
        if (!zero && !(ok = warp_wait(bar(kDqAcc), (kLong ? accs : used) & 1, abort_flag, p.timeout_ns))) break;
        ptx::tc_fence_after();
        if (!v.skip) {
          const Seq& s = v.s;
          const uint32_t tacc = tQ + lane_base + 64 * g;
          const bool any = kCheck && !zero && last && *static_cast<volatile int*>(poison + kD);
          const int sees = kCausal ? min(v.q0 + row + v.off + 1, s.sk) : s.sk;
          auto is_nan = [&](int col) -> bool { return any && poison[64 * g + col] < sees; };
          auto terms = [&]() -> float4* {
            const size_t slots = static_cast<size_t>(p.q_slots) * (kVarlen ? p.Hq : p.BH);
            const size_t slot = static_cast<size_t>(s.slot_q) + static_cast<size_t>(s.head) * p.q_slots + s.tile;
            return reinterpret_cast<float4*>(
                       p.part + (static_cast<size_t>(s.split) * slots + slot) * kTile * kD) + 16 * g * kTile + row;
          };
          if (last && p.n_splits == 1) {
            const int first = v.q0 + 32 * wq;  // of the warp's rows
            const int rows = dbg_ok(s.q_base + s.sq <= p.Sq) ? s.sq - first : 0;
            uint16_t* dst =
                p.dq + row_at(p.layout, s.batch, p.Hq, p.Sq, s.head, s.q_base + (rows > 0 ? first : 0)) + 64 * g;
            store_rows<64>(tacc, zero, p.scale, p.mode, dst, static_cast<size_t>(p.layout == 0 ? 1 : p.Hq) * kD, rows,
                           lane, kLong && n > kAccTiles ? terms() : nullptr, any, is_nan);
          } else {
            store_part<64>(tacc, zero, terms(), kLong && j > kAccTiles, is_nan);
          }
          if (any && !(ok = clear_poison(poison, kNever, all, lane))) break;
        }
        if (!zero) {
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar(kDqAccFree));
          if (kLong) ++accs;
          if (last) {
            k_base += n + 1;
            ++used;
          }
        }
      } while (kLong && j < n);
      // (The loop ends by its condition too. With this the compiler's order of the masked forms
      // is the faster one, causal 4K 321 -> 313 us, and that of the unmasked one 1% slower.)
      if (kCheck && !ok) break;
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
  // A CTA leaves only after the kernel before it on the stream has finished, so
  // that this grid's end is the end of both.
  ptx::grid_dependency_wait();
}

// ---------------------------------------------------------------- join of the splits
//
// A result owned by n_splits CTAs: their fp32 terms are added in split order, scaled
// and rounded. One block per 16 rows of a tile, eight columns a thread. Both kernels' results
// in one launch after both (a join of its own between them held up the second one).
struct JoinPart {
  const float* part;
  uint16_t* out[2];  // dq, or dk and dv
  float factor[2];
  const int* cu;     // packed batch: the owned axis's offsets
  const int* cu2;    // and the other axis's (a sequence with bad offsets is left alone)
  int S, S2, H, max_s, max_s2, slots, n_tiles, n_splits, results;
};
struct JoinParams {
  JoinPart dq, dkv;
  int dq_blocks;     // the grid's first blocks: dq
  int B, layout, mode;
};

constexpr int kJoinRows = 16;

template <bool kVarlen>
__device__ __forceinline__ void join_rows(const JoinPart& j, int B, int layout, int mode, int block) {
  constexpr int kPer = kTile / kJoinRows;  // blocks per tile
  const int r = (block % kPer) * kJoinRows + (threadIdx.x % kJoinRows);
  int item = block / kPer;
  const int tile = item % j.n_tiles;
  item /= j.n_tiles;
  const int h = item % j.H;
  item /= j.H;
  const int b = item % B, result = item / B;
  ptx::grid_dependency_wait();
  int base = 0, len = j.S, batch = b;
  size_t slot = (static_cast<size_t>(b) * j.H + h) * j.slots + tile;
  if (kVarlen) {
    base = __ldg(j.cu + b);
    len = packed_len(base, __ldg(j.cu + b + 1), j.max_s, j.S);
    if (len < 0 || packed_len(__ldg(j.cu2 + b), __ldg(j.cu2 + b + 1), j.max_s2, j.S2) < 0) return;
    batch = 0;
    slot = static_cast<size_t>(h) * j.slots + tile_slot<true>(base, b) + tile;
  }
  const int row = tile * kTile + r;
  if (row >= len) return;
  const size_t slots = static_cast<size_t>(j.slots) * j.H * (kVarlen ? 1 : B);
  const int c0 = threadIdx.x / kJoinRows * 8;
  float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int k = 0; k < j.n_splits; ++k) {
    const float4* src = reinterpret_cast<const float4*>(
        j.part + ((static_cast<size_t>(k) * j.results + result) * slots + slot) * kTile * kD);
    const float4 u = src[c0 / 4 * kTile + r], v = src[(c0 / 4 + 1) * kTile + r];
    x[0] += u.x; x[1] += u.y; x[2] += u.z; x[3] += u.w;
    x[4] += v.x; x[5] += v.y; x[6] += v.z; x[7] += v.w;
  }
  const float f = result ? j.factor[1] : j.factor[0];
  uint16_t* out = result ? j.out[1] : j.out[0];
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = round_bf16_bits(x[2 * i] * f, mode) | (round_bf16_bits(x[2 * i + 1] * f, mode) << 16);
  *reinterpret_cast<uint4*>(out + row_at(layout, batch, j.H, j.S, h, base + row) + c0) =
      make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool kVarlen>
__global__ void __launch_bounds__(16 * kJoinRows) attn_bwd_join(const JoinParams p) {
  const int block = static_cast<int>(blockIdx.x);
  if (block < p.dq_blocks)
    join_rows<kVarlen>(p.dq, p.B, p.layout, p.mode, block);
  else
    join_rows<kVarlen>(p.dkv, p.B, p.layout, p.mode, block - p.dq_blocks);
}

}  // namespace bwd
}  // namespace attn
