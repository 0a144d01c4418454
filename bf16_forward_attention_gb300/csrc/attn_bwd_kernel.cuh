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
//
// Both kernels: 384 threads. Warp 0: TMA producer. Warp 1: TMEM allocation and
// the tcgen05.mma issue (one elected lane, in warp-uniform code). Warps 2-3: check of the tiles where some pairs
// are hidden (see check_rows / check_keys). Warps 4-7 and 8-11: softmax, each
// thread one TMEM lane (a key in dkv, a query in dq) and one 64-column half.
// Every wait is bounded, as in the forward kernel.
#pragma once
#include "attn_fwd_kernel.cuh"

namespace attn {
namespace bwd {

constexpr int kTile = 128;             // queries and keys per tile
constexpr int kStatFloats = 2 * kTile; // per query tile: 128 of -lse log2(e), 128 of -D

struct BwdParams {
  int Sq, Sk;              // per batch entry, or packed totals
  int Hq, Hkv, group;      // group = Hq / Hkv
  int BH;                  // heads of the grid: B * Hq (dq) or B * Hkv (dkv)
  int n_tiles;             // tiles of the owned axis per head (grid)
  int head_group;          // heads scheduled together (causal: longest first)
  int n_splits;            // CTAs per owned tile, each over a part of the streamed tiles
  int layout, mode;
  float c, scale;          // c = scale * log2(e)
  unsigned long long timeout_ns;
  const int* cu_q;         // packed batch: B + 1 offsets each (else null)
  const int* cu_k;
  int max_sq, max_sk;
  int q_slots, k_slots;    // tile slots per head (see tile_slot)
  const float* lse;
  float* stats;            // [head][slot][2][128]: written by dq, read by dkv
  float* part;             // n_splits > 1: [split][result][head * slots][128][128] fp32
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
  s.split = block % p.n_splits;
  const int item = block / p.n_splits;
  const int span = p.n_tiles * p.head_group;
  const int g = item / span, r = item - g * span;
  const int gs = min(p.head_group, p.BH - g * p.head_group);
  const int t = r / gs;
  const int bh = g * p.head_group + r % gs;
  // Longest ranges first under the causal mask: late queries see most keys, early
  // keys are seen by most queries.
  s.tile = (kOwnQ && kCausal) ? p.n_tiles - 1 - t : t;
  const int H = kOwnQ ? p.Hq : p.Hkv;
  const int b = bh / H;
  s.head = bh % H;
  s.bad = false;
  if (kVarlen) {
    s.q_base = __ldg(p.cu_q + b);
    s.sq = __ldg(p.cu_q + b + 1) - s.q_base;
    s.k_base = __ldg(p.cu_k + b);
    s.sk = __ldg(p.cu_k + b + 1) - s.k_base;
    s.bad = s.q_base < 0 || s.sq < 0 || s.sq > p.max_sq || s.q_base + s.sq > p.Sq || s.k_base < 0 ||
            s.sk < 0 || s.sk > p.max_sk || s.k_base + s.sk > p.Sk;
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

// Part `split` of n streamed tiles: [first, first + count).
__device__ __forceinline__ void part_of(int n, int splits, int split, int& first, int& count) {
  const int base = n / splits, rem = n % splits;
  first = split * base + min(split, rem);
  count = base + (split < rem ? 1 : 0);
}

// 64 columns of a TMEM row as 32 packed pairs of fp32.
using Half = uint64_t[32];

__device__ __forceinline__ void load_half(uint32_t taddr, uint32_t (&a)[32], uint32_t (&b)[32]) {
  ptx::tmem_ld32_nowait(taddr, a);
  ptx::tmem_ld32_nowait(taddr + 32, b);
  ptx::tmem_wait_ld32(a);
  ptx::reg_fence32(b);
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

// kCols finished columns of a row of a result in TMEM -> bf16 in global memory (dst null:
// a row past the end; its lane still takes part in the loads). A thread holds one row,
// so its stores are 16 bytes of consecutive addresses each and need no staging.
// `poison(col)`: the column is NaN; any: there is such a column. zero: no product
// was formed, the result is 0.
template <int kCols, typename F>
__device__ __forceinline__ void store_row(uint32_t tacc, bool zero, float factor, int mode, uint16_t* dst,
                                          bool any, F poison) {
  const uint64_t f2 = ptx::f2_pack(factor, factor);
  const uint32_t bias = mode == 1 ? 0x8000u : 0u;
#pragma unroll
  for (int ch = 0; ch < kCols / 32; ++ch) {
    uint32_t r[32];
    if (!zero) {
      ptx::tmem_ld32(tacc + 32 * ch, r);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) r[i] = 0;
    }
    if (any) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (poison(32 * ch + i)) r[i] = 0x7FC00000u;
    }
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float x0, x1;
      ptx::f2_unpack(ptx::f2_mul(ptx::f2_pack(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), f2),
                     x0, x1);
      w[i] = mode == 0 ? round_pair_bf16_rtne(x0, x1) : round_pair_bf16(x0, x1, bias);
    }
    if (dst) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        reinterpret_cast<uint4*>(dst)[4 * ch + u] = make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
    }
  }
}

// The same row as fp32 into the split workspace (one of n_splits terms of a sum).
template <int kCols, typename F>
__device__ __forceinline__ void store_part(uint32_t tacc, bool zero, float* dst, F poison) {
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
      *reinterpret_cast<float4*>(dst + 16 * ch + i) = make_float4(x[0], x[1], x[2], x[3]);
    }
  }
}

// The softmax threads' turns, over 64 columns each. kMask is a template argument:
// as a run-time test inside, its compares ran in every tile (half of the
// instructions of the unmasked loop).
__device__ __forceinline__ uint64_t pair_of(const uint32_t (&r)[32], int x) {
  return ptx::f2_pack(__uint_as_float(r[x]), __uint_as_float(r[x + 1]));
}

// dkv: P from S (a lane's key against 64 queries, whose -lse log2(e) are in shared
// memory); kept in pr, and written over S as bf16.
template <bool kMask>
__device__ __forceinline__ void dkv_p(uint32_t tS, const ulonglong2* stat, uint64_t c2, int lo, int hi,
                                      Half& pr) {
  uint32_t a[32], b[32];
  load_half(tS, a, b);
#pragma unroll
  for (int ch = 0; ch < 2; ++ch) {
    uint32_t w[16];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const ulonglong2 nl = stat[8 * ch + e];  // four columns
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int x = 4 * e + 2 * u;
        float t0, t1;
        ptx::f2_unpack(ptx::f2_fma(pair_of(ch ? b : a, x), c2, u ? nl.y : nl.x), t0, t1);
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
  }
}

// dkv: dS from dP and P, written over dP as bf16.
template <bool kMask>
__device__ __forceinline__ void dkv_ds(uint32_t tP, const ulonglong2* stat, int lo, int hi, const Half& pr) {
  uint32_t a[32], b[32];
  load_half(tP, a, b);
#pragma unroll
  for (int ch = 0; ch < 2; ++ch) {
    uint32_t w[16];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const ulonglong2 nd = stat[32 + 8 * ch + e];  // four columns of -D
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int x = 4 * e + 2 * u;
        float s0, s1;
        ptx::f2_unpack(
            ptx::f2_mul(pr[16 * ch + 2 * e + u], ptx::f2_add(pair_of(ch ? b : a, x), u ? nd.y : nd.x)), s0, s1);
        if (kMask) {
          const int col = 32 * ch + x;
          if (col < lo || col >= hi) s0 = 0.f;
          if (col + 1 < lo || col + 1 >= hi) s1 = 0.f;
        }
        w[2 * e + u] = ptx::pack_bf16x2(s0, s1);
      }
    }
    ptx::tmem_st16(tP + 16 * ch, w);
  }
}

// dq: dS from dP and P (a lane's query against 64 keys), written over S as bf16.
template <bool kMask>
__device__ __forceinline__ void dq_ds(uint32_t tP, uint32_t tS, uint64_t nd2, int hi, const Half& pr) {
  uint32_t a[32], b[32];
  load_half(tP, a, b);
#pragma unroll
  for (int ch = 0; ch < 2; ++ch) {
    uint32_t w[16];
#pragma unroll
    for (int x = 0; x < 16; ++x) {
      float s0, s1;
      ptx::f2_unpack(ptx::f2_mul(pr[16 * ch + x], ptx::f2_add(pair_of(ch ? b : a, 2 * x), nd2)), s0, s1);
      if (kMask) {
        if (32 * ch + 2 * x >= hi) s0 = 0.f;
        if (32 * ch + 2 * x + 1 >= hi) s1 = 0.f;
      }
      w[x] = ptx::pack_bf16x2(s0, s1);
    }
    ptx::tmem_st16(tS + 16 * ch, w);
  }
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
// subtract-multiplies.
constexpr int kDkvStages = 2;
enum : int {
  kDkvKV = 0,
  kDkvQFull,
  kDkvQEmpty = kDkvQFull + kDkvStages,
  kDkvOFull = kDkvQEmpty + kDkvStages,
  kDkvOEmpty = kDkvOFull + kDkvStages,
  kDkvSFull = kDkvOEmpty + kDkvStages,
  kDkvPFull,
  kDkvDpFull,
  kDkvDsFull,
  kDkvAcc,
  kDkvLanded,
  kDkvChecked,
  kDkvDrain,
  kDkvBars
};
constexpr int kDkvOffK = 0, kDkvOffV = kTileBytes, kDkvOffQ = 2 * kTileBytes,
              kDkvOffO = kDkvOffQ + kDkvStages * kTileBytes,
              kDkvOffStats = kDkvOffO + kDkvStages * kTileBytes,
              kDkvOffPoison = kDkvOffStats + kDkvStages * kStatFloats * 4,
              kDkvOffBar = kDkvOffPoison + kD * 4 + 16, kDkvOffSlot = kDkvOffBar + kDkvBars * 8,
              kDkvSmem = kDkvOffSlot + 8 + 1024;
static_assert(kDkvSmem <= 232448, "shared memory budget (dkv)");

// The streamed tiles of a CTA: `per` query tiles from first_qt on, for each query
// head of the group.
struct DkvRange {
  int first_qt, per, t0, n;
};
template <bool kCausal>
__device__ __forceinline__ DkvRange dkv_range(const BwdParams& p, const Seq& s) {
  DkvRange r;
  const int nqt = (s.sq + kTile - 1) / kTile;
  r.first_qt = 0;
  if (kCausal) r.first_qt = min(max(0, s.tile * kTile - (s.sk - s.sq)) / kTile, nqt);
  r.per = nqt - r.first_qt;
  part_of(r.per * p.group, p.n_splits, s.split, r.t0, r.n);
  return r;
}

template <bool kCausal, bool kVarlen>
__global__ void __launch_bounds__(kThreads, 1)
    attn_bwd_dkv(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                 const BwdParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kDkvOffSlot);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kDkvOffSlot + 4);
  int* poison_q = reinterpret_cast<int*>(smem + kDkvOffPoison);
  volatile int* poison_any = poison_q + kD;
  auto bar = [&](int i) -> uint32_t { return sbase + kDkvOffBar + 8u * static_cast<uint32_t>(i); };
  // (Through a shuffle, so that the compiler knows it to be the same on every lane.)
  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  constexpr bool kCheck = kCausal || kVarlen;

  const Seq s = seq_of<kCausal, kVarlen, false>(p, static_cast<int>(blockIdx.x));
  if (kVarlen) {
    if (s.bad) {
      if (threadIdx.x == 0) atomicOr(&g_attn_status, 2u);
      ptx::grid_dependency_wait();
      return;
    }
    if (s.tile * kTile >= s.sk) {
      ptx::grid_dependency_wait();
      return;
    }
  }
  const DkvRange rg = dkv_range<kCausal>(p, s);
  const int off = s.sk - s.sq;   // key j is visible to query i iff j <= i + off (causal)
  const int k0 = s.tile * kTile; // first key of the tile
  // A tile some of whose pairs are hidden: crossed by the diagonal, or past the end.
  auto masked = [&](int q0) -> bool {
    return q0 + kTile > s.sq || (kCausal && q0 + off < k0 + kTile - 1);
  };

  if (threadIdx.x == 0) {
    for (int i = 0; i < kDkvBars; ++i)
      ptx::mbar_init(bar(i), (i == kDkvPFull || i == kDkvDsFull) ? 8 : 1);
    *abort_flag = 0;
    *poison_any = 0;
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
  }
  if (threadIdx.x < kD) poison_q[threadIdx.x] = -1;
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
  const uint32_t tS = tmem, tP = tmem + 128, tK = tmem + 256, tV = tmem + 384;

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    if (lane == 0 && rg.n > 0) {
      const uint64_t pol_once = ptx::l2_policy_evict_first();
      const uint64_t pol_reuse = ptx::l2_policy_evict_last();
      dbg_ok(s.k_base + k0 < p.Sk);
      ptx::mbar_arrive_expect_tx(bar(kDkvKV), 2 * kTileBytes);
      load_tile(sbase + kDkvOffK, &tm_k, bar(kDkvKV), p.layout, s.k_base + k0, s.head, s.batch, pol_once);
      load_tile(sbase + kDkvOffV, &tm_v, bar(kDkvKV), p.layout, s.k_base + k0, s.head, s.batch, pol_once);
      ptx::grid_dependency_wait();  // the row statistics
      int q_issued = 0, o_issued = 0;
      for (int i = 0; i < rg.n; ++i) {
        const int st = i % kDkvStages;
        const uint32_t par = ((i / kDkvStages) & 1) ^ 1;
        const int t = rg.t0 + i;
        const int h = s.head * p.group + t / rg.per;
        const int qt = rg.first_qt + t % rg.per;
        dbg_ok(s.q_base + qt * kTile < p.Sq && h < p.Hq);
        if (!wait_bounded(bar(kDkvQEmpty + st), par, abort_flag, p.timeout_ns, true)) break;
        ptx::mbar_arrive_expect_tx(bar(kDkvQFull + st), kTileBytes + kStatFloats * 4);
        load_tile(sbase + kDkvOffQ + st * kTileBytes, &tm_q, bar(kDkvQFull + st), p.layout,
                  s.q_base + qt * kTile, h, s.batch, pol_reuse);
        const float* src = p.stats + (static_cast<size_t>(s.slot_q) + static_cast<size_t>(h) * p.q_slots + qt) *
                                         kStatFloats;
        ptx::bulk_load(sbase + kDkvOffStats + st * kStatFloats * 4, src, kStatFloats * 4,
                       bar(kDkvQFull + st));
        ++q_issued;
        if (!wait_bounded(bar(kDkvOEmpty + st), par, abort_flag, p.timeout_ns, true)) break;
        ptx::mbar_arrive_expect_tx(bar(kDkvOFull + st), kTileBytes);
        load_tile(sbase + kDkvOffO + st * kTileBytes, &tm_do, bar(kDkvOFull + st), p.layout,
                  s.q_base + qt * kTile, h, s.batch, pol_reuse);
        ++o_issued;
      }
      // Every copy this thread started lands before the CTA can exit.
      wait_bounded(bar(kDkvKV), 0, abort_flag, p.timeout_ns, false);
      for (int st = 0; st < kDkvStages; ++st) {
        if (st < q_issued)
          wait_bounded(bar(kDkvQFull + st), ((q_issued - 1 - st) / kDkvStages) & 1, abort_flag,
                       p.timeout_ns, false);
        if (st < o_issued)
          wait_bounded(bar(kDkvOFull + st), ((o_issued - 1 - st) / kDkvStages) & 1, abort_flag,
                       p.timeout_ns, false);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer (whole warp)
    if (rg.n > 0) {
      const uint32_t k_desc = desc_lo(sbase + kDkvOffK, 16), v_desc = desc_lo(sbase + kDkvOffV, 16);
      auto q_tile = [&](int i) -> uint32_t { return sbase + kDkvOffQ + (i % kDkvStages) * kTileBytes; };
      auto o_tile = [&](int i) -> uint32_t { return sbase + kDkvOffO + (i % kDkvStages) * kTileBytes; };
      auto wait = [&](int b, uint32_t par) -> bool {
        const bool r = warp_wait(bar(b), par & 1, abort_flag, p.timeout_ns);
        ptx::tc_fence_after();
        return r;
      };
      int checks = 0;
      // S_i: Q_i has landed; a masked tile's rows have been checked first (both of
      // its tiles, so dO_i has landed too).
      auto do_s = [&](int i) -> bool {
        if (!wait(kDkvQFull + i % kDkvStages, i / kDkvStages)) return false;
        if (kCheck && masked((rg.first_qt + (rg.t0 + i) % rg.per) * kTile)) {
          if (!wait(kDkvOFull + i % kDkvStages, i / kDkvStages)) return false;
          if (lane == 0) ptx::mbar_arrive(bar(kDkvLanded));
          if (!wait(kDkvChecked, checks)) return false;
          ++checks;
        }
        issue_s(tS, k_desc, desc_lo(q_tile(i), 16));
        ptx::mma_commit_warp(bar(kDkvSFull));
        return true;
      };
      auto do_dp = [&](int i) -> bool {
        if (!wait(kDkvOFull + i % kDkvStages, i / kDkvStages)) return false;
        issue_s(tP, v_desc, desc_lo(o_tile(i), 16));
        ptx::mma_commit_warp(bar(kDkvDpFull));
        return true;
      };
      bool ok = wait(kDkvKV, 0) && do_s(0) && do_dp(0);
      for (int i = 0; ok && i < rg.n; ++i) {
        const bool more = i + 1 < rg.n;
        if (!(ok = wait(kDkvPFull, i))) break;
        issue_second(tV, tS, desc_lo(o_tile(i), kHalfBytes), i > 0);
        ptx::mma_commit_warp(bar(kDkvOEmpty + i % kDkvStages));
        if (more && !(ok = do_s(i + 1))) break;
        if (!(ok = wait(kDkvDsFull, i))) break;
        issue_second(tK, tP, desc_lo(q_tile(i), kHalfBytes), i > 0);
        ptx::mma_commit_warp(bar(kDkvQEmpty + i % kDkvStages));
        if (more && !(ok = do_dp(i + 1))) break;
      }
      if (ok) ptx::mma_commit_warp(bar(kDkvAcc));
      ptx::mma_commit_warp(bar(kDkvDrain));
      wait_bounded(bar(kDkvDrain), 0, abort_flag, p.timeout_ns, false);
    }
    __syncwarp();
  } else if (warp < kSoftmaxWarp0) {
    // ------------------------------------------------ check of the masked tiles (warps 2-3)
    // A hidden pair has P = dS = 0, and 0 * NaN in the second products would carry a
    // non-finite element of its Q or dO row to keys that do not see it. Rows that
    // take no part (past the sequence's end, or seeing no key) are set to 0. A row
    // with a non-finite element has a NaN among its statistics; its non-finite
    // elements are set to 0 as well. The keys that do see it still get NaN: in
    // every column of dK (and of dV, when it is Q) through the statistics, and in
    // the column of a non-finite dO element through poison_q, the last row that
    // has one there.
    if constexpr (kCheck) {
      const int tid = static_cast<int>(threadIdx.x) - 64;
      int m = 0;
      for (int i = 0; i < rg.n; ++i) {
        const int q0 = (rg.first_qt + (rg.t0 + i) % rg.per) * kTile;
        if (!masked(q0)) continue;
        const bool ok = wait_bounded(bar(kDkvLanded), m & 1, abort_flag, p.timeout_ns, true);
        if (ptx::named_barrier_or(1, 64, !ok)) break;
        ++m;
        const int st = i % kDkvStages;
        const uint32_t qt = sbase + kDkvOffQ + st * kTileBytes, ot = sbase + kDkvOffO + st * kTileBytes;
        const float* stat = reinterpret_cast<const float*>(smem + kDkvOffStats) + st * kStatFloats;
        bool dirty = false;
        for (int r = tid; r < kTile; r += 64) {
          const float nl = stat[r], nd = stat[kTile + r];
          const bool past = q0 + r >= s.sq;  // (zero already in a dense tensor's tile)
          if (past && !kVarlen) continue;
          if (past || nl == -__int_as_float(0x7F800000)) {
            zero_row(qt, r);
            zero_row(ot, r);
            dirty = true;
          } else if (isnan(nl) || isnan(nd)) {
            clean_row(qt, r, [](int) {});
            clean_row(ot, r, [&](int col) {
              atomicMax(&poison_q[col], q0 + r);
              *poison_any = 1;
            });
            dirty = true;
          }
        }
        if (dirty) ptx::fence_proxy_async_smem();
        __syncwarp();
        ptx::named_barrier_sync(1, 64);
        if (tid == 0) ptx::mbar_arrive(bar(kDkvChecked));
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
    bool ok = true;
    int q0 = rg.n > 0 ? (rg.first_qt + rg.t0 % rg.per) * kTile : 0;  // the tile's first query
    const int q_last = (rg.first_qt + rg.per - 1) * kTile;           // of a head
    for (int i = 0; i < rg.n; ++i, q0 = q0 == q_last ? rg.first_qt * kTile : q0 + kTile) {
      const bool mk = masked(q0);
      // The columns of this half that this key is visible to: [lo, hi).
      const int lo = kCausal ? k0 + row - off - q0 - 64 * g : 0;
      const int hi = s.sq - q0 - 64 * g;
      const ulonglong2* stat = reinterpret_cast<const ulonglong2*>(
          smem + kDkvOffStats + (i % kDkvStages) * kStatFloats * 4 + 256 * g);
      Half pr;
      if (!(ok = warp_wait(bar(kDkvSFull), i & 1, abort_flag, p.timeout_ns))) break;
      // (Q's barrier, for the statistics that landed with it: long complete.)
      if (!(ok = warp_wait(bar(kDkvQFull + i % kDkvStages), (i / kDkvStages) & 1, abort_flag,
                           p.timeout_ns)))
        break;
      ptx::tc_fence_after();
      if (mk)
        dkv_p<true>(tSh, stat, c2, lo, hi, pr);
      else
        dkv_p<false>(tSh, stat, c2, lo, hi, pr);
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(kDkvPFull));

      if (!(ok = warp_wait(bar(kDkvDpFull), i & 1, abort_flag, p.timeout_ns))) break;
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
    // ---- epilogue: warpgroup 0 stores dK, warpgroup 1 dV.
    if (ok && rg.n > 0) ok = warp_wait(bar(kDkvAcc), 0, abort_flag, p.timeout_ns);
    if (ok) {
      ptx::tc_fence_after();
      const uint32_t tacc = (g == 0 ? tK : tV) + lane_base;
      const bool zero = rg.n == 0;
      // The last query row whose non-finite dO element a key may see (see above).
      const int seen = kCausal ? max(0, k0 + row - off) : 0;
      auto poison = [&](int col) -> bool { return kCheck && g == 1 && poison_q[col] >= seen; };
      if (p.n_splits == 1) {
        const bool in = k0 + row < s.sk && dbg_ok(s.k_base + k0 + row < p.Sk);
        uint16_t* dst = (g == 0 ? p.dk : p.dv) +
                        row_at(p.layout, s.batch, p.Hkv, p.Sk, s.head, s.k_base + k0 + (in ? row : 0));
        store_row<kD>(tacc, zero, g == 0 ? p.scale : 1.f, p.mode, in ? dst : nullptr,
                      kCheck && g == 1 && *poison_any, poison);
      } else {
        const size_t slots = static_cast<size_t>(p.k_slots) * (kVarlen ? p.Hkv : p.BH);
        const size_t slot = static_cast<size_t>(s.slot_k) + static_cast<size_t>(s.head) * p.k_slots + s.tile;
        float* dst = p.part + (((static_cast<size_t>(s.split) * 2 + g) * slots + slot) * kTile + row) * kD;
        store_part<kD>(tacc, zero, dst, poison);
      }
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
// dS once dP_{j+1} is there) has 1536 tensor cycles.
//
// It also leaves the row statistics that dkv reads: per query row -lse log2(e) and -D,
// D = sum_c dO_ic O_ic, formed from the dO tile it has and the O tile, which passes
// through K's third stage before that is first needed. (A kernel of its own for them
// read dO once more and cost 25 us of 2.35 ms on 8K self-attention, 47 of 1039 us on a
// packed batch, and a launch.) Rows past the end, and rows that see no key, get -Inf
// and 0 (P = 0). A non-finite D becomes NaN: it marks a row whose dO or O has a
// non-finite element.
constexpr int kDqKStages = 3, kDqVStages = 2;  // K_j is in use while K_{j+2} loads
constexpr int kDqMasked = 2;  // 128 rows' causal limits span at most 127 keys
enum : int {
  kDqQ = 0,
  kDqKFull,
  kDqKEmpty = kDqKFull + kDqKStages,
  kDqVFull = kDqKEmpty + kDqKStages,
  kDqVEmpty = kDqVFull + kDqVStages,
  kDqSFull = kDqVEmpty + kDqVStages,
  kDqDpFull = kDqSFull + 2,
  kDqDsFull,
  kDqAcc,
  kDqOutFull,   // O has landed in K's last stage
  kDqOutRead,   // and has been read
  kDqLanded,
  kDqChecked = kDqLanded + kDqMasked,
  kDqDrain = kDqChecked + kDqMasked,
  kDqBars
};
constexpr int kDqOffQ = 0, kDqOffO = kTileBytes, kDqOffK = 2 * kTileBytes,
              kDqOffV = kDqOffK + kDqKStages * kTileBytes,
              kDqOffPoison = kDqOffV + kDqVStages * kTileBytes, kDqOffDots = kDqOffPoison + kD * 4 + 16,
              kDqOffBar = kDqOffDots + 2 * kTile * 4,
              kDqOffSlot = kDqOffBar + kDqBars * 8, kDqSmem = kDqOffSlot + 8 + 1024;
static_assert(kDqSmem <= 232448, "shared memory budget (dq)");

template <bool kCausal, bool kVarlen>
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
  int* poison_k = reinterpret_cast<int*>(smem + kDqOffPoison);
  volatile int* poison_any = poison_k + kD;
  auto bar = [&](int i) -> uint32_t { return sbase + kDqOffBar + 8u * static_cast<uint32_t>(i); };
  // (Through a shuffle, so that the compiler knows it to be the same on every lane.)
  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  constexpr bool kCheck = kCausal || kVarlen;
  constexpr int kNever = 0x7FFFFFFF;

  const Seq s = seq_of<kCausal, kVarlen, true>(p, static_cast<int>(blockIdx.x));
  if (kVarlen) {
    if (s.bad) {
      if (threadIdx.x == 0) atomicOr(&g_attn_status, 2u);
      ptx::grid_dependency_wait();
      return;
    }
    if (s.tile * kTile >= s.sq) {
      ptx::grid_dependency_wait();
      return;
    }
  }
  const int off = s.sk - s.sq;
  const int q0 = s.tile * kTile;
  // Key tiles any row sees, and of these the first in which some row does not see
  // every key: the causal diagonal, or the ragged last tile.
  int n_kv = (s.sk + kTile - 1) / kTile;
  int first_masked = s.sk / kTile;
  if (kCausal) {
    const int last = min(s.sq, q0 + kTile) - 1 + off + 1;  // keys the last row sees
    n_kv = min(n_kv, last <= 0 ? 0 : (last + kTile - 1) / kTile);
    first_masked = min(first_masked, max(0, q0 + off + 1) / kTile);
  }
  int t0, n;
  part_of(n_kv, p.n_splits, s.split, t0, n);
  auto masked = [&](int j) -> bool { return t0 + j >= first_masked; };
  const int kv_head = s.head / p.group;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kDqBars; ++i) ptx::mbar_init(bar(i), (i == kDqDsFull || i == kDqOutRead) ? 8 : 1);
    *abort_flag = 0;
    *poison_any = 0;
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
  }
  if (threadIdx.x < kD) poison_k[threadIdx.x] = kNever;
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

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    if (lane == 0 && n > 0) {
      const uint64_t pol_once = ptx::l2_policy_evict_first();
      const uint64_t pol_reuse = ptx::l2_policy_evict_last();
      dbg_ok(s.q_base + q0 < p.Sq);
      ptx::mbar_arrive_expect_tx(bar(kDqQ), 2 * kTileBytes);
      load_tile(sbase + kDqOffQ, &tm_q, bar(kDqQ), p.layout, s.q_base + q0, s.head, s.batch, pol_once);
      load_tile(sbase + kDqOffO, &tm_do, bar(kDqQ), p.layout, s.q_base + q0, s.head, s.batch, pol_once);
      constexpr int kOutStage = kDqKStages - 1;
      ptx::mbar_arrive_expect_tx(bar(kDqOutFull), kTileBytes);
      load_tile(sbase + kDqOffK + kOutStage * kTileBytes, &tm_out, bar(kDqOutFull), p.layout, s.q_base + q0,
                s.head, s.batch, pol_once);
      int k_issued = 0, v_issued = 0;
      for (int j = 0; j < n; ++j) {
        const int row = s.k_base + (t0 + j) * kTile;
        dbg_ok(row < p.Sk);
        const int ks = j % kDqKStages, vs = j % kDqVStages;
        if (!wait_bounded(bar(kDqKEmpty + ks), ((j / kDqKStages) & 1) ^ 1, abort_flag, p.timeout_ns, true))
          break;
        if (j == kOutStage && !wait_bounded(bar(kDqOutRead), 0, abort_flag, p.timeout_ns, true)) break;
        ptx::mbar_arrive_expect_tx(bar(kDqKFull + ks), kTileBytes);
        load_tile(sbase + kDqOffK + ks * kTileBytes, &tm_k, bar(kDqKFull + ks), p.layout, row, kv_head,
                  s.batch, pol_reuse);
        ++k_issued;
        if (!wait_bounded(bar(kDqVEmpty + vs), ((j / kDqVStages) & 1) ^ 1, abort_flag, p.timeout_ns, true))
          break;
        ptx::mbar_arrive_expect_tx(bar(kDqVFull + vs), kTileBytes);
        load_tile(sbase + kDqOffV + vs * kTileBytes, &tm_v, bar(kDqVFull + vs), p.layout, row, kv_head,
                  s.batch, pol_reuse);
        ++v_issued;
      }
      wait_bounded(bar(kDqQ), 0, abort_flag, p.timeout_ns, false);
      wait_bounded(bar(kDqOutFull), 0, abort_flag, p.timeout_ns, false);
      for (int st = 0; st < kDqKStages && st < k_issued; ++st)
        wait_bounded(bar(kDqKFull + st), ((k_issued - 1 - st) / kDqKStages) & 1, abort_flag, p.timeout_ns,
                     false);
      for (int st = 0; st < kDqVStages && st < v_issued; ++st)
        wait_bounded(bar(kDqVFull + st), ((v_issued - 1 - st) / kDqVStages) & 1, abort_flag, p.timeout_ns,
                     false);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer (whole warp)
    if (n > 0) {
      const uint32_t q_desc = desc_lo(sbase + kDqOffQ, 16), o_desc = desc_lo(sbase + kDqOffO, 16);
      auto k_tile = [&](int j) -> uint32_t { return sbase + kDqOffK + (j % kDqKStages) * kTileBytes; };
      auto v_tile = [&](int j) -> uint32_t { return sbase + kDqOffV + (j % kDqVStages) * kTileBytes; };
      auto wait = [&](int b, uint32_t par) -> bool {
        const bool r = warp_wait(bar(b), par & 1, abort_flag, p.timeout_ns);
        ptx::tc_fence_after();
        return r;
      };
      const int jm = max(0, first_masked - t0);  // first masked tile of this CTA's part
      auto do_s = [&](int j) -> bool {
        if (!wait(kDqKFull + j % kDqKStages, j / kDqKStages)) return false;
        issue_s(tmem + 128 * (j & 1), q_desc, desc_lo(k_tile(j), 16));
        ptx::mma_commit_warp(bar(kDqSFull + (j & 1)));
        if (kCheck && masked(j) && lane == 0) ptx::mbar_arrive(bar(kDqLanded + (j - jm)));
        return true;
      };
      auto do_dp = [&](int j) -> bool {
        if (!wait(kDqVFull + j % kDqVStages, j / kDqVStages)) return false;
        issue_s(tP, o_desc, desc_lo(v_tile(j), 16));
        ptx::mma_commit_warp(bar(kDqDpFull));
        ptx::mma_commit_warp(bar(kDqVEmpty + j % kDqVStages));
        return true;
      };
      bool ok = wait(kDqQ, 0) && do_s(0) && do_dp(0) && (n == 1 || do_s(1));
      for (int j = 0; ok && j < n; ++j) {
        if (!(ok = wait(kDqDsFull, j))) break;
        if (j + 1 < n && !(ok = do_dp(j + 1))) break;
        if (kCheck && masked(j) && !(ok = wait(kDqChecked + (j - jm), 0))) break;
        issue_second(tQ, tmem + 128 * (j & 1), desc_lo(k_tile(j), kHalfBytes), j > 0);
        ptx::mma_commit_warp(bar(kDqKEmpty + j % kDqKStages));
        if (j + 2 < n && !(ok = do_s(j + 2))) break;
      }
      if (ok) ptx::mma_commit_warp(bar(kDqAcc));
      ptx::mma_commit_warp(bar(kDqDrain));
      wait_bounded(bar(kDqDrain), 0, abort_flag, p.timeout_ns, false);
    }
    __syncwarp();
  } else if (warp < kSoftmaxWarp0) {
    // ------------------------------------------------ check of the masked tiles (warps 2-3)
    // A hidden pair has dS = 0, and 0 * NaN in dS K would carry a non-finite element of
    // its key to a query that does not see it. Once S has been formed, the tile's
    // rows past the sequence's end and its non-finite elements are set to 0; the
    // queries that see such a key get NaN in that column through poison_k, the
    // first key that has one there.
    if constexpr (kCheck) {
      const int tid = static_cast<int>(threadIdx.x) - 64;
      for (int j = max(0, first_masked - t0), m = 0; j < n && m < kDqMasked; ++j, ++m) {
        const bool ok = wait_bounded(bar(kDqLanded + m), 0, abort_flag, p.timeout_ns, true) &&
                        wait_bounded(bar(kDqSFull + (j & 1)), (j >> 1) & 1, abort_flag, p.timeout_ns, true);
        if (ptx::named_barrier_or(1, 64, !ok)) break;
        const uint32_t kt = sbase + kDqOffK + (j % kDqKStages) * kTileBytes;
        const int first = (t0 + j) * kTile;
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
            clean_row(kt, r, [&](int col) {
              atomicMin(&poison_k[col], first + r);
              *poison_any = 1;
            });
            dirty = true;
          }
        }
        if (dirty) ptx::fence_proxy_async_smem();
        __syncwarp();
        ptx::named_barrier_sync(1, 64);
        if (tid == 0) ptx::mbar_arrive(bar(kDqChecked + m));
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax
    const int g = (warp - kSoftmaxWarp0) >> 2;  // 64-key half of the tile
    const int wq = warp & 3;
    const int row = wq * 32 + lane;             // query within the tile
    const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tPh = tP + lane_base + 64 * g;
    // Keys this row sees.
    const int limit = kCausal ? min(q0 + row + off + 1, s.sk) : s.sk;
    const uint64_t c2 = ptx::f2_pack(p.c, p.c);
    bool ok = true;
    uint64_t nl2 = 0, nd2 = 0;
    if (n > 0) {
      // The row's statistics: each warpgroup adds its 64 columns of dO O. (lse is read
      // before the waits, whose time covers its latency.)
      float dot = 0.f, lse = -__int_as_float(0x7F800000);
      if (q0 + row < s.sq)
        lse = __ldg(p.lse + (kVarlen ? static_cast<size_t>(s.head) * p.Sq + s.q_base + q0 + row
                                     : (static_cast<size_t>(s.batch) * p.Hq + s.head) * p.Sq + q0 + row));
      ok = warp_wait(bar(kDqQ), 0, abort_flag, p.timeout_ns) &&
           warp_wait(bar(kDqOutFull), 0, abort_flag, p.timeout_ns);
      if (ok) {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint4 x = ptx::ld_shared_v4(sbase + kDqOffO + chunk_at(row, 8 * g + c));
          const uint4 y =
              ptx::ld_shared_v4(sbase + kDqOffK + (kDqKStages - 1) * kTileBytes + chunk_at(row, 8 * g + c));
          const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            dot = fmaf(__uint_as_float(xs[e] << 16), __uint_as_float(ys[e] << 16), dot);
            dot = fmaf(__uint_as_float(xs[e] & 0xFFFF0000u), __uint_as_float(ys[e] & 0xFFFF0000u), dot);
          }
        }
        // (The stage is refilled by TMA: order these reads before it.)
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(kDqOutRead));
      }
      float* dots = reinterpret_cast<float*>(smem + kDqOffDots);
      dots[g * kTile + row] = dot;
      ptx::named_barrier_sync(2, 256);  // (both warpgroups, whatever their waits said)
      const float D = dots[row] + dots[kTile + row];
      float nl = -__int_as_float(0x7F800000), nd = 0.f;
      if (lse != -__int_as_float(0x7F800000)) {
        nl = -lse * 1.4426950408889634f;
        nd = isfinite(D) ? -D : __int_as_float(0x7FC00000);
      }
      if (g == 0 && s.split == 0) {
        float* st = p.stats + (static_cast<size_t>(s.slot_q) + static_cast<size_t>(s.head) * p.q_slots + s.tile) *
                                  kStatFloats;
        st[row] = nl;
        st[kTile + row] = nd;
      }
      nl2 = ptx::f2_pack(nl, nl);
      nd2 = ptx::f2_pack(nd, nd);
    }
    for (int j = 0; ok && j < n; ++j) {
      const uint32_t tSh = tmem + 128 * (j & 1) + lane_base + 64 * g;
      const bool mk = masked(j);
      const int hi = limit - (t0 + j) * kTile - 64 * g;  // columns of this half the row sees
      Half pr;
      if (!(ok = warp_wait(bar(kDqSFull + (j & 1)), (j >> 1) & 1, abort_flag, p.timeout_ns))) break;
      ptx::tc_fence_after();
      {
        uint32_t a[32], b[32];
        load_half(tSh, a, b);
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          const uint64_t s2 = x < 16 ? ptx::f2_pack(__uint_as_float(a[2 * x]), __uint_as_float(a[2 * x + 1]))
                                     : ptx::f2_pack(__uint_as_float(b[2 * x - 32]), __uint_as_float(b[2 * x - 31]));
          float e0, e1;
          ptx::f2_unpack(ptx::f2_fma(s2, c2, nl2), e0, e1);
          pr[x] = ptx::f2_pack(ptx::ex2(e0), ptx::ex2(e1));
        }
      }
      if (!(ok = warp_wait(bar(kDqDpFull), j & 1, abort_flag, p.timeout_ns))) break;
      ptx::tc_fence_after();
      if (mk)
        dq_ds<true>(tPh, tSh, nd2, hi, pr);
      else
        dq_ds<false>(tPh, tSh, nd2, hi, pr);
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(kDqDsFull));
    }
    // ---- epilogue: each warpgroup stores 64 columns of the rows.
    if (ok && n > 0) ok = warp_wait(bar(kDqAcc), 0, abort_flag, p.timeout_ns);
    if (ok) {
      ptx::tc_fence_after();
      const uint32_t tacc = tQ + lane_base + 64 * g;
      auto poison = [&](int col) -> bool { return kCheck && poison_k[64 * g + col] < limit; };
      if (p.n_splits == 1) {
        const bool in = q0 + row < s.sq && dbg_ok(s.q_base + q0 + row < p.Sq);
        uint16_t* dst =
            p.dq + row_at(p.layout, s.batch, p.Hq, p.Sq, s.head, s.q_base + q0 + (in ? row : 0)) + 64 * g;
        store_row<64>(tacc, n == 0, p.scale, p.mode, in ? dst : nullptr, kCheck && *poison_any, poison);
      } else {
        const size_t slots = static_cast<size_t>(p.q_slots) * (kVarlen ? p.Hq : p.BH);
        const size_t slot = static_cast<size_t>(s.slot_q) + static_cast<size_t>(s.head) * p.q_slots + s.tile;
        float* dst = p.part + ((static_cast<size_t>(s.split) * slots + slot) * kTile + row) * kD + 64 * g;
        store_part<64>(tacc, n == 0, dst, poison);
      }
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
// and rounded. One block per 16 rows of a tile, 16 threads per row (32 bytes each).
struct JoinParams {
  const float* part;
  uint16_t* out[2];  // dq, or dk and dv
  float factor[2];
  const int* cu;     // packed batch: the owned axis's offsets
  const int* cu2;    // and the other axis's (a sequence with bad offsets is left alone)
  int S, S2, H, max_s, max_s2, slots, B, n_tiles, n_splits, results, layout, mode;
};

constexpr int kJoinRows = 16;

template <bool kVarlen>
__global__ void __launch_bounds__(16 * kJoinRows) attn_bwd_join(const JoinParams p) {
  constexpr int kPer = kTile / kJoinRows;  // blocks per tile
  const int r = (blockIdx.x % kPer) * kJoinRows + (threadIdx.x >> 4);
  int item = blockIdx.x / kPer;
  const int tile = item % p.n_tiles;
  item /= p.n_tiles;
  const int h = item % p.H;
  item /= p.H;
  const int b = item % p.B, result = item / p.B;
  ptx::grid_dependency_wait();
  int base = 0, len = p.S, batch = b;
  size_t slot = (static_cast<size_t>(b) * p.H + h) * p.slots + tile;
  if (kVarlen) {
    base = __ldg(p.cu + b);
    len = __ldg(p.cu + b + 1) - base;
    const int base2 = __ldg(p.cu2 + b), len2 = __ldg(p.cu2 + b + 1) - base2;
    if (base < 0 || len < 0 || len > p.max_s || base + len > p.S || base2 < 0 || len2 < 0 ||
        len2 > p.max_s2 || base2 + len2 > p.S2)
      return;
    batch = 0;
    slot = static_cast<size_t>(h) * p.slots + tile_slot<true>(base, b) + tile;
  }
  const int row = tile * kTile + r;
  if (row >= len) return;
  const size_t slots = static_cast<size_t>(p.slots) * p.H * (kVarlen ? 1 : p.B);
  const int c0 = (threadIdx.x & 15) * 8;
  float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int k = 0; k < p.n_splits; ++k) {
    const float4* src = reinterpret_cast<const float4*>(
        p.part + (((static_cast<size_t>(k) * p.results + result) * slots + slot) * kTile + r) * kD + c0);
    const float4 u = src[0], v = src[1];
    x[0] += u.x; x[1] += u.y; x[2] += u.z; x[3] += u.w;
    x[4] += v.x; x[5] += v.y; x[6] += v.z; x[7] += v.w;
  }
  const float f = result ? p.factor[1] : p.factor[0];
  uint16_t* out = result ? p.out[1] : p.out[0];
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = round_bf16_bits(x[2 * i] * f, p.mode) | (round_bf16_bits(x[2 * i + 1] * f, p.mode) << 16);
  *reinterpret_cast<uint4*>(out + row_at(p.layout, batch, p.H, p.S, h, base + row) + c0) =
      make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace bwd
}  // namespace attn
