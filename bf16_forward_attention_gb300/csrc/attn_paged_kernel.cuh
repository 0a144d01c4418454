// attn_paged_kernel.cuh - attention of new tokens over a paged key-value cache.
//
// The rows (new tokens times the group's heads) of a sequence and a key/value head go
// through the sequence's keys in blocks of at most 32; an item is one such block with all its
// keys, cut into tiles of 16. The keys are read once per block, so few rows are bound by HBM.
// All items' tiles in a row, sequence by sequence, are cut into equal runs, one a CTA: lengths
// are on the device, and a long sequence among short ones is spread over as many CTAs as its
// keys are worth. A CTA that has an item whole finishes it; an item that is cut leaves
// unnormalised rows and (reference, sum) per part, joined by attn_paged_join:
//   O = sum_s 2^(r_s - R) O_s / sum_s 2^(r_s - R) l_s,   lse = ln 2 (R + log2 L).
// With the keys' weights wanted, the logits s_ij go to the workspace too, and
// attn_paged_mass adds  sum_i 2^(s_ij - lse_i)  to every key's mass.
#pragma once
#include "few_rows.cuh"

namespace attn {
namespace paged {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 3;
constexpr int kStageBytes = 2 * few::kKvBytes;
constexpr int kWarpBytes = kStages * kStageBytes;
constexpr int kMaxRows = 32;                       // rows of a block at most
constexpr int kOffQ = kWarps * kWarpBytes;         // the block's queries
constexpr int kOffMl = kOffQ + kMaxRows * kD * 2;  // [warp][row][2] floats
constexpr int kSmem = kOffMl + kWarps * kMaxRows * 8;
constexpr int kRowPitch = kD + 4;                  // fp32 rows in shared memory: distinct banks
static_assert(kWarpBytes >= kMaxRows * kRowPitch * 4, "a warp's stages hold its fp32 rows at the end");
constexpr int kMinTiles = 8;                       // of a run: with fewer tiles there are fewer runs

// What a run leaves for the join: the item that it begins and does not end, and in how many
// parts (0: none).
struct Cut {
  int b, item, parts, unused;
};

struct Params {
  const uint16_t* q;
  const uint16_t* k;       // pages
  const uint16_t* v;
  const int* table;        // (B, max_pages)
  const int* seqlens;      // keys of each sequence, 0..cap
  uint16_t* out;
  float* lse;              // (B, Hq, Sq)
  float* mass;             // (B, Hkv, cap) or null
  float* part_o;           // [2 run + begins its item][rows8][128]
  float* part_rl;          // [2 run + begins its item][rows8][2]
  Cut* cuts;               // [run]
  float* lse2;             // with mass: [b][kv head][block][rows8], log2 units; +Inf: not to be used
  float* logits;           // with mass: [b][kv head][cap][block][rows8], log2 units
  int B, Hq, Hkv, group, Sq, cap, layout, causal, mode;
  int n_pages, page_size, page_shift, max_pages;  // page_shift: log2 of the page size, or -1
  int page_rows;           // rows of 128 from a page to the next
  int rows;                // Sq * group
  int blocks, block_rows, rows8;  // blocks of at most block_rows rows; rows8: that, in eights
  float c;                 // scale * log2(e)
};

__device__ __forceinline__ int tiles_of(int len, int cap) {
  return len < 0 || len > cap ? 1 : max(1, (len + few::kKeys - 1) / few::kKeys);
}

// Where a run of tiles begins. Units: the tiles of all items in a row (sequence, then kv head
// and block); `per` items a sequence.
struct Run {
  long long lo, hi;     // units
  long long first;      // of sequence b
  long long total;
  int b, runs;
};

// Run blockIdx.x of at most gridDim.x runs of at least `least` tiles. All threads of the block;
// false: there is no such run.
template <int kBlock>
__device__ __forceinline__ bool find_run(const int* seqlens, int B, int cap, int per, int least, Run& run) {
  __shared__ long long warp_sum[kBlock / 32], at_first;
  __shared__ int at_b;
  const int each = (B + kBlock - 1) / kBlock;
  const int b0 = min(B, static_cast<int>(threadIdx.x) * each), b1 = min(B, b0 + each);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += tiles_of(__ldg(seqlens + b), cap);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long x = __shfl_up_sync(0xFFFFFFFFu, upto, d);
    if (lane >= d) upto += x;
  }
  if (lane == 31) warp_sum[warp] = upto;
  __syncthreads();
  long long total = 0, before = upto - mine;
#pragma unroll
  for (int w = 0; w < kBlock / 32; ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  total *= per;
  const long long most = (total + least - 1) / least;
  run.runs = static_cast<int>(most < static_cast<long long>(gridDim.x) ? most : static_cast<long long>(gridDim.x));
  run.total = total;
  if (static_cast<int>(blockIdx.x) >= run.runs) return false;
  run.lo = total * blockIdx.x / run.runs;
  run.hi = total * (blockIdx.x + 1) / run.runs;
  if (run.lo >= before * per && run.lo < (before + mine) * per) {
    long long x = before;
    int b = b0;
    for (; b + 1 < b1; ++b) {
      const int t = tiles_of(__ldg(seqlens + b), cap);
      if (run.lo < (x + t) * per) break;
      x += t;
    }
    at_b = b;
    at_first = x * per;
  }
  __syncthreads();
  run.b = at_b;
  run.first = at_first;
  return true;
}

// A row's result, four columns a lane, from its unnormalised sums and (reference, sum).
__device__ __forceinline__ void store_row(const Params& p, int b, int kvh, int block, int r, int lane, float4 o,
                                          float R, float L) {
  const int row = block * p.block_rows + r;
  if (!dbg_ok(r >= 0 && r < p.block_rows && row < p.rows && b >= 0 && b < p.B && kvh < p.Hkv)) return;
  const float inv = __frcp_rn(L);
  *reinterpret_cast<uint2*>(p.out + few::query_at(p.layout, p.Hq, p.Sq, p.group, b, kvh, row) + 4 * lane) =
      make_uint2(round_bf16_bits(o.x * inv, p.mode) | (round_bf16_bits(o.y * inv, p.mode) << 16),
                 round_bf16_bits(o.z * inv, p.mode) | (round_bf16_bits(o.w * inv, p.mode) << 16));
  if (lane == 0) {
    const int h = kvh * p.group + row % p.group;
    store_lse(p.lse, (static_cast<size_t>(b) * p.Hq + h) * p.Sq + row / p.group, R, L);
    if (p.mass)
      p.lse2[(static_cast<size_t>(b) * p.Hkv + kvh) * p.blocks * p.rows8 + block * p.rows8 + r] = R + log2f(L);
  }
}

// A row whose keys cannot be read: its results stay as they were, and attn_paged_mass is told.
__device__ __forceinline__ void skip_row(const Params& p, int b, int kvh, int block, int r) {
  if (p.mass)
    p.lse2[(static_cast<size_t>(b) * p.Hkv + kvh) * p.blocks * p.rows8 + block * p.rows8 + r] =
        __int_as_float(0x7F800000);
}

// One CTA: a run of tiles. The four warps take an item's tiles in turn, each with a ring of its own
// (cp.async, 3 stages of 8 KiB), and are joined in shared memory at the item's end.
template <int kNT, bool kFold, bool kMass>
__global__ void __launch_bounds__(kThreads, 2) attn_paged_fwd(const Params p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int bad_page;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float neg_inf = -__int_as_float(0x7F800000);
  const int per = p.Hkv * p.blocks;
  if (threadIdx.x == 0) p.cuts[blockIdx.x].parts = 0;
  Run run;
  if (!find_run<kThreads>(p.seqlens, p.B, p.cap, per, kMinTiles, run)) return;
  const uint32_t ring = ptx::smem_u32(smem) + warp * kWarpBytes, qs = ptx::smem_u32(smem) + kOffQ;
  const int half = lane >> 4, chunk = lane & 15;
  const uint32_t lane_dst = ring + few::row_at(half, chunk);  // keys 2 u + half: + 512 u, chunk turned by 2 u

  long long u = run.lo, first = run.first;
  int b = run.b;
  while (u < run.hi) {
    const int len = __ldg(p.seqlens + b), tiles = tiles_of(len, p.cap);
    const int item = static_cast<int>((u - first) / tiles), t_first = static_cast<int>((u - first) % tiles);
    const long long left = run.hi - u;
    const int t_end = left < tiles - t_first ? t_first + static_cast<int>(left) : tiles;
    const int kvh = item / p.blocks, block = item - kvh * p.blocks;
    const int row0 = block * p.block_rows, n_rows = min(p.block_rows, p.rows - row0);
    const bool whole = t_first == 0 && t_end == tiles;
    if (!dbg_ok(b < p.B && item >= 0 && item < per && n_rows >= 1 && n_rows <= 8 * kNT && t_first < t_end)) return;
    const int here = b;
    const long long u_item = u - t_first;
    u += t_end - t_first;
    if (u == first + static_cast<long long>(tiles) * per) {
      first = u;
      ++b;
    }
    if (len < 0 || len > p.cap) {  // one tile a sequence, so this item is whole
      if (threadIdx.x == 0) atomicOr(&g_attn_status, 2u);
      for (int r = threadIdx.x; r < n_rows; r += kThreads) skip_row(p, here, kvh, block, r);
      continue;
    }
    // ---- queries.
    __syncthreads();  // the last item's rows have been read
    if (threadIdx.x == 0) bad_page = 0;
#pragma unroll
    for (int it = 0; it < kNT; ++it) {
      const int r = it * 8 + (threadIdx.x >> 4), c = threadIdx.x & 15;
      uint4 x = make_uint4(0, 0, 0, 0);
      if (r < n_rows)
        x = __ldg(reinterpret_cast<const uint4*>(
                      p.q + few::query_at(p.layout, p.Hq, p.Sq, p.group, here, kvh, row0 + r)) + c);
      ptx::st_shared_v4(qs + few::row_at(r, c), x.x, x.y, x.z, x.w);
    }
    few::Rows<kNT, kFold> rows;
    rows.clear();
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * nt + 2 * (lane & 3) + e;
        rows.lim[nt][e] = r < n_rows ? few::own_limit((row0 + r) / p.group, len, p.Sq, p.causal) : 0;
      }
    const int min_lim = few::own_limit(row0 / p.group, len, p.Sq, p.causal);

    // Row of 128 (in the pages) of key `lane % 16` of tile t, -1: none.
    const int* pages = p.table + static_cast<size_t>(here) * p.max_pages;
    bool bad = false;
    auto row_of = [&](int t) {
      const int key = t * few::kKeys + chunk;
      if (key >= len) return -1;
      const int page = p.page_shift >= 0 ? key >> p.page_shift : key / p.page_size;
      const int at = key - page * p.page_size, id = __ldg(pages + page);
      if (id < 0 || id >= p.n_pages) {
        bad = true;
        return -1;
      }
      return id * p.page_rows + (p.layout == 0 ? kvh * p.page_size + at : at * p.Hkv + kvh);
    };
    auto load = [&](int row, int s) {
      const uint32_t dst = lane_dst + s * kStageBytes;
#pragma unroll
      for (int x = 0; x < few::kKeys / 2; ++x) {
        const int r = __shfl_sync(0xFFFFFFFFu, row, half + 2 * x);
        const uint32_t d = (dst ^ ((2 * x & 6) << 4)) + 512 * x;
        const size_t at = static_cast<size_t>(max(r, 0)) * kD + 8 * chunk;
        ptx::cp_async16(d, p.k + at, r >= 0);
        ptx::cp_async16(d + few::kKvBytes, p.v + at, r >= 0);
      }
    };
    const int t0 = t_first + warp;
    const int n = t0 < t_end ? (t_end - t0 + kWarps - 1) / kWarps : 0;  // this warp's tiles
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) {
      if (s < n) load(row_of(t0 + s * kWarps), s);
      ptx::cp_async_commit();
    }
    int next = kStages - 1 < n ? row_of(t0 + (kStages - 1) * kWarps) : -1;
    __syncthreads();  // the queries
    rows.load_q(qs, lane);
    for (int i = 0; i < n; ++i) {
      ptx::cp_async_wait<kStages - 2>();
      __syncwarp();  // every lane's copies of this tile; every lane is done with the last one
      if (i + kStages - 1 < n) load(next, (i + kStages - 1) % kStages);
      ptx::cp_async_commit();
      if (i + kStages < n) next = row_of(t0 + (i + kStages) * kWarps);
      const uint32_t kt = ring + (i % kStages) * kStageBytes;
      const int key0 = (t0 + i * kWarps) * few::kKeys;
      const bool masked = key0 + few::kKeys > min_lim;
      rows.tile(kt, kt + few::kKvBytes, key0, masked, masked && p.causal, p.c, lane,
                [&](const float (&s)[kNT][4]) {
                  if constexpr (kMass) {
                    float* to = p.logits + ((static_cast<size_t>(here) * p.Hkv + kvh) * p.cap + key0 + (lane >> 2)) *
                                               (p.blocks * p.rows8) + block * p.rows8 + 2 * (lane & 3);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                      if (key0 + (lane >> 2) + 8 * e < len) {
#pragma unroll
                        for (int nt = 0; nt < kNT; ++nt)
                          *reinterpret_cast<float2*>(to + 8 * nt) = make_float2(s[nt][2 * e], s[nt][2 * e + 1]);
                      }
                      to += 8 * (p.blocks * p.rows8);
                    }
                  }
                });
    }
    // ---- the warps' rows, joined through shared memory (each warp's own ring).
    ptx::cp_async_wait<0>();
    if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) {
      atomicOr(&g_attn_status, 8u);
      bad_page = 1;
    }
    __syncwarp();
    rows.finish_sums();
    float* ml = reinterpret_cast<float*>(smem + kOffMl) + warp * kMaxRows * 2;
    float* mine = reinterpret_cast<float*>(smem + warp * kWarpBytes);
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * nt + 2 * (lane & 3) + e;
        if ((lane >> 2) == 0) {
          ml[2 * r] = rows.ref[nt][e];
          ml[2 * r + 1] = rows.sum[nt][e];
        }
#pragma unroll
        for (int dt = 0; dt < 8; ++dt) {
          mine[r * kRowPitch + 16 * dt + (lane >> 2)] = rows.o[dt][nt][e];
          mine[r * kRowPitch + 16 * dt + 8 + (lane >> 2)] = rows.o[dt][nt][2 + e];
        }
      }
    __syncthreads();
    const size_t part = 2 * static_cast<size_t>(blockIdx.x) + (t_first == 0 ? 1 : 0);
    const float2* all_ml = reinterpret_cast<const float2*>(smem + kOffMl);
    for (int r = warp; r < n_rows; r += kWarps) {
      float2 x2[kWarps];
      float M = neg_inf;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        x2[w] = all_ml[w * kMaxRows + r];
        M = fmaxf(M, x2[w].x);
      }
      const float ref = M == neg_inf ? 0.f : M;
      float L = 0.f;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ptx::ex2(x2[w].x - ref);
        const float4 y = reinterpret_cast<const float4*>(smem + w * kWarpBytes)[r * (kRowPitch / 4) + lane];
        L = fmaf(x2[w].y, f, L);
        x.x = fmaf(y.x, f, x.x);
        x.y = fmaf(y.y, f, x.y);
        x.z = fmaf(y.z, f, x.z);
        x.w = fmaf(y.w, f, x.w);
      }
      if (whole) {
        if (!bad_page)
          store_row(p, here, kvh, block, r, lane, x, M, L);
        else if (lane == 0)
          skip_row(p, here, kvh, block, r);
      } else {
        reinterpret_cast<float4*>(p.part_o)[(part * p.rows8 + r) * (kD / 4) + lane] = x;
        // A sum is not negative: -1 tells the join that the rows cannot be formed.
        if (lane == 0)
          reinterpret_cast<float2*>(p.part_rl)[part * p.rows8 + r] = make_float2(M, bad_page ? -1.f : L);
      }
    }
    if (t_first == 0 && !whole && threadIdx.x == 0) {
      // The item's last tile is in the last run that begins before its end.
      const long long end = u_item + tiles;
      const int last = static_cast<int>((end * run.runs + run.total - 1) / run.total) - 1;
      p.cuts[blockIdx.x] = {here, item, last - static_cast<int>(blockIdx.x) + 1, 0};
    }
  }
}

// ---------------------------------------------------------------- join
constexpr int kJoinWarps = 4;

// A block per (run, row): the run's cut item, if it has one, its parts over the four warps in a
// fixed order.
__global__ void __launch_bounds__(32 * kJoinWarps) attn_paged_join(const Params p) {
  __shared__ float4 sum_o[kJoinWarps][32];
  __shared__ float sum_l[kJoinWarps];
  ptx::grid_dependency_wait();
  const Cut cut = p.cuts[blockIdx.x];
  if (cut.parts == 0) return;
  const int kvh = cut.item / p.blocks, block = cut.item - kvh * p.blocks, r = blockIdx.y;
  if (r >= min(p.block_rows, p.rows - block * p.block_rows)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float neg_inf = -__int_as_float(0x7F800000);
  const float2* rl = reinterpret_cast<const float2*>(p.part_rl);
  // Part 0 begins the item; the others are the first of their runs.
  auto part_at = [&](int i) {
    return (2 * (static_cast<size_t>(blockIdx.x) + i) + (i == 0 ? 1 : 0)) * p.rows8 + r;
  };
  float R = neg_inf;
  bool skip = false;
  for (int i = lane; i < cut.parts; i += 32) {
    const float2 x = rl[part_at(i)];
    R = fmaxf(R, x.x);  // a NaN is left out: it comes back through its weight
    skip = skip || x.y < 0.f;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) R = fmaxf(R, __shfl_xor_sync(0xFFFFFFFFu, R, d));
  if (__any_sync(0xFFFFFFFFu, skip)) {
    if (threadIdx.x == 0) skip_row(p, cut.b, kvh, block, r);
    return;
  }
  const float ref = R == neg_inf ? 0.f : R;
  float L = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = warp; i < cut.parts; i += kJoinWarps) {
    const size_t at = part_at(i);
    const float2 x = rl[at];
    const float w = ptx::ex2(x.x - ref);
    const float4 y = reinterpret_cast<const float4*>(p.part_o)[at * (kD / 4) + lane];
    L = fmaf(x.y, w, L);
    o.x = fmaf(y.x, w, o.x);
    o.y = fmaf(y.y, w, o.y);
    o.z = fmaf(y.z, w, o.z);
    o.w = fmaf(y.w, w, o.w);
  }
  sum_o[warp][lane] = o;
  if (lane == 0) sum_l[warp] = L;
  __syncthreads();
  if (warp != 0) return;
#pragma unroll
  for (int w = 1; w < kJoinWarps; ++w) {
    const float4 y = sum_o[w][lane];
    L += sum_l[w];
    o.x += y.x;
    o.y += y.y;
    o.z += y.z;
    o.w += y.w;
  }
  store_row(p, cut.b, kvh, block, r, lane, o, R, L);
}

// ---------------------------------------------------------------- mass
constexpr int kMassThreads = 128;
constexpr int kMassTiles = 8;  // of a run at least: a key a thread

// mass[b, kvh, j] += sum over the rows that see key j of 2^(s_ij - lse_i), a key a thread, the
// rows in order. A row whose log-sum-exp is -Inf (it sees no key) adds nothing.
__global__ void __launch_bounds__(kMassThreads) attn_paged_mass(const Params p) {
  const float inf = __int_as_float(0x7F800000);
  Run run;
  const bool any = find_run<kMassThreads>(p.seqlens, p.B, p.cap, p.Hkv, kMassTiles, run);
  ptx::grid_dependency_wait();
  if (!any) return;
  const int pitch = p.blocks * p.rows8;
  long long u = run.lo, first = run.first;
  int b = run.b;
  while (u < run.hi) {
    const int len = __ldg(p.seqlens + b), tiles = tiles_of(len, p.cap);
    const int kvh = static_cast<int>((u - first) / tiles), t_first = static_cast<int>((u - first) % tiles);
    const long long left = run.hi - u;
    const int t_end = left < tiles - t_first ? t_first + static_cast<int>(left) : tiles;
    const int here = b;
    u += t_end - t_first;
    if (u == first + static_cast<long long>(tiles) * p.Hkv) {
      first = u;
      ++b;
    }
    if (len < 0 || len > p.cap) continue;
    const size_t head = static_cast<size_t>(here) * p.Hkv + kvh;
    const float* lse2 = p.lse2 + head * pitch;
    bool skip = false;
    for (int r = threadIdx.x; r < p.rows; r += kMassThreads)
      skip = skip || lse2[r / p.block_rows * p.rows8 + r % p.block_rows] == inf;
    if (__syncthreads_or(skip)) continue;  // a page of the sequence could not be read
    const int end = min(t_end * few::kKeys, len);
    for (int key = t_first * few::kKeys + threadIdx.x; key < end; key += kMassThreads) {
      const float* s = p.logits + (head * p.cap + key) * pitch;
      float sum = 0.f;
      for (int block = 0; block < p.blocks; ++block) {
        const int n_rows = min(p.block_rows, p.rows - block * p.block_rows);
        for (int r = 0; r < n_rows; r += 4) {
          const float4 s4 = *reinterpret_cast<const float4*>(s + block * p.rows8 + r);
          const float4 l4 = *reinterpret_cast<const float4*>(lse2 + block * p.rows8 + r);
          const float sv[4] = {s4.x, s4.y, s4.z, s4.w}, lv[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (r + e >= n_rows || lv[e] == -inf) continue;
            if (p.causal &&
                key >= few::own_limit((block * p.block_rows + r + e) / p.group, len, p.Sq, 1))
              continue;
            sum += ptx::ex2(sv[e] - lv[e]);
          }
        }
      }
      p.mass[head * p.cap + key] += sum;
    }
  }
}

}  // namespace paged
}  // namespace attn
