// attn_paged_kernel.cuh - attention of new tokens over a paged key-value cache.
//
// The rows (new tokens times the group's heads) of a sequence and a key/value head go
// through the sequence's keys in blocks of at most 128; an item is one such block with all its
// keys, cut into units of 64. The keys are read once per block, so few rows are bound by HBM.
// Up to 16 rows go through warp-level products (attn_paged_fwd), more through the tensor cores
// (attn_paged_rows).
// All items' units in a row, sequence by sequence, are cut into equal runs, one a CTA: lengths
// are on the device, and a long sequence among short ones is spread over as many CTAs as its
// keys are worth. A CTA that has an item whole finishes it; an item that is cut leaves
// unnormalised rows and (reference, sum) per part, joined by attn_paged_finish:
//   O = sum_s 2^(r_s - R) O_s / sum_s 2^(r_s - R) l_s,   lse = ln 2 (R + log2 L).
// With the keys' weights wanted, the logits s_ij go to the workspace too, and blocks beside the
// join's add  sum_i 2^(s_ij - lse_i)  to every key's mass.
#pragma once
#include "few_rows.cuh"

namespace attn {
namespace paged {

constexpr int kTeams = 4;                          // of a CTA, 16 keys of a unit each
constexpr int kUnit = kTeams * few::kKeys;
constexpr int kStageBytes = 2 * few::kKvBytes;     // a team's K and V
constexpr int kMaxRows = 128;                      // rows of a block at most
// What an item costs a run beside its units, in units (its queries, its rows' addition and stores). In
// attn_paged_rows that is some 13700 cycles an item. Runs of equal numbers of units made those of many short
// items the last to end (48 x 5 drafted tokens: 63 to 108 us a run, and 47 to 64 with the items counted).
// One number for all its rows, us a call at 24 / 35 / 64 / 128 of them (4, 2, 2 copies and 1):
//   64 caches of up to 300 keys:   3: 38.5 / 44.8 / 50.8 / 69.2   4: 37.5 / 43.3 / 48.2 / 66.6   6: 38.1 / 45.4 / 50.2 / 67.7
//   48 of up to 5003, 4 kv heads:  3: 67.0 / 81.4 / 88.5 / 121    4: 66.3 / 80.5 / 86.9 / 120    6: 67.2 / 80.5 / 85.8 / 119
//   64 of up to 8192, 8 kv heads:  3: 219 / 264 / 282 / 393       4: 209 / 255 / 270 / 375       6: 208 / 247 / 261 / 367
constexpr int kItemCost = 1, kRowsItemCost = 4;

// kGroups warps a team, 8 rows each: blocks of up to 8 kGroups rows; two CTAs an SM.
template <int kGroups_>
struct Shape {
  static constexpr int kGroups = kGroups_, kStages = 3;
  static constexpr int kThreads = 32 * kTeams * kGroups;
  static constexpr int kRows = 8 * kGroups;
  static constexpr int kOffX = kTeams * kStages * kStageBytes;       // half of every warp's O^T
  static constexpr int kOffMl = kOffX + kTeams * kGroups * 4 * 512;  // [team][row][2] floats
  static constexpr int kSmem = kOffMl + kTeams * kRows * 8;
};

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
  float* part_o;           // [2 run + begins its item][8-row group][16-column group][lane][4]: as the warps hold it
  float* part_rl;          // [2 run + begins its item][rows8][2]
  Cut* cuts;               // [run]
  float* lse2;             // with mass, of rows not cut: [b][kv head][rows4], log2 units; +Inf: not to be used
  float* logits;           // with mass: [b][kv head][cap][rows4], log2 units
  int B, Hq, Hkv, group, Sq, cap, layout, causal, mode;
  int n_pages, page_size, page_shift, max_pages;
  uint32_t page_mul;       // with page_shift: see page_divisor
  int page_rows;           // rows of 128 from a page to the next
  int rows, rows4;         // Sq * group; that, in fours
  int blocks, block_rows, rows8;  // blocks of at most block_rows rows; rows8: the kernel's rows of a block
  int cost, runs;          // an item's cost and the most runs, as the kernel of the runs has them
  int join_groups;         // blocks of a run in attn_paged_finish: 8-row groups
  float c;                 // scale * log2(e)
  unsigned long long timeout_ns;  // of a wait for the tensor cores
  int withhold;            // self-test: never tell of a run's first S
};

__device__ __forceinline__ int units_of(int len, int cap) {
  return len < 0 || len > cap ? 1 : max(1, (len + kUnit - 1) / kUnit);
}

__device__ __forceinline__ int runs_of(long long total, int least, int count) {
  const long long most = (total + least - 1) / least;
  return static_cast<int>(most < count ? most : static_cast<long long>(count));
}
// The run in which place x lies.
__device__ __forceinline__ int run_of(long long x, long long total, int runs) {
  return static_cast<int>(((x + 1) * runs + total - 1) / total) - 1;
}

// A run of units: all items in a row (sequence, then kv head and block; `per` items a sequence), each
// as many places long as it has units and `cost` more in front, cut into runs of equal length.
struct Run {
  long long lo, hi;     // places
  long long first;      // place of sequence b, in which the run begins
  long long total;
  int b, runs;
  int n;                // units
};

// Run `index` of at most `count` runs of at least `least` places. All threads of the block; false: there
// is no such run.
template <int kBlock>
__device__ __forceinline__ bool find_run(const int* seqlens, int B, int cap, int per, int cost, int least, int index,
                                         int count, Run& run) {
  __shared__ long long warp_sum[kBlock / 32], at_first[2];
  __shared__ int at_b[2];
  const int each = (B + kBlock - 1) / kBlock;
  const int b0 = min(B, static_cast<int>(threadIdx.x) * each), b1 = min(B, b0 + each);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += units_of(__ldg(seqlens + b), cap) + cost;
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
  run.runs = runs_of(total, least, count);
  run.total = total;
  if (index >= run.runs) return false;
  run.lo = total * index / run.runs;
  run.hi = total * (index + 1) / run.runs;
  // The sequences of the first place, and of the last.
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const long long place = e == 0 ? run.lo : run.hi - 1;
    if (place >= before * per && place < (before + mine) * per) {
      long long x = before;
      int b = b0;
      for (; b + 1 < b1; ++b) {
        const int t = units_of(__ldg(seqlens + b), cap) + cost;
        if (place < (x + t) * per) break;
        x += t;
      }
      at_b[e] = b;
      at_first[e] = x * per;
    }
  }
  __syncthreads();
  run.b = at_b[0];
  run.first = at_first[0];
  // Units before place x of sequence b, which begins at place `first`.
  auto units_before = [&](long long x, int b, long long first) {
    const int units = units_of(__ldg(seqlens + b), cap);
    const long long item = (x - first) / (units + cost), in = (x - first) % (units + cost) - cost;
    return first - static_cast<long long>(per) * cost * b + item * units + (in > 0 ? in : 0);
  };
  run.n = static_cast<int>(units_before(run.hi, at_b[1], at_first[1]) - units_before(run.lo, run.b, run.first));
  return run.n > 0;
}

// A run's units one after another.
struct Walk {
  int b, item, t;       // sequence, its item, the item's unit
  int kvh, block;       // the item's kv head and block
  int len, units;       // the sequence's keys (-1: out of range), its items' units
  int next_len;         // what the length of the next sequence reads, on its way
  long long first;      // place of the sequence

  __device__ __forceinline__ void enter(const Params& p) {
    len = next_len;
    next_len = __ldg(p.seqlens + min(b + 1, p.B - 1));
    units = units_of(len, p.cap);
    if (len > p.cap) len = -1;
    len = max(len, -1);
  }
  __device__ __forceinline__ void start(const Params& p, const Run& run, int cost) {
    b = run.b;
    first = run.first;
    next_len = __ldg(p.seqlens + b);
    enter(p);
    const long long rel = run.lo - run.first;
    item = static_cast<int>(rel / (units + cost));
    t = max(0, static_cast<int>(rel - static_cast<long long>(item) * (units + cost)) - cost);
    kvh = item / p.blocks;
    block = item - kvh * p.blocks;
  }
  __device__ __forceinline__ void step(const Params& p, int per, int cost) {
    if (++t < units) return;
    t = 0;
    if (++block == p.blocks) {
      block = 0;
      ++kvh;
    }
    if (++item < per) return;
    item = kvh = 0;
    first += static_cast<long long>(per) * (units + cost);
    if (++b < p.B) enter(p);
  }
  // In how many runs the item lies, of which this one has its first unit.
  __device__ __forceinline__ int parts(const Run& run, int cost) const {
    const long long end = first + static_cast<long long>(item + 1) * (units + cost);
    return run_of(end - 1, run.total, run.runs) - static_cast<int>(blockIdx.x) + 1;
  }
};

// A key's place in the pages, in two steps: the page's number is read a unit before it is looked at (a read
// waited for at once cost 600 cycles a unit).
struct Place {
  int id, at;  // at: row of 128 within the page; -1: there is no such key
};
__device__ __forceinline__ Place place_of(const Params& p, const Walk& w, int key) {
  if (key >= w.len) return {0, -1};
  const int page = few::page_of(key, p.page_mul, p.page_shift), i = key - page * p.page_size;
  return {__ldg(p.table + static_cast<size_t>(w.b) * p.max_pages + page),
          p.layout == 0 ? w.kvh * p.page_size + i : i * p.Hkv + w.kvh};
}
// Its row of 128 in the pages; -1: none, -2: its page is out of range.
__device__ __forceinline__ int row_of(const Params& p, const Place& x) {
  if (x.at < 0) return -1;
  return x.id >= 0 && x.id < p.n_pages ? x.id * p.page_rows + x.at : -2;
}

// An item's rows.
struct Item {
  int b, kvh, row0, n_rows;
};
__device__ __forceinline__ Item item_of(const Params& p, int b, int kvh, int block) {
  const int row0 = block * p.block_rows;
  return {b, kvh, row0, min(p.block_rows, p.rows - row0)};
}

__device__ __forceinline__ float& lse2_at(const Params& p, const Item& it, int r) {
  return p.lse2[(static_cast<size_t>(it.b) * p.Hkv + it.kvh) * p.rows4 + it.row0 + r];
}

// Rows 8 g + 2 (lane % 4) + {0, 1} of the item, columns 16 dt + lane / 4 (x[0], x[1]) and + 8: as
// the warps hold O^T. Normalised, rounded and stored; a transposition puts a row's
// neighbouring columns in one lane.
__device__ __forceinline__ void store_out(const Params& p, const Item& it, int g, int dt, int lane, const float (&x)[4],
                                          float inv0, float inv1) {
  const uint32_t a = round_bf16_bits(x[0] * inv0, p.mode) | (round_bf16_bits(x[1] * inv1, p.mode) << 16);
  const uint32_t c = round_bf16_bits(x[2] * inv0, p.mode) | (round_bf16_bits(x[3] * inv1, p.mode) << 16);
  const uint32_t at = ptx::movmatrix_trans(a), ct = ptx::movmatrix_trans(c);
  const int r = 8 * g + (lane >> 2);
  if (r >= it.n_rows || !dbg_ok(it.row0 + r < p.rows && it.b < p.B && it.kvh < p.Hkv)) return;
  uint16_t* to = p.out + few::query_at(p.layout, p.Hq, p.Sq, p.group, it.b, it.kvh, it.row0 + r) + 16 * dt + 2 * (lane & 3);
  *reinterpret_cast<uint32_t*>(to) = at;
  *reinterpret_cast<uint32_t*>(to + 8) = ct;
}

__device__ __forceinline__ void store_lse_of(const Params& p, const Item& it, int r, float R, float L,
                                             bool whole = true) {
  if (r >= it.n_rows) return;
  const int row = it.row0 + r, i = row / p.group, h = it.kvh * p.group + row - i * p.group;
  store_lse(p.lse, (static_cast<size_t>(it.b) * p.Hq + h) * p.Sq + i, R, L);
  if (whole && p.mass) lse2_at(p, it, r) = R + log2f(L);
}

// A row whose keys cannot be read: its results stay as they were, and add_mass is told.
__device__ __forceinline__ void skip_row(const Params& p, const Item& it, int r) {
  if (r < it.n_rows && p.mass) lse2_at(p, it, r) = __int_as_float(0x7F800000);
}

// One CTA: a run of units. A team of kGroups warps takes 16 keys of every unit, each warp 8 of
// the block's rows, over a ring of its own (cp.async, kStages of 8 KiB) that runs on from item to
// item; the teams meet only at an item's end, to add their rows. Bound by HBM where caches are long
// (64 caches of up to 8192 keys, 8 kv heads of 4 rows, 1.08 GB: 165 us, 6.6 TB/s; runs end after 148 to
// 163 us, as SMs differ in their share of the bandwidth); a few short ones by the chain of lengths, page
// numbers, keys and products (7.5 us for 4 caches of up to 1000 keys).
template <int kGroups, bool kMass>
__global__ void __launch_bounds__(Shape<kGroups>::kThreads, 2) attn_paged_fwd(const Params p) {
  using S = Shape<kGroups>;
  constexpr int kStages = S::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int team = warp / kGroups, grp = warp - team * kGroups;
  const float neg_inf = -__int_as_float(0x7F800000);
  const int per = p.Hkv * p.blocks;
  if (threadIdx.x == 0) p.cuts[blockIdx.x].parts = 0;
  Run run;
  constexpr int kCost = kItemCost;
  if (!find_run<S::kThreads>(p.seqlens, p.B, p.cap, per, kCost, kCost + 1, blockIdx.x, gridDim.x, run)) return;
  const uint32_t ring = ptx::smem_u32(smem) + team * kStages * kStageBytes;
  const int half = lane >> 4, chunk = lane & 15;

  // ---- loads: unit by unit, kStages - 1 ahead of the products.
  Walk ahead;
  ahead.start(p, run, kCost);
  uint32_t bad_stages = 0;  // of those in the ring, which hold a key without a page
  auto look_up = [&]() { return place_of(p, ahead, ahead.t * kUnit + team * few::kKeys + chunk); };
  auto load = [&](const Place& place, int s) {
    const int row = row_of(p, place);
    const bool bad = __any_sync(0xFFFFFFFFu, row == -2);
    bad_stages = (bad_stages & ~(1u << s)) | (bad ? 1u << s : 0u);
    const uint32_t dst = ring + s * kStageBytes;
#pragma unroll
    for (int x = 0; x < (few::kKeys / 2 + kGroups - 1) / kGroups; ++x) {
      const int pair = x * kGroups + grp;
      if (few::kKeys / 2 % kGroups != 0 && pair >= few::kKeys / 2) break;
      const int r = __shfl_sync(0xFFFFFFFFu, row, half + 2 * pair);
      const uint32_t d = dst + few::row_at(half + 2 * pair, chunk);
      const size_t at = static_cast<size_t>(max(r, 0)) * kD + 8 * chunk;
      ptx::cp_async16(d, p.k + at, r >= 0);
      ptx::cp_async16(d + few::kKvBytes, p.v + at, r >= 0);
    }
  };
  const int n = run.n;
  Place next = look_up();
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    if (s < n) {
      load(next, s);
      if (s + 1 < n) {
        ahead.step(p, per, kCost);
        next = look_up();
      }
    }
    ptx::cp_async_commit();
  }

  // ---- products.
  Walk at;
  at.start(p, run, kCost);
  few::Rows rows;
  Item it;
  int t_first = 0, min_lim = 0;
  bool bad = false, fresh = true;
  for (int i = 0; i < n; ++i) {
    if (fresh) {  // an item begins
      fresh = false;
      it = item_of(p, at.b, at.kvh, at.block);
      t_first = at.t;
      bad = false;
      rows.clear();
      const int r = 8 * grp + (lane >> 2);
      rows.load_q(r < it.n_rows && at.len >= 0
                      ? p.q + few::query_at(p.layout, p.Hq, p.Sq, p.group, it.b, it.kvh, it.row0 + r)
                      : nullptr,
                  lane);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int x = 8 * grp + 2 * (lane & 3) + e;
        rows.lim[e] = x < it.n_rows ? few::own_limit((it.row0 + x) / p.group, at.len, p.Sq, p.causal) : 0;
      }
      min_lim = few::own_limit(it.row0 / p.group, at.len, p.Sq, p.causal);
    }
    // Every lane's copies of this unit; the team is done with the last one.
    ptx::cp_async_wait<kStages - 2>();
    if constexpr (kGroups == 1)
      __syncwarp();
    else
      ptx::named_barrier_sync(1 + team, 32 * kGroups);
    const int s = i % kStages;
    const bool bad_now = bad_stages >> s & 1u;
    if (i + kStages - 1 < n) load(next, (i + kStages - 1) % kStages);
    ptx::cp_async_commit();
    if (i + kStages < n) {
      ahead.step(p, per, kCost);
      next = look_up();
    }
    const uint32_t kt = ring + s * kStageBytes;
    const int key0 = at.t * kUnit + team * few::kKeys;
    bad = bad || bad_now;
    if (key0 < at.len) {
      const bool masked = key0 + few::kKeys > min_lim;
      rows.tile(kt, kt + few::kKvBytes, key0, masked, masked && p.causal, p.c, lane,
                [&](const float (&x)[4]) {
                  if constexpr (kMass) {
                    const int r = 8 * grp + 2 * (lane & 3);
                    if (r >= it.n_rows) return;
                    float* to = p.logits + ((static_cast<size_t>(it.b) * p.Hkv + it.kvh) * p.cap + key0 + (lane >> 2)) *
                                               p.rows4 + it.row0 + r;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                      if (key0 + (lane >> 2) + 8 * e < at.len)
                        *reinterpret_cast<float2*>(to) = make_float2(x[2 * e], x[2 * e + 1]);
                      to += 8 * static_cast<size_t>(p.rows4);
                    }
                  }
                });
    }
    const bool ends = at.t + 1 == at.units;
    if (!ends && i + 1 < n) {
      ++at.t;
      continue;
    }
    // ---- the item's end, or the run's: the teams' rows are added, 64 columns at a time.
    fresh = true;
    const bool whole = ends && t_first == 0;
    rows.finish_sums();
    float2* ml = reinterpret_cast<float2*>(smem + S::kOffMl);  // [team][row]
    float4* xs = reinterpret_cast<float4*>(smem + S::kOffX);   // [group][team][dt % 4][lane]
    const size_t part = 2 * static_cast<size_t>(blockIdx.x) + (t_first == 0 ? 1 : 0);
    float f[kTeams][2], R[2], L[2];
    bool skip = false;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      __syncthreads();  // what was there has been read
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const float(&o)[4] = rows.o[4 * hf + d];
        xs[((grp * kTeams + team) * 4 + d) * 32 + lane] = make_float4(o[0], o[1], o[2], o[3]);
      }
      if (hf == 0 && (lane >> 2) == 0) {
#pragma unroll
        for (int e = 0; e < 2; ++e)  // a sum is not negative: -1 says that the rows cannot be formed
          ml[team * S::kRows + 8 * grp + 2 * lane + e] = make_float2(rows.ref[e], bad ? -1.f : rows.sum[e]);
      }
      __syncthreads();
      if (hf == 0) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 8 * grp + 2 * (lane & 3) + e;
          float2 x[kTeams];
          float M = neg_inf;
#pragma unroll
          for (int w = 0; w < kTeams; ++w) {
            x[w] = ml[w * S::kRows + r];
            M = fmaxf(M, x[w].x);
            skip = skip || x[w].y < 0.f;
          }
          const float ref = M == neg_inf ? 0.f : M;
          float sum = 0.f;
#pragma unroll
          for (int w = 0; w < kTeams; ++w) {
            f[w][e] = ptx::ex2(x[w].x - ref);
            sum = fmaf(x[w].y, f[w][e], sum);
          }
          R[e] = M;
          L[e] = sum;
        }
        skip = __any_sync(0xFFFFFFFFu, skip);
        if (team == 0 && (lane >> 2) == 0) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = 8 * grp + 2 * lane + e;
            if (!whole)
              reinterpret_cast<float2*>(p.part_rl)[part * p.rows8 + r] = make_float2(R[e], skip ? -1.f : L[e]);
            else if (skip || at.len < 0)
              skip_row(p, it, r);
            else
              store_lse_of(p, it, r, R[e], L[e]);
          }
          if (lane == 0 && grp == 0 && (skip || at.len < 0)) atomicOr(&g_attn_status, skip ? 8u : 2u);
        }
      }
      // This team's 16 of the 64 columns.
      float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kTeams; ++w) {
        const float4 y = xs[((grp * kTeams + w) * 4 + team) * 32 + lane];
        x[0] = fmaf(y.x, f[w][0], x[0]);
        x[1] = fmaf(y.y, f[w][1], x[1]);
        x[2] = fmaf(y.z, f[w][0], x[2]);
        x[3] = fmaf(y.w, f[w][1], x[3]);
      }
      const int dt = 4 * hf + team;
      if (!whole)
        reinterpret_cast<float4*>(p.part_o)[((part * (p.rows8 / 8) + grp) * 8 + dt) * 32 + lane] =
            make_float4(x[0], x[1], x[2], x[3]);
      else if (!skip && at.len >= 0)
        store_out(p, it, grp, dt, lane, x, __frcp_rn(L[0]), __frcp_rn(L[1]));
    }
    if (!ends && t_first == 0 && threadIdx.x == 0) p.cuts[blockIdx.x] = {it.b, at.item, at.parts(run, kCost), 0};
    if (i + 1 < n) at.step(p, per, kCost);
  }
}

// ---------------------------------------------------------------- many rows
// Blocks of 17 to 128 rows, on the tensor cores: S = Q K^T and O = P V as 128 x 64 x 128 and 128 x 128
// x 64 products, Q and P in tensor memory. A block of up to 32 (64) rows stands in the 128 lanes
// four times (twice): each copy takes its own 16 (32) of a unit's 64 keys and has zeros for P
// elsewhere, so that all four warps have a share of the exponentials; the copies are added at the
// item's end. A lane keeps its row of O in registers: what the tensor cores have summed over at most
// four units is added to it, to nearest; a warp with a row whose reference rises does so at once.
//
// The CTA goes through a unit in step: loads (cp.async, two units ahead), S, exponentials, P V; two CTAs
// an SM fill each other's waits. P V is waited for before the next S is issued (2 us of the case below). 48 x 5
// drafted tokens of 28/4 heads (35 rows, caches of up to 5003 keys, 244 MB): 65 to 68 us, 3.7 TB/s; the join 10 by itself.
// By warp-level products it was 154 to 205 us: one of 16 x 8 x 16 occupies a quarter of an SM's tensor cores
// for some 24 to 32 cycles, and there are 144 of them for every 16 keys. Bound by the instructions of 8 warps an SM
// (issue slots 36% busy): O takes 128 registers a lane, so there is no room for more. P enters as two bf16 terms
// (few_rows.cuh says what that leaves); a third would need 32 columns of tensor memory that two CTAs an SM do not have.
constexpr int kRowsThreads = 128;
constexpr int kRowsStages = 3;
constexpr int kRowsTile = kUnit * kD * 2;                 // 16 KiB: a unit's K or V, as two halves of 64 columns
constexpr int kRowsStage = 2 * kRowsTile;
constexpr int kRowsOffX = kRowsStages * kRowsStage;       // 16 columns of every lane's row
constexpr int kXPitch = 20;                               // floats: distinct banks
constexpr int kRowsOffMl = kRowsOffX + 128 * kXPitch * 4; // [lane of 128][2] floats
constexpr int kRowsOffBar = kRowsOffMl + 128 * 8;
constexpr int kRowsSmem = kRowsOffBar + 64 + 1024;        // slack to align the base to 1024 bytes
static_assert(2 * (kRowsSmem + 1024 + 256) <= 228 * 1024, "two CTAs an SM");
constexpr int kRowsFold = 4;                              // units that O is summed over in tensor memory
constexpr uint32_t kColS = 0, kColQ = 64, kColO = 128, kRowsCols = 256;  // tensor memory; P stands in S's place

// Shared-memory offset of 16-byte chunk c of key r in a tile: 128-byte swizzle, 64 columns a half.
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
  return static_cast<uint32_t>((c >> 3) * (kRowsTile / 2) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// S = Q K^T, Q in tensor memory (K-major, 8 columns for 16 of head_dim), K the K-major B operand:
// steps 4..7 use the second half, 8 KiB further.
template <int... kK>
__device__ __forceinline__ void issue_rows_s(uint32_t tmem, uint32_t k_lo, std::integer_sequence<int, kK...>) {
  constexpr uint32_t idesc = idesc_bf16(128, kUnit, 0);
  (ptx::mma_ts_warp<8 * kK, ((kK >> 2) << 9) + ((kK & 3) << 1)>(tmem + kColS, tmem + kColQ, k_lo, kDescHi, idesc,
                                                                kK > 0 ? 1u : 0u),
   ...);
}
// O += P_hi V + P_lo V (from 0 unless `accumulate`): 16 columns of P for 16 keys, P_hi in the first 8; V the
// MN-major B operand, 16 keys 2048 bytes.
template <int... kK>
__device__ __forceinline__ void issue_rows_pv(uint32_t tmem, uint32_t v_lo, uint32_t accumulate,
                                              std::integer_sequence<int, kK...>) {
  constexpr uint32_t idesc = idesc_bf16(128, kD, 1);
  ((ptx::mma_ts_warp<16 * kK + 8, (kK << 7)>(tmem + kColO, tmem + kColS, v_lo, kDescHi, idesc,
                                             kK == 0 ? accumulate : 1u),
    ptx::mma_ts_warp<16 * kK, (kK << 7)>(tmem + kColO, tmem + kColS, v_lo, kDescHi, idesc, 1u)),
   ...);
}

// Where column d of row r stands in a part's rows (attn_paged_fwd's order): in floats.
__device__ __forceinline__ int part_place(int r, int d) {
  const int lane = (d & 7) * 4 + ((r & 7) >> 1), e = (r & 1) + ((d & 8) >> 2);
  return (((r >> 3) * 8 + (d >> 4)) * 32 + lane) * 4 + e;
}

template <int kCopies, bool kMass>
__global__ void __launch_bounds__(kRowsThreads, 2) attn_paged_rows(const Params p) {
  constexpr int kLanes = 128 / kCopies;      // rows of a copy
  constexpr int kChunks = kUnit / 16 / kCopies;  // 16-key chunks of a copy
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int copy = static_cast<int>(threadIdx.x) / kLanes;  // the same for a warp
  const int r = static_cast<int>(threadIdx.x) % kLanes;     // this lane's row of the block
  const float neg_inf = -__int_as_float(0x7F800000);
  const int per = p.Hkv * p.blocks;
  if (threadIdx.x == 0) p.cuts[blockIdx.x].parts = 0;
  Run run;
  constexpr int kCost = kRowsItemCost;
  if (!find_run<kRowsThreads>(p.seqlens, p.B, p.cap, per, kCost, kCost + 1, blockIdx.x, gridDim.x, run)) return;

  const uint32_t base = ptx::smem_u32(smem);
  const uint32_t bar_s = base + kRowsOffBar, bar_o = bar_s + 8, bar_end = bar_s + 16;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kRowsOffBar + 24);
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + kRowsOffBar + 28);
  if (threadIdx.x == 0) {
    ptx::mbar_init(bar_s, 1);
    ptx::mbar_init(bar_o, 1);
    ptx::mbar_init(bar_end, 1);
    ptx::fence_mbar_init();
    *abort_flag = 0;
  }
  if (warp == 0) {
    ptx::tmem_alloc(base + kRowsOffBar + 28, kRowsCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot, mine = tmem + (static_cast<uint32_t>(warp * 32) << 16);

  // ---- loads: a warp 16 keys of every unit, kRowsStages - 1 units ahead.
  const int half = lane >> 4, chunk = lane & 15;
  Walk ahead;
  ahead.start(p, run, kCost);
  uint32_t bad_stages = 0;
  auto look_up = [&]() { return place_of(p, ahead, ahead.t * kUnit + warp * 16 + chunk); };
  auto load = [&](const Place& place, int s) {
    const int row = row_of(p, place);
    const bool bad = __any_sync(0xFFFFFFFFu, row == -2);
    bad_stages = (bad_stages & ~(1u << s)) | (bad ? 1u << s : 0u);
    const uint32_t dst = base + s * kRowsStage;
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const int from = __shfl_sync(0xFFFFFFFFu, row, half + 2 * x);
      const uint32_t d = dst + swizzled(warp * 16 + half + 2 * x, chunk);
      const size_t at = static_cast<size_t>(max(from, 0)) * kD + 8 * chunk;
      ptx::cp_async16(d, p.k + at, from >= 0);
      ptx::cp_async16(d + kRowsTile, p.v + at, from >= 0);
    }
  };
  const int n = run.n;
  Place next = look_up();
#pragma unroll
  for (int s = 0; s < kRowsStages - 1; ++s) {
    if (s < n) {
      load(next, s);
      if (s + 1 < n) {
        ahead.step(p, per, kCost);
        next = look_up();
      }
    }
    ptx::cp_async_commit();
  }

  Walk at;
  at.start(p, run, kCost);
  Item it;
  uint64_t o[kD / 2];                       // the lane's row, column pairs
  float ref = neg_inf, sum = 0.f;
  int lim = 0, min_lim = 0, t_first = 0;
  bool bad = false, fresh = true, ok = true;
  uint32_t phase_s = 0, phase_o = 0;        // phase_o: P V products issued
  bool pv_pending = false;                  // the last one has not been waited for
  int summed = 0;                           // units of O in tensor memory
  auto fold = [&]() {                       // o += what is there
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t y[32];
      ptx::tmem_ld32(mine + kColO + 32 * q, y);
#pragma unroll
      for (int d = 0; d < 16; ++d)
        o[16 * q + d] = ptx::f2_add(o[16 * q + d], ptx::f2_pack(__uint_as_float(y[2 * d]), __uint_as_float(y[2 * d + 1])));
    }
  };
  for (int i = 0; i < n; ++i) {
    if (fresh) {  // an item begins
      fresh = false;
      it = item_of(p, at.b, at.kvh, at.block);
      t_first = at.t;
      bad = false;
      ref = neg_inf;
      sum = 0.f;
      summed = 0;
#pragma unroll
      for (int d = 0; d < kD / 2; ++d) o[d] = 0;
      const bool there = r < it.n_rows && at.len >= 0;
      lim = there ? few::own_limit((it.row0 + r) / p.group, at.len, p.Sq, p.causal) : 0;
      min_lim = few::own_limit(it.row0 / p.group, at.len, p.Sq, p.causal);
      const uint4* from = reinterpret_cast<const uint4*>(
          p.q + (there ? few::query_at(p.layout, p.Hq, p.Sq, p.group, it.b, it.kvh, it.row0 + r) : 0));
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // 32 of head_dim: 16 columns
        uint32_t w[16];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint4 x = there ? __ldg(from + 4 * j + u) : make_uint4(0, 0, 0, 0);
          w[4 * u] = x.x, w[4 * u + 1] = x.y, w[4 * u + 2] = x.z, w[4 * u + 3] = x.w;
        }
        ptx::tmem_st16(mine + kColQ + 16 * j, w);
      }
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
    }
    const int s = i % kRowsStages;
    const uint32_t kt = base + s * kRowsStage, vt = kt + kRowsTile;
    ptx::cp_async_wait<kRowsStages - 2>();
    // A non-finite element of V times a weight of 0 (a hidden key's, another copy's) would be a NaN:
    // such a unit goes key by key. Each lane looks at what it copied.
    uint32_t acc = 0;
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const uint4 v = ptx::ld_shared_v4(vt + swizzled(warp * 16 + half + 2 * x, chunk));
      acc = ptx::bf16x2_nonfinite_acc(v.x, ptx::bf16x2_nonfinite_acc(v.y, acc));
      acc = ptx::bf16x2_nonfinite_acc(v.z, ptx::bf16x2_nonfinite_acc(v.w, acc));
    }
    ptx::fence_proxy_async_smem();  // the copies, before the tensor cores read them
    const bool apart = __syncthreads_or(acc != 0);
    if (warp == 0) {
      // S comes where the last unit's P stands: products of other shapes and accumulators have no order of
      // their own.
      if (pv_pending) ok = warp_wait(bar_o, (phase_o & 1) ^ 1, abort_flag, p.timeout_ns) && ok;
      ptx::tc_fence_after();
      if (ok) {
        issue_rows_s(tmem, desc_lo(kt, 16), std::make_integer_sequence<int, 8>{});
        if (!p.withhold) ptx::mma_commit_warp(bar_s);
      }
    }
    pv_pending = false;
    bad = bad || (bad_stages >> s & 1u);
    // ---- the copy's 16 kChunks keys of S; the products before it are done too.
    ok = warp_wait(bar_s, phase_s & 1, abort_flag, p.timeout_ns) && ok;
    ++phase_s;
    ptx::tc_fence_after();
    if (i + kRowsStages - 1 < n && ok) load(next, (i + kRowsStages - 1) % kRowsStages);  // where unit i - 1 was
    ptx::cp_async_commit();
    if (i + kRowsStages < n) {
      ahead.step(p, per, kCost);
      next = look_up();
    }
    uint32_t x[kChunks][16];
#pragma unroll
    for (int u = 0; u < kChunks; ++u) ptx::tmem_ld16_nowait(mine + kColS + 16 * (copy * kChunks + u), x[u]);
#pragma unroll
    for (int u = 0; u < kChunks; ++u) ptx::tmem_wait_ld16(x[u]);
    const int key0 = at.t * kUnit + copy * 16 * kChunks;
    const uint64_t c2 = ptx::f2_pack(p.c, p.c);
    uint64_t v[kChunks][8];  // logits of key pairs, log2 units
#pragma unroll
    for (int u = 0; u < kChunks; ++u)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[u][j] = ptx::f2_mul(ptx::f2_pack(__uint_as_float(x[u][2 * j]), __uint_as_float(x[u][2 * j + 1])), c2);
    if (key0 + 16 * kChunks > min_lim) {  // some row does not see some key
#pragma unroll
      for (int u = 0; u < kChunks; ++u)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float lo, hi;
          ptx::f2_unpack(v[u][j], lo, hi);
          if (key0 + 16 * u + 2 * j >= lim) lo = neg_inf;
          if (key0 + 16 * u + 2 * j + 1 >= lim) hi = neg_inf;
          v[u][j] = ptx::f2_pack(lo, hi);
        }
    }
    float mx = neg_inf;  // a NaN is left out here and comes back through its weight
#pragma unroll
    for (int u = 0; u < kChunks; ++u)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float lo, hi;
        ptx::f2_unpack(v[u][j], lo, hi);
        mx = fmaxf(mx, fmaxf(lo, hi));
      }
    if constexpr (kMass) {
      if (r < it.n_rows) {
        float* to = p.logits + ((static_cast<size_t>(it.b) * p.Hkv + it.kvh) * p.cap + key0) * p.rows4 + it.row0 + r;
#pragma unroll
        for (int u = 0; u < kChunks; ++u)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float lo, hi;
            ptx::f2_unpack(v[u][j], lo, hi);
            if (key0 + 16 * u + 2 * j < at.len) to[0] = lo;
            if (key0 + 16 * u + 2 * j + 1 < at.len) to[p.rows4] = hi;
            to += 2 * static_cast<size_t>(p.rows4);
          }
      }
    }
    const bool full = summed == kRowsFold || (apart && summed > 0);  // the same for all: O starts from 0 again
    const bool rises = mx > ref + kTau;
    if (full || __any_sync(0xFFFFFFFFu, rises)) {
      if (summed > 0) {
        fold();
        if (!full) {  // the other warps' lanes go on
          const uint32_t zero[16] = {};
#pragma unroll
          for (int q = 0; q < 8; ++q) ptx::tmem_st16(mine + kColO + 16 * q, zero);
        }
      }
      const float f = rises ? ptx::ex2(ref - mx) : 1.f;  // 0 from -Inf
      const uint64_t f2 = ptx::f2_pack(f, f);
#pragma unroll
      for (int d = 0; d < kD / 2; ++d) o[d] = ptx::f2_mul(o[d], f2);
      sum *= f;
      if (rises) ref = mx;
    }
    if (full) summed = 0;
    const float sub = ref == neg_inf ? 0.f : ref;
    const uint64_t sub2 = ptx::f2_pack(-sub, -sub);
    uint64_t sum2 = 0;
#pragma unroll
    for (int u = 0; u < kChunks; ++u) {
      uint32_t w[16];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float w0, w1;
        ptx::f2_unpack(ptx::f2_add(v[u][j], sub2), w0, w1);
        w0 = ptx::ex2(w0);
        w1 = ptx::ex2(w1);
        const uint64_t ww = ptx::f2_pack(w0, w1);
        sum2 = ptx::f2_add(sum2, ww);
        const uint32_t h = ptx::pack_bf16x2(w0, w1);
        w[j] = h;
        float l0, l1;
        ptx::f2_unpack(ptx::f2_sub(ww, ptx::f2_pack(__uint_as_float(h << 16), __uint_as_float(h & 0xFFFF0000u))), l0, l1);
        w[8 + j] = ptx::pack_bf16x2(l0, l1);
      }
      ptx::tmem_st16(mine + kColS + 16 * (copy * kChunks + u), w);
    }
    {
      float s0, s1;
      ptx::f2_unpack(sum2, s0, s1);
      sum += s0 + s1;
    }
    if constexpr (kCopies > 1) {  // zeros at the other copies' keys
      const uint32_t zero[16] = {};
#pragma unroll
      for (int u = kChunks; u < kUnit / 16; ++u)
        ptx::tmem_st16(mine + kColS + 16 * ((copy * kChunks + u) % (kUnit / 16)), zero);
    }
    ptx::tmem_wait_st();
    ptx::tc_fence_before();
    if (__syncthreads_or(!ok)) {
      ok = false;
      break;
    }
    if (!apart) {
      if (warp == 0) {
        ptx::tc_fence_after();
        issue_rows_pv(tmem, desc_lo(vt, kRowsTile / 2), summed > 0 ? 1u : 0u, std::make_integer_sequence<int, 4>{});
        ptx::mma_commit_warp(bar_o);
      }
      ++phase_o;
      pv_pending = true;
      ++summed;
    } else {
      // Key by key over what the row sees, weights read back two at a time.
#pragma unroll 1
      for (int j = 0; j < 8 * kChunks; ++j) {
        const uint32_t col = mine + kColS + 16 * (copy * kChunks + (j >> 3)) + (j & 7);
        const uint32_t h = ptx::tmem_ld1(col), l = ptx::tmem_ld1(col + 8);
#pragma unroll 1
        for (int e = 0; e < 2; ++e) {
          if (key0 + 2 * j + e < lim) {
            const float w = e == 0 ? __uint_as_float(h << 16) + __uint_as_float(l << 16)
                                   : __uint_as_float(h & 0xFFFF0000u) + __uint_as_float(l & 0xFFFF0000u);
            const uint64_t w2 = ptx::f2_pack(w, w);
            const int key = copy * 16 * kChunks + 2 * j + e;
#pragma unroll
            for (int d = 0; d < 16; ++d) {
              const uint4 v = ptx::ld_shared_v4(vt + swizzled(key, d));
              const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int y = 0; y < 4; ++y)
                o[4 * d + y] = ptx::f2_fma(
                    w2, ptx::f2_pack(__uint_as_float(vw[y] << 16), __uint_as_float(vw[y] & 0xFFFF0000u)), o[4 * d + y]);
            }
          }
        }
        __syncwarp();  // the loads from tensor memory are the whole warp's
      }
      __syncwarp();
      ptx::tc_fence_before();
    }
    const bool ends = at.t + 1 == at.units;
    if (!ends && i + 1 < n) {
      ++at.t;
      continue;
    }
    // ---- the item's end, or the run's: the copies are added, 16 columns at a time.
    // (Its last unit's P V, if that was not key by key: the ones before it are waited for already.)
    if (summed > 0) {
      ok = warp_wait(bar_o, (phase_o & 1) ^ 1, abort_flag, p.timeout_ns);
      pv_pending = false;
      ptx::tc_fence_after();
      fold();
      ptx::tc_fence_before();
    }
    fresh = true;
    const bool whole = ends && t_first == 0;
    const int failed = __syncthreads_or((bad ? 1 : 0) | (ok ? 0 : 2));
    if (__syncthreads_or(!ok)) {
      ok = false;
      break;
    }
    const bool skip = failed != 0;
    float2* ml = reinterpret_cast<float2*>(smem + kRowsOffMl);
    ml[threadIdx.x] = make_float2(ref, sum);
    __syncthreads();
    float M = neg_inf, L = 0.f;
#pragma unroll
    for (int y = 0; y < kCopies; ++y) M = fmaxf(M, ml[y * kLanes + r].x);
    const float m0 = M == neg_inf ? 0.f : M, scale = ptx::ex2(ref - m0);
#pragma unroll
    for (int y = 0; y < kCopies; ++y) {
      const float2 z = ml[y * kLanes + r];
      L = fmaf(z.y, ptx::ex2(z.x - m0), L);
    }
    const size_t part = 2 * static_cast<size_t>(blockIdx.x) + (t_first == 0 ? 1 : 0);
    const float inv = __frcp_rn(L);
    float* xs = reinterpret_cast<float*>(smem + kRowsOffX);
    constexpr int kN = 16 / kCopies;  // columns of a lane in the end, of every 16
    const bool there = r < it.n_rows && dbg_ok(it.row0 + r < p.rows && it.b < p.B && it.kvh < p.Hkv);
    float* to_part = p.part_o + part * p.rows8 * kD + part_place(r, copy * kN);
    uint16_t* to_out =
        p.out + (there ? few::query_at(p.layout, p.Hq, p.Sq, p.group, it.b, it.kvh, it.row0 + r) : 0) + copy * kN;
    const bool good = !skip && at.len >= 0;
    // A short loop that moves the row along, not eight copies of its body (48 x 5 drafted tokens 80 -> 75 us, of
    // which kRowsItemCost 4 for 3 is one).
#pragma unroll 1
    for (int q = 0; q < 8; ++q) {
      float y[16];
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        float lo, hi;
        ptx::f2_unpack(o[d], lo, hi);
        y[2 * d] = lo * scale;
        y[2 * d + 1] = hi * scale;
      }
#pragma unroll
      for (int d = 0; d < kD / 2 - 8; ++d) o[d] = o[d + 8];
      if constexpr (kCopies > 1) {
#pragma unroll
        for (int d = 0; d < 4; ++d)
          *reinterpret_cast<float4*>(xs + threadIdx.x * kXPitch + 4 * d) = make_float4(y[4 * d], y[4 * d + 1], y[4 * d + 2], y[4 * d + 3]);
        __syncthreads();
#pragma unroll
        for (int d = 0; d < kN; ++d) y[d] = 0.f;
#pragma unroll
        for (int z = 0; z < kCopies; ++z)
#pragma unroll
          for (int d = 0; d < kN; d += 4) {
            const float4 v = *reinterpret_cast<const float4*>(xs + (z * kLanes + r) * kXPitch + copy * kN + d);
            y[d] += v.x;
            y[d + 1] += v.y;
            y[d + 2] += v.z;
            y[d + 3] += v.w;
          }
        __syncthreads();
      }
      if (there && !whole) {
        // Columns copy * kN + d of 16: d's bits 0..2 and the rest of them apart in part_place.
#pragma unroll
        for (int d = 0; d < kN; ++d) to_part[q * 128 + (d & 7) * 16 + (d & 8) / 4] = y[d];
      } else if (there && good) {
#pragma unroll
        for (int d = 0; d < kN; d += 4)
          *reinterpret_cast<uint2*>(to_out + 16 * q + d) =
              make_uint2(round_bf16_bits(y[d] * inv, p.mode) | (round_bf16_bits(y[d + 1] * inv, p.mode) << 16),
                         round_bf16_bits(y[d + 2] * inv, p.mode) | (round_bf16_bits(y[d + 3] * inv, p.mode) << 16));
      }
    }
    if (copy == 0) {
      if (!whole)
        reinterpret_cast<float2*>(p.part_rl)[part * p.rows8 + r] = make_float2(M, skip ? -1.f : L);
      else if (skip || at.len < 0)
        skip_row(p, it, r);
      else
        store_lse_of(p, it, r, M, L);
    }
    if (threadIdx.x == 0) {
      if (skip || at.len < 0) atomicOr(&g_attn_status, skip ? 8u : 2u);
      if (!ends && t_first == 0) p.cuts[blockIdx.x] = {it.b, at.item, at.parts(run, kCost), 0};
    }
    if (i + 1 < n) at.step(p, per, kCost);
  }
  // ---- copies and products that are still under way (after a wait that ran out), then the end.
  ptx::cp_async_wait<0>();
  if (warp == 0) {
    ptx::mma_commit_warp(bar_end);
    wait_bounded(bar_end, 0, abort_flag, p.timeout_ns, false);
    __syncwarp();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 0) ptx::tmem_dealloc(tmem, kRowsCols);
}

// ---------------------------------------------------------------- join and masses
constexpr int kJoinThreads = 32 * 8;  // times kSplits
// An item has at most runs / (kv heads * blocks) + 2 parts, as all of a sequence's are as long; with
// more than this many, four warps share them. (With four always, 1024-thread blocks that mostly leave at
// once took 5 waves: 14 us for 48 x 35 rows.)
constexpr int kJoinFew = 96;
constexpr int kJoinBatch = 8;         // parts on their way at once
constexpr int kMassUnits = 2;         // of a run of keys at least
constexpr int kMassRows = 256;        // whose log-sum-exp a block holds at once
constexpr int kMassKeys = 4;          // of a thread at once

__device__ __forceinline__ size_t part_at(int run, bool begins) { return 2 * static_cast<size_t>(run) + (begins ? 1 : 0); }

// The cut item of `run`, if it has one, rows 8 g .. 8 g + 7. A warp takes 16 columns of every kSplits-th
// part; parts are added in a fixed order.
template <int kSplits>
__device__ __forceinline__ void join(const Params& p, int run, int g) {
  extern __shared__ __align__(16) float weights[];  // [part][8 rows]
  __shared__ float4 sum_o[kSplits][8][32];          // of split 0: not used
  __shared__ float row_r[8], row_l[8];
  const Cut cut = p.cuts[run];
  if (cut.parts == 0) return;
  const int kvh = cut.item / p.blocks;
  const Item it = item_of(p, cut.b, kvh, cut.item - kvh * p.blocks);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (8 * g >= it.n_rows || !dbg_ok(cut.b < p.B && cut.parts <= p.runs - run)) return;
  const float neg_inf = -__int_as_float(0x7F800000);
  const float2* rl = reinterpret_cast<const float2*>(p.part_rl);
  // ---- a warp a row: the largest reference, the parts' weights, the sum.
  bool skip = false;
  if (warp < 8) {
    float R = neg_inf;
    for (int i = lane; i < cut.parts; i += 32) {
      const float2 x = rl[part_at(run + i, i == 0) * p.rows8 + 8 * g + warp];
      R = fmaxf(R, x.x);  // a NaN is left out: it comes back through its weight
      skip = skip || x.y < 0.f;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) R = fmaxf(R, __shfl_xor_sync(0xFFFFFFFFu, R, d));
    const float ref = R == neg_inf ? 0.f : R;
    float L = 0.f;
    for (int i = lane; i < cut.parts; i += 32) {
      const float2 x = rl[part_at(run + i, i == 0) * p.rows8 + 8 * g + warp];
      const float w = ptx::ex2(x.x - ref);
      weights[8 * i + warp] = w;
      L = fmaf(x.y, w, L);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) L += __shfl_xor_sync(0xFFFFFFFFu, L, d);
    if (lane == 0) {
      row_r[warp] = R;
      row_l[warp] = L;
    }
  }
  if (__syncthreads_or(skip)) return;  // a page of the sequence could not be read
  const int dt = warp & 7, split = warp >> 3;
  float x[4] = {0.f, 0.f, 0.f, 0.f};
  const float4* part_o = reinterpret_cast<const float4*>(p.part_o) + (g * 8 + dt) * 32 + lane;
  const size_t pitch = p.rows8 / 8 * 8 * 32;
  for (int i0 = split; i0 < cut.parts; i0 += kJoinBatch * kSplits) {
    float4 y[kJoinBatch];
#pragma unroll
    for (int j = 0; j < kJoinBatch; ++j) {
      const int i = i0 + j * kSplits;
      y[j] = i < cut.parts ? part_o[part_at(run + i, i == 0) * pitch] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int j = 0; j < kJoinBatch; ++j) {
      const int i = i0 + j * kSplits;
      if (i >= cut.parts) break;
      const float2 w = *reinterpret_cast<const float2*>(weights + 8 * i + 2 * (lane & 3));
      x[0] = fmaf(y[j].x, w.x, x[0]);
      x[1] = fmaf(y[j].y, w.y, x[1]);
      x[2] = fmaf(y[j].z, w.x, x[2]);
      x[3] = fmaf(y[j].w, w.y, x[3]);
    }
  }
  if constexpr (kSplits > 1) {
    if (split != 0) sum_o[split][dt][lane] = make_float4(x[0], x[1], x[2], x[3]);
    __syncthreads();
    if (split != 0) return;
  }
#pragma unroll
  for (int w = 1; w < kSplits; ++w) {
    const float4 y = sum_o[w][dt][lane];
    x[0] += y.x;
    x[1] += y.y;
    x[2] += y.z;
    x[3] += y.w;
  }
  const int r = 2 * (lane & 3);
  store_out(p, it, g, dt, lane, x, __frcp_rn(row_l[r]), __frcp_rn(row_l[r + 1]));
  if (threadIdx.x < 8) store_lse_of(p, it, 8 * g + threadIdx.x, row_r[threadIdx.x], row_l[threadIdx.x], false);
}

// A row's log-sum-exp, log2 units, from what the runs left: its item's single run wrote it, or the parts
// are added here as join adds them (beside this block, so not by way of it), a lane every 32nd part. +Inf:
// not to be used. first: the place of the sequence, whose items have `units` units; total and runs of the
// kernel of the runs. A warp.
__device__ __forceinline__ float row_lse2(const Params& p, int b, int kvh, int row, long long first, int units,
                                          long long total, int runs, int lane) {
  const int block = row / p.block_rows, r = row - block * p.block_rows;
  const long long place = first + static_cast<long long>(kvh * p.blocks + block) * (units + p.cost);
  const int i0 = run_of(place + p.cost, total, runs), i1 = run_of(place + p.cost + units - 1, total, runs);
  if (i0 == i1) return p.lse2[(static_cast<size_t>(b) * p.Hkv + kvh) * p.rows4 + row];
  const float inf = __int_as_float(0x7F800000);
  const float2* rl = reinterpret_cast<const float2*>(p.part_rl) + r;
  float R = -inf, L = 0.f;
  bool skip = false;
  for (int i = i0 + lane; i <= i1; i += 32) {
    const float2 x = rl[part_at(i, i == i0) * p.rows8];
    skip = skip || x.y < 0.f;
    R = fmaxf(R, x.x);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) R = fmaxf(R, __shfl_xor_sync(0xFFFFFFFFu, R, d));
  const float ref = R == -inf ? 0.f : R;
  for (int i = i0 + lane; i <= i1; i += 32) {
    const float2 x = rl[part_at(i, i == i0) * p.rows8];
    L = fmaf(x.y, ptx::ex2(x.x - ref), L);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) L += __shfl_xor_sync(0xFFFFFFFFu, L, d);
  return __any_sync(0xFFFFFFFFu, skip) ? inf : R + log2f(L);
}

// mass[b, kvh, j] += sum over the rows that see key j of 2^(s_ij - lse_i), a key a thread, the
// rows in order. A row whose log-sum-exp is -Inf (it sees no key) adds nothing. Runs of keys, `index` of
// `count`.
template <int kBlock>
__device__ __forceinline__ void add_mass(const Params& p, int index, int count) {
  __shared__ __align__(16) float lse2[kMassRows];
  const float inf = __int_as_float(0x7F800000);
  Run run;
  if (!find_run<kBlock>(p.seqlens, p.B, p.cap, p.Hkv, 0, kMassUnits, index, count, run)) return;
  // The places and runs of the kernel that left the logits.
  const long long total = (run.total + static_cast<long long>(p.Hkv) * p.cost * p.B) * p.blocks;
  const int runs = runs_of(total, p.cost + 1, p.runs);
  long long u = run.lo, first = run.first;
  int b = run.b;
  while (u < run.hi) {
    const int len = __ldg(p.seqlens + b), units = units_of(len, p.cap);
    const int kvh = static_cast<int>((u - first) / units), t_first = static_cast<int>((u - first) % units);
    const long long left = run.hi - u;
    const int t_end = left < units - t_first ? t_first + static_cast<int>(left) : units;
    const int here = b;
    const long long place = (first + static_cast<long long>(p.Hkv) * p.cost * b) * p.blocks;
    u += t_end - t_first;
    if (u == first + static_cast<long long>(units) * p.Hkv) {
      first = u;
      ++b;
    }
    if (len < 0 || len > p.cap) continue;
    const size_t head = static_cast<size_t>(here) * p.Hkv + kvh;
    const int end = min(t_end * kUnit, len);
    for (int r0 = 0; r0 < p.rows; r0 += kMassRows) {
      const int n = min(kMassRows, p.rows - r0);
      __syncthreads();  // the rows before have been read
      bool skip = false;
      for (int r = threadIdx.x >> 5; r < n; r += kBlock / 32) {
        const float x = row_lse2(p, here, kvh, r0 + r, place, units, total, runs, threadIdx.x & 31);
        if ((threadIdx.x & 31) == 0) lse2[r] = x;
        skip = skip || x == inf;
      }
      if (__syncthreads_or(skip)) break;  // a page of the sequence could not be read: so say all its rows
      for (int base = t_first * kUnit; base < end; base += kMassKeys * kBlock) {
        float sum[kMassKeys] = {};
        int key[kMassKeys];
#pragma unroll
        for (int j = 0; j < kMassKeys; ++j) key[j] = base + j * kBlock + static_cast<int>(threadIdx.x);
        float* to = p.mass + head * p.cap;
        float was[kMassKeys];
#pragma unroll
        for (int j = 0; j < kMassKeys; ++j) was[j] = key[j] < end ? to[key[j]] : 0.f;
        for (int r = 0; r < n; r += 4) {
          const float4 l4 = *reinterpret_cast<const float4*>(lse2 + r);
          const float lv[4] = {l4.x, l4.y, l4.z, l4.w};
          float4 s4[kMassKeys];
#pragma unroll
          for (int j = 0; j < kMassKeys; ++j)
            if (key[j] < end)
              s4[j] = *reinterpret_cast<const float4*>(p.logits + (head * p.cap + key[j]) * p.rows4 + r0 + r);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (r + e >= n || lv[e] == -inf) continue;
            const int lim = p.causal ? few::own_limit((r0 + r + e) / p.group, len, p.Sq, 1) : len;
#pragma unroll
            for (int j = 0; j < kMassKeys; ++j) {
              const float s = e == 0 ? s4[j].x : e == 1 ? s4[j].y : e == 2 ? s4[j].z : s4[j].w;
              if (key[j] < end && key[j] < lim) sum[j] += ptx::ex2(s - lv[e]);
            }
          }
        }
#pragma unroll
        for (int j = 0; j < kMassKeys; ++j)
          if (key[j] < end) to[key[j]] = was[j] + sum[j];
      }
    }
  }
}

// Blocks of join (run by run, join_groups each), and behind them those of the masses.
template <int kSplits, bool kMass>
__global__ void __launch_bounds__(kJoinThreads * kSplits, kSplits == 1 ? 4 : 1) attn_paged_finish(const Params p) {
  ptx::grid_dependency_wait();
  const int joins = p.runs * p.join_groups, block = blockIdx.x;
  if (block < joins) {
    join<kSplits>(p, block / p.join_groups, block % p.join_groups);
    return;
  }
  if constexpr (kMass) add_mass<kJoinThreads * kSplits>(p, block - joins, static_cast<int>(gridDim.x) - joins);
}

}  // namespace paged
}  // namespace attn
