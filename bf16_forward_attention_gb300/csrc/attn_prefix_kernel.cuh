// attn_prefix_kernel.cuh - attention of a batch whose sequences share a prefix.
//
// Every query sees the Sp shared keys and the keys of its own sequence. With the two
// parts' unnormalised sums O_s, l_s relative to references r_s (log2 units),
//   O = sum_s 2^(r_s - R) O_s / sum_s 2^(r_s - R) l_s,   lse = ln 2 (R + log2 L),
// for any R. The parts are computed apart and joined:
//   * the prefix, once for all sequences: the queries of one key/value head (all
//     sequences, all heads of the group) are packed as the rows of one product
//     with the prefix, which the fused kernel's split form computes on the tensor
//     cores; the prefix is read once per 256 rows instead of once per sequence;
//   * each sequence's own keys, by attn_prefix_own below: few rows against keys
//     that nobody else reads, so it is bound by HBM. It runs beside the prefix product,
//     on the SMs that this leaves: one is bound by the tensor cores, the other by memory;
//   * the join, attn_prefix_join, in a fixed order.
#pragma once
#include "attn_fwd_kernel.cuh"

namespace attn {
namespace prefix {

constexpr int kWarps = 4;
constexpr int kOwnThreads = 32 * kWarps;
constexpr int kKeys = 16;                       // keys per warp tile
constexpr int kKvBytes = kKeys * kD * 2;        // 4 KiB: a tile of K or of V
constexpr int kOwnStages = 3;
constexpr int kWarpBytes = kOwnStages * 2 * kKvBytes;
constexpr int kMaxRows = 32;                    // rows of a block at most
constexpr int kOwnOffQ = kWarps * kWarpBytes;   // the block's queries
constexpr int kOwnOffMl = kOwnOffQ + kMaxRows * kD * 2;  // [warp][row][2] floats
constexpr int kOwnSmem = kOwnOffMl + kWarps * kMaxRows * 8;
constexpr int kFoldKeys = 16384;                // keys of a part beyond which kFold is taken
constexpr int kRowPitch = kD + 4;               // fp32 rows in shared memory: distinct banks
static_assert(kWarpBytes >= kMaxRows * kRowPitch * 4, "a warp's stages hold its fp32 rows at the end");

struct OwnParams {
  const uint16_t* q;
  const uint16_t* k;       // caches: (B, cap, Hkv, 128) or (B, Hkv, cap, 128)
  const uint16_t* v;
  const uint16_t* kp;      // the prefix, when its rows are few (prefix_items > 0)
  const uint16_t* vp;
  const int* seqlens;      // keys of each sequence, 0..cap
  int beside_prefix;       // the launch before this one is the prefix product
  float* part_o;           // [part][kv head][rows_pad][128], the prefix's parts first
  float* part_rl;          // [part][kv head][rows_pad][2]
  int B, Hq, Hkv, group, Sq, Sp, cap, layout, causal;
  int rows;                // B * Sq * group: packed rows of a kv head
  int rows_pad;
  int own_splits, own_blocks;        // blocks of block_rows rows per (sequence, kv head)
  int prefix_splits;
  int block_rows;          // at most 8 * kNT
  int prefix_items;        // the grid's first blocks: prefix, all packed rows of a kv head each
  float c;                 // scale * log2(e)
};

// Packed row r of a kv head is token (r / group) of the batch, head r % group of the
// group. Element offset of its query (or output) row.
__device__ __forceinline__ size_t query_at(int layout, int Hq, int Sq, int group, int kvh, int r) {
  const unsigned tok = static_cast<unsigned>(r) / static_cast<unsigned>(group);
  const int h = kvh * group + r - static_cast<int>(tok) * group;
  if (layout != 0) return (static_cast<size_t>(tok) * Hq + h) * kD;
  const unsigned b = tok / static_cast<unsigned>(Sq);
  return ((static_cast<size_t>(b) * Hq + h) * Sq + (tok - b * Sq)) * kD;
}

// Keys of its own sequence that query token i sees.
__device__ __forceinline__ int own_limit(int i, int len, int Sq, int causal) {
  return causal ? max(0, min(len, i + len - Sq + 1)) : len;
}

// Shared-memory offset of 16-byte chunk c of row r: the chunk's low bits are turned by
// the row, so that the 8 rows of an ldmatrix lie in distinct banks.
__device__ __forceinline__ uint32_t kv_at(int r, int c) {
  return static_cast<uint32_t>(r * 256 + ((c ^ (r & 7)) << 4));
}

// This kernel starts while the prefix product runs and reads nothing of it; its last block
// stays until that grid has finished, so that the end of this grid is the end of both.
__device__ __forceinline__ void end_with_prefix(const OwnParams& p) {
  if (p.beside_prefix && blockIdx.x == gridDim.x - 1) ptx::grid_dependency_wait();
}

// The queries of each kv head as consecutive rows, in the layout of a batch of one: 16
// bytes a thread.
struct PackParams {
  const uint16_t* q;
  uint16_t* packed;
  int Hq, Hkv, group, Sq, layout, rows;
};

constexpr int kPackThreads = 256;

__global__ void __launch_bounds__(kPackThreads) attn_prefix_pack(const PackParams p) {
  ptx::launch_dependents();
  const long long x = static_cast<long long>(blockIdx.x) * (kPackThreads / 16) + (threadIdx.x >> 4);
  if (x >= static_cast<long long>(p.rows) * p.Hkv) return;
  const int kvh = static_cast<int>(x / p.rows), r = static_cast<int>(x % p.rows);
  const size_t dst = (p.layout == 0 ? static_cast<size_t>(x) : static_cast<size_t>(r) * p.Hkv + kvh) * kD;
  reinterpret_cast<uint4*>(p.packed + dst)[threadIdx.x & 15] = __ldg(
      reinterpret_cast<const uint4*>(p.q + query_at(p.layout, p.Hq, p.Sq, p.group, kvh, r)) + (threadIdx.x & 15));
}

// One block: up to 8 * kNT rows against one split of their keys: a sequence's rows of a
// kv head against its cache, or (few packed rows) those of the whole batch against the
// prefix. The four warps take the 16-key tiles in turn, each with a ring of its own
// (cp.async, 3 stages of 8 KiB: 96 KiB a block in flight or in use, two blocks a SM) and
// no synchronisation but __syncwarp, and are joined in shared memory at the end. Rows
// past the end and keys past the range are zeros.
// The products are transposed, S^T = K Q^T and O^T = V^T P^T, so that the rows are the
// short side of the 16 x 8 x 16 products: with the rows as the long side a decode's 4 to 8
// rows filled a quarter to a half of each product and of the softmax's registers (370
// instructions a tile at 4 rows; 200 this way). A lane holds the same two rows of S^T
// and O^T, and P^T turns into an operand by movmatrix. P enters as two bf16 terms, as in the
// fused kernel. Bound by HBM where ranges are long (256 caches of up to 2048 keys, 8 kv heads,
// 1.1 GB: 165 us, 6.7 TB/s; an SM by itself takes 62 GB/s, so beside the prefix product it
// needs 105 of them for that); a short one is bound by the latency of its first loads and
// the instructions around the loop, kept few for that. 25 to 32 rows a block take all 255
// registers and spill 80 bytes.
// The products' fp32 accumulation truncates, and a warp takes a quarter of a part's keys: with
// O^T as the accumulator throughout, 99.5% of outputs over 131072 unit-normal keys a part came
// within one unit in the last place, 99.88% over 32768 and 99.96% over 16384. kFold: a tile's
// two products start from 0 and are added to O^T to nearest (99.95% at any length); for parts
// of more than kFoldKeys keys. Where HBM is the bound it costs nothing (48 caches of 32768
// keys, 8 kv heads of up to 8 rows: 966 us either way); 24 rows 5%, 32 rows 28%.
template <int kNT, bool kFold>
__global__ void __launch_bounds__(kOwnThreads, 2) attn_prefix_own(const OwnParams p) {
  extern __shared__ __align__(128) uint8_t smem_own[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float neg_inf = -__int_as_float(0x7F800000);
  // ---- which rows and keys.
  int kvh, first, n_rows, len, min_lim, max_lim, split, n_splits, part;
  int i0 = 0;              // own keys: the block's first row within its sequence
  bool causal = false;
  const uint16_t *kb, *vb;  // key 0
  {
    int item = static_cast<int>(blockIdx.x);
    if (item < p.prefix_items) {
      n_splits = p.prefix_splits;
      split = item % n_splits;
      kvh = item / n_splits;
      first = 0;
      n_rows = p.rows;
      len = min_lim = max_lim = p.Sp;
      part = split;
      const size_t at = (p.layout == 0 ? static_cast<size_t>(kvh) * p.Sp : static_cast<size_t>(kvh)) * kD;
      kb = p.kp + at;
      vb = p.vp + at;
    } else {
      item -= p.prefix_items;
      n_splits = p.own_splits;
      split = item % n_splits;
      item /= n_splits;
      const int block = item % p.own_blocks;
      item /= p.own_blocks;
      kvh = item % p.Hkv;
      const int b = item / p.Hkv;
      len = __ldg(p.seqlens + b);
      const int R = p.Sq * p.group;  // rows of the sequence
      i0 = block * p.block_rows;
      n_rows = min(p.block_rows, R - i0);
      first = b * R + i0;
      causal = p.causal != 0;
      part = p.prefix_splits + split;
      const size_t at = (p.layout == 0 ? (static_cast<size_t>(b) * p.Hkv + kvh) * p.cap
                                       : static_cast<size_t>(b) * p.cap * p.Hkv + kvh) * kD;
      kb = p.k + at;
      vb = p.v + at;
    }
  }
  dbg_ok(kvh >= 0 && kvh < p.Hkv && first >= 0 && n_rows >= 1 && n_rows <= 8 * kNT && first + n_rows <= p.rows &&
         part < p.prefix_splits + p.own_splits);
  // ---- queries: into shared memory.
  const uint32_t qs = ptx::smem_u32(smem_own) + kOwnOffQ;
#pragma unroll
  for (int it = 0; it < kNT; ++it) {
    const int r = it * 8 + (threadIdx.x >> 4), c = threadIdx.x & 15;
    uint4 x = make_uint4(0, 0, 0, 0);
    if (r < n_rows && dbg_ok(first + r < p.rows))
      x = __ldg(reinterpret_cast<const uint4*>(
                    p.q + query_at(p.layout, p.Hq, p.Sq, p.group, kvh, first + r)) + c);
    ptx::st_shared_v4(qs + kv_at(r, c), x.x, x.y, x.z, x.w);
  }
  const bool own = static_cast<int>(blockIdx.x) >= p.prefix_items;
  if (own) {
    if (len < 0 || len > p.cap) {
      if (threadIdx.x == 0) atomicOr(&g_attn_status, 2u);
      end_with_prefix(p);
      return;
    }
    // Limits rise with the row: the block's least and largest.
    min_lim = own_limit(i0 / p.group, len, p.Sq, causal);
    max_lim = own_limit((i0 + n_rows - 1) / p.group, len, p.Sq, causal);
  }
  const int tiles = (max_lim + kKeys - 1) / kKeys;
  const int t_first = static_cast<int>(static_cast<long long>(tiles) * split / n_splits);
  const int t_end = static_cast<int>(static_cast<long long>(tiles) * (split + 1) / n_splits);

  // Tile t into stage s: a half-warp reads one key's 256 bytes.
  const size_t key_stride = (p.layout == 0 ? 1 : static_cast<size_t>(p.Hkv)) * kD;
  const uint32_t ring = ptx::smem_u32(smem_own) + warp * kWarpBytes;
  const int half = lane >> 4, chunk = lane & 15;
  const uint32_t lane_dst = ring + kv_at(half, chunk);  // keys 2 u + half: + 512 u, chunk turned by 2 u
  auto load = [&](int t, int s) {
    if (!dbg_ok(t >= 0 && t * kKeys < len && len <= (own ? p.cap : p.Sp))) return;
    const int key = t * kKeys + half;
    const size_t at = key * key_stride + 8 * chunk;
    const uint16_t *ks = kb + at, *vs = vb + at;
    const uint32_t dst = lane_dst + s * 2 * kKvBytes;
    if ((t + 1) * kKeys <= len) {  // a whole tile (most): no key to test
#pragma unroll
      for (int u = 0; u < kKeys / 2; ++u) {
        const uint32_t d = (dst ^ ((2 * u & 6) << 4)) + 512 * u;
        ptx::cp_async16(d, ks);
        ptx::cp_async16(d + kKvBytes, vs);
        ks += 2 * key_stride;
        vs += 2 * key_stride;
      }
      return;
    }
#pragma unroll
    for (int u = 0; u < kKeys / 2; ++u) {
      const int ok = key + 2 * u < len;
      const uint32_t d = (dst ^ ((2 * u & 6) << 4)) + 512 * u;
      const size_t step = ok ? 2 * u * key_stride : 0;
      ptx::cp_async16(d, ok ? ks + step : kb, ok);
      ptx::cp_async16(d + kKvBytes, ok ? vs + step : vb, ok);
    }
  };

  // O^T: d = 16 dt + lane / 4 (elements 0, 1) and + 8 (2, 3) of rows 8 nt + 2 (lane % 4)
  // + {0, 1}; S^T has keys in the place of d.
  float o[8][kNT][4];
  float mref[kNT][2], l[kNT][2];
  int lim[kNT][2];  // keys the lane's rows see
#pragma unroll
  for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
    for (int dt = 0; dt < 8; ++dt)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[dt][nt][e] = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 8 * nt + 2 * (lane & 3) + e;
      lim[nt][e] = r >= n_rows ? 0 : causal ? own_limit((i0 + r) / p.group, len, p.Sq, 1) : len;
      mref[nt][e] = neg_inf;
      l[nt][e] = 0.f;
    }
  }
  const int t0 = t_first + warp;
  const int n = t0 < t_end ? (t_end - t0 + kWarps - 1) / kWarps : 0;  // this warp's tiles
#pragma unroll
  for (int s = 0; s < kOwnStages - 1; ++s) {
    if (s < n) load(t0 + s * kWarps, s);
    ptx::cp_async_commit();
  }
  __syncthreads();  // the queries
  uint32_t qf[kNT][4][4];  // Q^T of two 16-column steps each
#pragma unroll
  for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
    for (int k2 = 0; k2 < 4; ++k2)
      ptx::ldmatrix4(qs + kv_at(8 * nt + (lane & 7), 4 * k2 + (lane >> 3)), qf[nt][k2]);
  // Row and chunk of this lane's address in an ldmatrix of K (keys x d), and of V (read
  // transposed).
  const int k_row = (((lane >> 3) & 1) << 3) + (lane & 7), k_chunk = lane >> 4;
  const int v_row = ((lane >> 4) << 3) + (lane & 7), v_chunk = (lane >> 3) & 1;
  for (int i = 0; i < n; ++i) {
    ptx::cp_async_wait<kOwnStages - 2>();
    __syncwarp();  // every lane's copies of this tile; every lane is done with the last one
    if (i + kOwnStages - 1 < n)
      load(t0 + (i + kOwnStages - 1) * kWarps, (i + kOwnStages - 1) % kOwnStages);
    ptx::cp_async_commit();
    const uint32_t kt = ring + (i % kOwnStages) * 2 * kKvBytes, vt = kt + kKvBytes;
    const int key0 = (t0 + i * kWarps) * kKeys;
    const bool masked = key0 + kKeys > min_lim;

    float s[kNT][4];
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      uint32_t kf[4];
      ptx::ldmatrix4(kt + kv_at(k_row, 2 * ks + k_chunk), kf);
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
        ptx::mma_16816(s[nt], kf, qf[nt][ks >> 1][2 * (ks & 1)], qf[nt][ks >> 1][2 * (ks & 1) + 1]);
    }
    uint32_t hi[kNT][2], lo[kNT][2];  // P^T: keys lane / 4 and + 8, the lane's two rows
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      float mx[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        s[nt][e] *= p.c;
        s[nt][2 + e] *= p.c;
        if (masked) {
          if (key0 + (lane >> 2) >= lim[nt][e]) s[nt][e] = neg_inf;
          if (key0 + (lane >> 2) + 8 >= lim[nt][e]) s[nt][2 + e] = neg_inf;
        }
        // The row's largest (a NaN is left out here and comes back through its weight).
        mx[e] = fmaxf(s[nt][e], s[nt][2 + e]);
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xFFFFFFFFu, mx[e], 4));
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xFFFFFFFFu, mx[e], 8));
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xFFFFFFFFu, mx[e], 16));
      }
      const bool need0 = mx[0] > mref[nt][0] + kTau, need1 = mx[1] > mref[nt][1] + kTau;
      if (__any_sync(0xFFFFFFFFu, need0 || need1)) {
        const float f0 = need0 ? ptx::ex2(mref[nt][0] - mx[0]) : 1.f;  // 0 from -Inf
        const float f1 = need1 ? ptx::ex2(mref[nt][1] - mx[1]) : 1.f;
        if (need0) mref[nt][0] = mx[0];
        if (need1) mref[nt][1] = mx[1];
        l[nt][0] *= f0;
        l[nt][1] *= f1;
#pragma unroll
        for (int dt = 0; dt < 8; ++dt) {
          o[dt][nt][0] *= f0;
          o[dt][nt][1] *= f1;
          o[dt][nt][2] *= f0;
          o[dt][nt][3] *= f1;
        }
      }
      const float ref0 = mref[nt][0] == neg_inf ? 0.f : mref[nt][0];
      const float ref1 = mref[nt][1] == neg_inf ? 0.f : mref[nt][1];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float w0 = ptx::ex2(s[nt][2 * u] - ref0), w1 = ptx::ex2(s[nt][2 * u + 1] - ref1);
        l[nt][0] += w0;
        l[nt][1] += w1;
        const uint32_t h = ptx::pack_bf16x2(w0, w1);
        hi[nt][u] = h;
        lo[nt][u] =
            ptx::pack_bf16x2(w0 - __uint_as_float(h << 16), w1 - __uint_as_float(h & 0xFFFF0000u));
      }
    }
    // A key that some row does not see has weight 0 there, and 0 * NaN would carry a
    // non-finite element of its V to that row. Only tiles at the causal edge have
    // such keys; if V holds a non-finite element there, the rows are summed key by
    // key over what they see.
    bool apart = false;
    if (masked && causal) {
      uint32_t acc = 0;
#pragma unroll
      for (int u = 0; u < kKvBytes / 512; ++u) {
        const uint4 x = ptx::ld_shared_v4(vt + (u * 32 + lane) * 16);
        acc = ptx::bf16x2_nonfinite_acc(x.x, ptx::bf16x2_nonfinite_acc(x.y, acc));
        acc = ptx::bf16x2_nonfinite_acc(x.z, ptx::bf16x2_nonfinite_acc(x.w, acc));
      }
      apart = __any_sync(0xFFFFFFFFu, acc != 0);
    }
    if (!apart) {
      uint32_t ph[kNT][2], pl[kNT][2];
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          ph[nt][u] = ptx::movmatrix_trans(hi[nt][u]);
          pl[nt][u] = ptx::movmatrix_trans(lo[nt][u]);
        }
#pragma unroll
      for (int dt = 0; dt < 8; ++dt) {
        uint32_t vf[4];
        ptx::ldmatrix4_trans(vt + kv_at(v_row, 2 * dt + v_chunk), vf);
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
          if constexpr (kFold) {
            float x[4] = {0.f, 0.f, 0.f, 0.f};
            ptx::mma_16816(x, vf, pl[nt][0], pl[nt][1]);
            ptx::mma_16816(x, vf, ph[nt][0], ph[nt][1]);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[dt][nt][e] += x[e];
          } else {
            ptx::mma_16816(o[dt][nt], vf, ph[nt][0], ph[nt][1]);
            ptx::mma_16816(o[dt][nt], vf, pl[nt][0], pl[nt][1]);
          }
        }
      }
    } else {
#pragma unroll 1
      for (int kk = 0; kk < kKeys; ++kk) {
        const int src = ((kk & 7) << 2) | (lane & 3);
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
          const uint32_t h = __shfl_sync(0xFFFFFFFFu, kk < 8 ? hi[nt][0] : hi[nt][1], src);
          const uint32_t w = __shfl_sync(0xFFFFFFFFu, kk < 8 ? lo[nt][0] : lo[nt][1], src);
          const float w0 = __uint_as_float(h << 16) + __uint_as_float(w << 16);
          const float w1 = __uint_as_float(h & 0xFFFF0000u) + __uint_as_float(w & 0xFFFF0000u);
          const bool see0 = key0 + kk < lim[nt][0], see1 = key0 + kk < lim[nt][1];
#pragma unroll
          for (int dt = 0; dt < 8; ++dt) {
            const float a = ptx::ld_shared_bf16(vt + kv_at(kk, 2 * dt) + 2 * (lane >> 2));
            const float c = ptx::ld_shared_bf16(vt + kv_at(kk, 2 * dt + 1) + 2 * (lane >> 2));
            if (see0) {
              o[dt][nt][0] = fmaf(w0, a, o[dt][nt][0]);
              o[dt][nt][2] = fmaf(w0, c, o[dt][nt][2]);
            }
            if (see1) {
              o[dt][nt][1] = fmaf(w1, a, o[dt][nt][1]);
              o[dt][nt][3] = fmaf(w1, c, o[dt][nt][3]);
            }
          }
        }
      }
    }
  }
  // ---- the warps' rows, joined through shared memory (each warp's own ring).
  ptx::cp_async_wait<0>();
  __syncwarp();
  float* ml = reinterpret_cast<float*>(smem_own + kOwnOffMl) + warp * kMaxRows * 2;
  float* mine = reinterpret_cast<float*>(smem_own + warp * kWarpBytes);
#pragma unroll
  for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float sum = l[nt][e];
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 4);
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 8);
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 16);
      const int r = 8 * nt + 2 * (lane & 3) + e;
      if ((lane >> 2) == 0) {
        ml[2 * r] = mref[nt][e];
        ml[2 * r + 1] = sum;
      }
#pragma unroll
      for (int dt = 0; dt < 8; ++dt) {
        mine[r * kRowPitch + 16 * dt + (lane >> 2)] = o[dt][nt][e];
        mine[r * kRowPitch + 16 * dt + 8 + (lane >> 2)] = o[dt][nt][2 + e];
      }
    }
  }
  __syncthreads();
  // Four rows at a time, a warp a row, four columns a lane.
  const float* all_ml = reinterpret_cast<const float*>(smem_own + kOwnOffMl);
  const size_t row_base = (static_cast<size_t>(part) * p.Hkv + kvh) * p.rows_pad + first;
  for (int r = warp; r < n_rows; r += kWarps) {
    if (!dbg_ok(first + r < p.rows_pad)) continue;
    float2 ml4[kWarps];
    float M = neg_inf;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      ml4[w] = reinterpret_cast<const float2*>(all_ml)[w * kMaxRows + r];
      M = fmaxf(M, ml4[w].x);
    }
    const float ref = M == neg_inf ? 0.f : M;
    float L = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = ptx::ex2(ml4[w].x - ref);
      const float4 y = reinterpret_cast<const float4*>(smem_own + w * kWarpBytes)[r * (kRowPitch / 4) + lane];
      L = fmaf(ml4[w].y, f, L);
      x.x = fmaf(y.x, f, x.x);
      x.y = fmaf(y.y, f, x.y);
      x.z = fmaf(y.z, f, x.z);
      x.w = fmaf(y.w, f, x.w);
    }
    reinterpret_cast<float4*>(p.part_o)[(row_base + r) * (kD / 4) + lane] = x;
    if (lane == 0) reinterpret_cast<float2*>(p.part_rl)[row_base + r] = make_float2(M, L);
  }
  end_with_prefix(p);
}

// ---------------------------------------------------------------- join
struct JoinParams {
  const float* part_o;   // [split][kv head][rows_pad][128], the prefix's splits first
  const float* part_rl;
  const int* seqlens;
  uint16_t* out;
  float* lse;            // (B, Hq, Sq)
  int Hq, Hkv, group, Sq, cap, layout, mode, rows, rows_pad, n_parts;
};

constexpr int kJoinRows = 4;
constexpr int kMaxParts = 128;  // 64 of the prefix, 64 of the own keys

// A warp per packed row, four columns a lane; parts in a fixed order. The parts were just
// written and lie in L2 (2048 rows of 14 parts: 15 MB, some 6 us).
__global__ void __launch_bounds__(32 * kJoinRows) attn_prefix_join(const JoinParams p) {
  const long long x = static_cast<long long>(blockIdx.x) * kJoinRows + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  ptx::grid_dependency_wait();
  if (x >= static_cast<long long>(p.rows) * p.Hkv) return;
  const int kvh = static_cast<int>(x / p.rows), r = static_cast<int>(x % p.rows);
  const int tok = r / p.group, h = kvh * p.group + r % p.group;
  const int b = tok / p.Sq, i = tok % p.Sq;
  if (!dbg_ok(h < p.Hq && static_cast<long long>(b) * p.Sq * p.group < p.rows && p.n_parts <= kMaxParts)) return;
  const int len = __ldg(p.seqlens + b);
  if (len < 0 || len > p.cap) return;  // reported by attn_prefix_own
  const float neg_inf = -__int_as_float(0x7F800000);
  const size_t pitch = static_cast<size_t>(p.Hkv) * p.rows_pad;
  const size_t row0 = static_cast<size_t>(kvh) * p.rows_pad + r;
  // Lane s holds the reference and row sum of parts s, s + 32, ...; the largest
  // reference is a warp's maximum (NaN left out: it comes back through its weight).
  const float2* rl = reinterpret_cast<const float2*>(p.part_rl);
  float2 mine[kMaxParts / 32];
  float R = neg_inf;
#pragma unroll
  for (int u = 0; u < kMaxParts / 32; ++u) {
    const int s = 32 * u + lane;
    mine[u] = s < p.n_parts ? rl[row0 + s * pitch] : make_float2(neg_inf, 0.f);
    R = fmaxf(R, mine[u].x);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) R = fmaxf(R, __shfl_xor_sync(0xFFFFFFFFu, R, d));
  const float ref = R == neg_inf ? 0.f : R;
  float L = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int u = 0; u < kMaxParts / 32; ++u) {
    if (32 * u >= p.n_parts) break;
    mine[u].x = ptx::ex2(mine[u].x - ref);
    const int n = min(32, p.n_parts - 32 * u);
#pragma unroll 8
    for (int s = 0; s < n; ++s) {
      const float w = __shfl_sync(0xFFFFFFFFu, mine[u].x, s), l = __shfl_sync(0xFFFFFFFFu, mine[u].y, s);
      const float4 y =
          *reinterpret_cast<const float4*>(p.part_o + (row0 + (32 * u + s) * pitch) * kD + 4 * lane);
      L = fmaf(l, w, L);
      o.x = fmaf(y.x, w, o.x);
      o.y = fmaf(y.y, w, o.y);
      o.z = fmaf(y.z, w, o.z);
      o.w = fmaf(y.w, w, o.w);
    }
  }
  const float inv = __frcp_rn(L);
  const uint2 w2 = make_uint2(
      round_bf16_bits(o.x * inv, p.mode) | (round_bf16_bits(o.y * inv, p.mode) << 16),
      round_bf16_bits(o.z * inv, p.mode) | (round_bf16_bits(o.w * inv, p.mode) << 16));
  *reinterpret_cast<uint2*>(p.out + query_at(p.layout, p.Hq, p.Sq, p.group, kvh, r) + 4 * lane) = w2;
  if (lane == 0) store_lse(p.lse, (static_cast<size_t>(b) * p.Hq + h) * p.Sq + i, R, L);
}

}  // namespace prefix
}  // namespace attn
