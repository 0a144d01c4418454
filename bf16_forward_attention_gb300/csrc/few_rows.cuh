// few_rows.cuh - few query rows against many keys, a warp at a time: what attention over a
// paged cache does with a tile of 16 keys.
//
// The products are transposed, S^T = K Q^T and O^T = V^T P^T, so that the rows are the short
// side of the 16 x 8 x 16 products. A lane holds rows 2 (lane % 4) + {0, 1} of S^T and
// of O^T alike, and P^T turns into an operand by movmatrix.
//
// P enters as two bf16 terms, as in the fused kernel: a weight is off by 2^-18 of itself at most, an output by
// 2.3e-6 of the outputs' size before it is rounded (4096 unit-normal keys; the tensor pipe's truncation of S
// makes 2e-7). So outputs come within one unit in the last place, and one in 400 differs from what fp32 weights
// round to. A third term makes that one in 1400; it took 173.2 us for 172.3 of a decode step over 64 caches of up
// to 8192 keys with 4 rows, and 227 for 212 with 16. Sums, references and masses are fp32.
//
// A tile's arithmetic is that of attn_prefix_own, which holds its rows otherwise (several groups of 8 a warp): what is
// mended in one belongs in the other.
#pragma once
#include "attn_fwd_kernel.cuh"

namespace attn {
namespace few {

constexpr int kKeys = 16;                // keys of a tile
constexpr int kKvBytes = kKeys * kD * 2; // 4 KiB: a tile of K or of V in shared memory

// Shared-memory offset of 16-byte chunk c of row r: the chunk's low bits are turned by
// the row, so that the 8 rows of an ldmatrix lie in distinct banks.
__device__ __forceinline__ uint32_t row_at(int r, int c) {
  return static_cast<uint32_t>(r * 256 + ((c ^ (r & 7)) << 4));
}

// Keys of its own sequence that query token i of Sq sees, of `len`.
__device__ __forceinline__ int own_limit(int i, int len, int Sq, int causal) {
  return causal ? max(0, len - (Sq - 1 - i)) : len;
}

// The page of key `key`: mul and shift of page_divisor.
__device__ __forceinline__ int page_of(int key, uint32_t mul, int shift) {
  return shift < 0 ? key : static_cast<int>(__umulhi(static_cast<uint32_t>(key), mul) >> shift);
}

// Row r of a (sequence, kv head)'s Sq * group rows, tokens first: element offset of its
// query (or output) row.
__device__ __forceinline__ size_t query_at(int layout, int Hq, int Sq, int group, int b, int kvh, int r) {
  const unsigned i = static_cast<unsigned>(r) / static_cast<unsigned>(group);
  const int h = kvh * group + r - static_cast<int>(i) * group;
  return (layout != 0 ? (static_cast<size_t>(b) * Sq + i) * Hq + h : (static_cast<size_t>(b) * Hq + h) * Sq + i) * kD;
}

// The state of up to 8 rows in one warp. A tile's two products of V start from 0 and are added
// to O^T to nearest: the tensor pipe truncates as it accumulates, which over 8192 unit-normal
// keys a warp would leave 99.88% of outputs within one unit in the last place.
struct Rows {
  float o[8][4];      // O^T: d = 16 dt + lane / 4 (elements 0, 1) and + 8 (2, 3)
  float ref[2];       // the row's reference, log2 units
  float sum[2];       // this lane's share of the row's sum
  int lim[2];         // keys the row sees; 0 for rows past the end
  uint32_t q[4][4];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int dt = 0; dt < 8; ++dt)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[dt][e] = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      ref[e] = -__int_as_float(0x7F800000);
      sum[e] = 0.f;
    }
  }

  // Queries: the lane's words of row lane / 4 at `row` (null: zeros).
  __device__ __forceinline__ void load_q(const uint16_t* row, int lane) {
#pragma unroll
    for (int k2 = 0; k2 < 4; ++k2)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        q[k2][j] = row ? __ldg(reinterpret_cast<const uint32_t*>(row) + 16 * k2 + 4 * j + (lane & 3)) : 0u;
  }

  // One tile: K at kt, V at vt (rows by row_at), keys key0 .. key0 + 15. masked: some row does
  // not see some key of it. check_v: keys that only some rows see may lie in it (the causal
  // edge; keys past the end are zeros). c: scale * log2(e). keep(s): the masked logits, log2
  // units: s[0, 1] of key lane / 4 and [2, 3] of + 8.
  template <typename Keep>
  __device__ __forceinline__ void tile(uint32_t kt, uint32_t vt, int key0, bool masked, bool check_v, float c,
                                       int lane, Keep&& keep) {
    const float neg_inf = -__int_as_float(0x7F800000);
    const int k_row = (((lane >> 3) & 1) << 3) + (lane & 7), k_chunk = lane >> 4;
    const int v_row = ((lane >> 4) << 3) + (lane & 7), v_chunk = (lane >> 3) & 1;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      uint32_t kf[4];
      ptx::ldmatrix4(kt + row_at(k_row, 2 * ks + k_chunk), kf);
      ptx::mma_16816(s, kf, q[ks >> 1][2 * (ks & 1)], q[ks >> 1][2 * (ks & 1) + 1]);
    }
    float mx[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      s[e] *= c;
      s[2 + e] *= c;
      if (masked) {
        if (key0 + (lane >> 2) >= lim[e]) s[e] = neg_inf;
        if (key0 + (lane >> 2) + 8 >= lim[e]) s[2 + e] = neg_inf;
      }
      // The row's largest (a NaN is left out here and comes back through its weight).
      mx[e] = fmaxf(s[e], s[2 + e]);
      mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xFFFFFFFFu, mx[e], 4));
      mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xFFFFFFFFu, mx[e], 8));
      mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xFFFFFFFFu, mx[e], 16));
    }
    keep(s);
    const bool need0 = mx[0] > ref[0] + kTau, need1 = mx[1] > ref[1] + kTau;
    if (__any_sync(0xFFFFFFFFu, need0 || need1)) {
      const float f0 = need0 ? ptx::ex2(ref[0] - mx[0]) : 1.f;  // 0 from -Inf
      const float f1 = need1 ? ptx::ex2(ref[1] - mx[1]) : 1.f;
      if (need0) ref[0] = mx[0];
      if (need1) ref[1] = mx[1];
      sum[0] *= f0;
      sum[1] *= f1;
#pragma unroll
      for (int dt = 0; dt < 8; ++dt) {
        o[dt][0] *= f0;
        o[dt][1] *= f1;
        o[dt][2] *= f0;
        o[dt][3] *= f1;
      }
    }
    const float ref0 = ref[0] == neg_inf ? 0.f : ref[0], ref1 = ref[1] == neg_inf ? 0.f : ref[1];
    uint32_t hi[2], lo[2];  // P^T: keys lane / 4 and + 8, the lane's two rows
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float w0 = ptx::ex2(s[2 * u] - ref0), w1 = ptx::ex2(s[2 * u + 1] - ref1);
      sum[0] += w0;
      sum[1] += w1;
      const uint32_t h = ptx::pack_bf16x2(w0, w1);
      hi[u] = h;
      lo[u] = ptx::pack_bf16x2(w0 - __uint_as_float(h << 16), w1 - __uint_as_float(h & 0xFFFF0000u));
    }
    // A key that some row does not see has weight 0 there, and 0 * NaN would carry a
    // non-finite element of its V to that row: where V holds one, the rows are summed key by
    // key over what they see.
    bool apart = false;
    if (check_v) {
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
      const uint32_t ph[2] = {ptx::movmatrix_trans(hi[0]), ptx::movmatrix_trans(hi[1])};
      const uint32_t pl[2] = {ptx::movmatrix_trans(lo[0]), ptx::movmatrix_trans(lo[1])};
#pragma unroll
      for (int dt = 0; dt < 8; ++dt) {
        uint32_t vf[4];
        ptx::ldmatrix4_trans(vt + row_at(v_row, 2 * dt + v_chunk), vf);
        float x[4] = {0.f, 0.f, 0.f, 0.f};
        ptx::mma_16816(x, vf, pl[0], pl[1]);
        ptx::mma_16816(x, vf, ph[0], ph[1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[dt][e] += x[e];
      }
      return;
    }
#pragma unroll 1
    for (int kk = 0; kk < kKeys; ++kk) {
      const int src = ((kk & 7) << 2) | (lane & 3);
      const uint32_t h = __shfl_sync(0xFFFFFFFFu, kk < 8 ? hi[0] : hi[1], src);
      const uint32_t w = __shfl_sync(0xFFFFFFFFu, kk < 8 ? lo[0] : lo[1], src);
      const float w0 = __uint_as_float(h << 16) + __uint_as_float(w << 16);
      const float w1 = __uint_as_float(h & 0xFFFF0000u) + __uint_as_float(w & 0xFFFF0000u);
      const bool see0 = key0 + kk < lim[0], see1 = key0 + kk < lim[1];
#pragma unroll
      for (int dt = 0; dt < 8; ++dt) {
        const float a = ptx::ld_shared_bf16(vt + row_at(kk, 2 * dt) + 2 * (lane >> 2));
        const float b = ptx::ld_shared_bf16(vt + row_at(kk, 2 * dt + 1) + 2 * (lane >> 2));
        if (see0) {
          o[dt][0] = fmaf(w0, a, o[dt][0]);
          o[dt][2] = fmaf(w0, b, o[dt][2]);
        }
        if (see1) {
          o[dt][1] = fmaf(w1, a, o[dt][1]);
          o[dt][3] = fmaf(w1, b, o[dt][3]);
        }
      }
    }
  }

  // The rows' sums over the lanes that share them.
  __device__ __forceinline__ void finish_sums() {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x = sum[e];
      x += __shfl_xor_sync(0xFFFFFFFFu, x, 4);
      x += __shfl_xor_sync(0xFFFFFFFFu, x, 8);
      x += __shfl_xor_sync(0xFFFFFFFFu, x, 16);
      sum[e] = x;
    }
  }
};

}  // namespace few
}  // namespace attn
