// attn_rope_kernel.cuh - per-head norms of queries and keys with the position rotation, and
// their gradients.
//
// A row x of 128 (one head of one token at position t) becomes
//   u = w o x r,   r = (mean x^2 + eps)^(-1/2),
//   y_a = u_a cos(t, i) - u_b sin(t, i),   y_b = u_b cos(t, i) + u_a sin(t, i)
// for the i-th of rot / 2 pairs (a, b) of columns: (i, i + rot / 2), or (2i, 2i + 1) in the
// interleaved form; columns at and after rot are u. Backwards, with dy turned back to du,
//   dw = sum over rows of du o x r,   dx = r (dn - x r mean(dn o x r)),   dn = w o du.
// All of it in fp32; y and dx are rounded once.
//
// 16 lanes hold a row, 8 columns (16 bytes) each, so both reductions are four shuffles, and a
// pair's other half is in the same lane (interleaved) or in one other lane.
#pragma once
#include "attn_fwd_kernel.cuh"

namespace attn {
namespace rope {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kRows = 8;  // rows a warp takes at once: 4 loads of 16 bytes a lane in flight

// A (B, S, H, 128) tensor wherever its rows lie: element strides.
struct Rows {
  uint16_t* p;
  long long batch, token, head;
};

struct Params {
  Rows q, k, v;            // v: the paged form
  Rows q_out, k_out;       // k_out: the dense form
  const uint16_t* wq;
  const uint16_t* wk;
  const float* cos;        // (max_pos, half)
  const float* sin;
  const int* positions;    // one a token
  const int* slots;        // the paged form: where a token's key and value go, -1: nowhere
  uint16_t* k_pages;
  uint16_t* v_pages;
  long long page_stride;   // elements
  long long items;         // tokens * chunks
  int S, Hq, Hkv, max_pos, half, mode, layout;
  int page_size, n_slots;
  int q_chunks, kv_chunks, chunks;  // of kRows heads, of a token
  float eps;
};

__device__ __forceinline__ uint4 load16(const uint16_t* p) { return *reinterpret_cast<const uint4*>(p); }

__device__ __forceinline__ void unpack8(const uint4& x, float (&f)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8], int mode) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = mode == 0 ? round_pair_bf16_rtne(f[2 * i], f[2 * i + 1])
                     : round_pair_bf16(f[2 * i], f[2 * i + 1], mode == 1 ? 0x8000u : 0u);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint4 shuffle4(const uint4& x, int src) {
  return make_uint4(__shfl_sync(0xFFFFFFFFu, x.x, src), __shfl_sync(0xFFFFFFFFu, x.y, src),
                    __shfl_sync(0xFFFFFFFFu, x.z, src), __shfl_sync(0xFFFFFFFFu, x.w, src));
}

// Sum over the 16 lanes of a row.
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
  return x;
}

// What a lane knows of the rotation: the lane that holds its columns' other halves (itself
// where there are none), their first column, and cos and +-sin of its 8 columns, such that
// y_j = u_j c_j + (the other half's u) s_j.
struct Turn {
  int src, other;
  float c[8], s[8];
};

template <bool kInter>
__device__ __forceinline__ void turn_lane(int lane, int half, Turn& t) {
  const int c0 = 8 * (lane & 15);
  t.src = lane;
  t.other = c0;
  if (!kInter && c0 < 2 * half) {
    const int step = c0 < half ? half : -half;
    t.src = lane + step / 8;
    t.other = c0 + step;
  }
}

template <bool kInter>
__device__ __forceinline__ void turn_load(const Params& p, int lane, int pos, Turn& t) {
  const int c0 = 8 * (lane & 15);
  if (c0 >= 2 * p.half) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      t.c[j] = 1.f;
      t.s[j] = 0.f;
    }
    return;
  }
  const size_t row = static_cast<size_t>(pos) * p.half;
  if constexpr (kInter) {
    const float4 c = __ldg(reinterpret_cast<const float4*>(p.cos + row + c0 / 2));
    const float4 s = __ldg(reinterpret_cast<const float4*>(p.sin + row + c0 / 2));
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      t.c[2 * j] = t.c[2 * j + 1] = cc[j];
      t.s[2 * j] = -ss[j];
      t.s[2 * j + 1] = ss[j];
    }
  } else {
    const bool first = c0 < p.half;
    const size_t at = row + (first ? c0 : c0 - p.half);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float4 c = __ldg(reinterpret_cast<const float4*>(p.cos + at) + u);
      const float4 s = __ldg(reinterpret_cast<const float4*>(p.sin + at) + u);
      const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        t.c[4 * u + j] = cc[j];
        t.s[4 * u + j] = first ? -ss[j] : ss[j];
      }
    }
  }
}

// The other halves of a lane's 8 columns.
template <bool kInter>
__device__ __forceinline__ uint4 others(const uint4& x, int src) {
  if constexpr (kInter)
    return make_uint4(__funnelshift_l(x.x, x.x, 16), __funnelshift_l(x.y, x.y, 16), __funnelshift_l(x.z, x.z, 16),
                      __funnelshift_l(x.w, x.w, 16));
  else
    return shuffle4(x, src);
}

// One warp: up to 8 heads of one token, two rows at a time. Bound by HBM: 512 bytes a row.
template <bool kInter, bool kPaged>
__global__ void __launch_bounds__(kThreads) attn_rope_fwd(const Params p) {
  const int lane = threadIdx.x & 31, half_warp = lane >> 4, c0 = 8 * (lane & 15);
  const long long item = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (item >= p.items) return;
  const int tok = static_cast<int>(item / p.chunks);
  int ch = static_cast<int>(item - static_cast<long long>(tok) * p.chunks);
  const int pos = __ldg(p.positions + tok);
  int slot = 0;
  bool ok = pos >= 0 && pos < p.max_pos;
  if constexpr (kPaged) {
    slot = __ldg(p.slots + tok);
    ok = ok && slot >= -1 && slot < p.n_slots;
  }
  if (!ok) {  // nothing of the token is written
    if (lane == 0) atomicOr(&g_attn_status, 8u);
    return;
  }
  const int kind = ch < p.q_chunks ? 0 : ch < p.q_chunks + p.kv_chunks ? 1 : 2;  // queries, keys, values
  if (kind != 0) ch -= p.q_chunks + (kind == 2 ? p.kv_chunks : 0);
  const int h0 = ch * kRows, n = min(kRows, (kind == 0 ? p.Hq : p.Hkv) - h0);
  const int b = tok / p.S, s = tok - b * p.S;
  const Rows& in = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
  const uint16_t* src = in.p + b * in.batch + s * in.token + h0 * in.head + c0;
  if (!dbg_ok(n >= 1 && ch >= 0)) return;
  uint4 x[kRows / 2];
#pragma unroll
  for (int i = 0; i < kRows / 2; ++i) {
    const int h = 2 * i + half_warp;
    x[i] = h < n ? load16(src + h * in.head) : make_uint4(0, 0, 0, 0);
  }
  // ---- where the rows go.
  uint16_t* dst;
  long long step;  // elements between heads
  if (kPaged && kind != 0) {
    if (slot < 0) return;
    const int page = slot / p.page_size, at = slot - page * p.page_size;
    step = p.layout == 0 ? static_cast<long long>(p.page_size) * kD : kD;
    dst = (kind == 1 ? p.k_pages : p.v_pages) + page * p.page_stride +
          static_cast<long long>(p.layout == 0 ? at : at * p.Hkv) * kD + h0 * step + c0;
    if (kind == 2) {
#pragma unroll
      for (int i = 0; i < kRows / 2; ++i) {
        const int h = 2 * i + half_warp;
        if (h < n) *reinterpret_cast<uint4*>(dst + h * step) = x[i];
      }
      return;
    }
  } else {
    const Rows& out = kind == 0 ? p.q_out : p.k_out;
    dst = out.p + b * out.batch + s * out.token + h0 * out.head + c0;
    step = out.head;
  }
  // ---- y_j = (x_j r) (w_j c_j) + (the other half's x r) (its w s_j).
  Turn t;
  turn_lane<kInter>(lane, p.half, t);
  turn_load<kInter>(p, lane, pos, t);
  {
    const uint16_t* w = kind == 0 ? p.wq : p.wk;
    const uint4 mine = load16(w + c0);
    float f[8];
    unpack8(mine, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) t.c[j] *= f[j];
    unpack8(kInter ? others<kInter>(mine, 0) : load16(w + t.other), f);
#pragma unroll
    for (int j = 0; j < 8; ++j) t.s[j] *= f[j];
  }
#pragma unroll
  for (int i = 0; i < kRows / 2; ++i) {
    if (2 * i >= n) break;
    float a[8], o[8];
    unpack8(x[i], a);
    unpack8(others<kInter>(x[i], t.src), o);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(a[j], a[j], sum);
    const float r = rsqrtf(fmaf(row_sum(sum), 1.f / kD, p.eps));
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = fmaf(o[j] * r, t.s[j], a[j] * r * t.c[j]);
    const int h = 2 * i + half_warp;
    if (h < n) *reinterpret_cast<uint4*>(dst + h * step) = pack8(a, p.mode);
  }
}

// ---------------------------------------------------------------- backward
struct BwdParams {
  Params f;                // q, k, weights, table and positions as in the forward call
  Rows dq_out, dk_out;     // the gradients of what it gave
  Rows dq, dk;
  float* part;             // [block][2][128]
};

constexpr int kBwdWarps = 8;
constexpr int kBwdThreads = 32 * kBwdWarps;

// Persistent blocks: a warp takes 8 rows at a time, first of the queries, then of the keys, and
// sums their terms of dw in registers; a block's sums go to the workspace, where
// attn_rope_join adds them in a fixed order. Bound by HBM: 768 bytes a row (x, dy, dx).
template <bool kInter>
__global__ void __launch_bounds__(kBwdThreads, 2) attn_rope_bwd(const BwdParams bp) {
  __shared__ float sums[2][kBwdWarps][kD];
  const Params& p = bp.f;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half_warp = lane >> 4, c0 = 8 * (lane & 15);
  const long long first = static_cast<long long>(blockIdx.x) * kBwdWarps + warp;
  const long long all = static_cast<long long>(gridDim.x) * kBwdWarps;
  Turn t;
  turn_lane<kInter>(lane, p.half, t);
#pragma unroll 1
  for (int kind = 0; kind < 2; ++kind) {
    const Rows in = kind == 0 ? p.q : p.k, gin = kind == 0 ? bp.dq_out : bp.dk_out, out = kind == 0 ? bp.dq : bp.dk;
    const int H = kind == 0 ? p.Hq : p.Hkv, chunks = kind == 0 ? p.q_chunks : p.kv_chunks;
    const long long items = kind == 0 ? p.items / p.chunks * p.q_chunks : p.items / p.chunks * p.kv_chunks;
    float w[8], dw[8];
    unpack8(load16((kind == 0 ? p.wq : p.wk) + c0), w);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[j] = 0.f;
#pragma unroll 1
    for (long long item = first; item < items; item += all) {
      const int tok = static_cast<int>(item / chunks);
      const int h0 = static_cast<int>(item - static_cast<long long>(tok) * chunks) * kRows, n = min(kRows, H - h0);
      const int pos = __ldg(p.positions + tok);
      if (pos < 0 || pos >= p.max_pos) {  // the token's gradients are not written, and it adds none to dw
        if (lane == 0) atomicOr(&g_attn_status, 8u);
        continue;
      }
      const int b = tok / p.S, s = tok - b * p.S;
      const uint16_t* px = in.p + b * in.batch + s * in.token + h0 * in.head + c0;
      const uint16_t* py = gin.p + b * gin.batch + s * gin.token + h0 * gin.head + c0;
      uint16_t* pd = out.p + b * out.batch + s * out.token + h0 * out.head + c0;
      uint4 x[kRows / 2], y[kRows / 2];
#pragma unroll
      for (int i = 0; i < kRows / 2; ++i) {
        const int h = 2 * i + half_warp;
        x[i] = y[i] = make_uint4(0, 0, 0, 0);
        if (h < n) {
          x[i] = load16(px + h * in.head);
          y[i] = load16(py + h * gin.head);
        }
      }
      turn_load<kInter>(p, lane, pos, t);
#pragma unroll
      for (int i = 0; i < kRows / 2; ++i) {
        if (2 * i >= n) break;
        float a[8], g[8], o[8];
        unpack8(x[i], a);
        unpack8(y[i], g);
        unpack8(others<kInter>(y[i], t.src), o);
        float ss = 0.f, gx = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          g[j] = fmaf(g[j], t.c[j], -o[j] * t.s[j]);  // du: turned back
          ss = fmaf(a[j], a[j], ss);
        }
        const float r = rsqrtf(fmaf(row_sum(ss), 1.f / kD, p.eps));
        const int h = 2 * i + half_warp;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          a[j] *= r;  // x r
          if (h < n) dw[j] = fmaf(g[j], a[j], dw[j]);
          g[j] *= w[j];  // dn
          gx = fmaf(g[j], a[j], gx);
        }
        const float m = row_sum(gx) * (1.f / kD);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = r * fmaf(-m, a[j], g[j]);
        if (h < n) *reinterpret_cast<uint4*>(pd + h * out.head) = pack8(g, p.mode);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[j] += __shfl_xor_sync(0xFFFFFFFFu, dw[j], 16);
    if (half_warp == 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) sums[kind][warp][c0 + j] = dw[j];
    }
  }
  __syncthreads();
  const int kind = threadIdx.x >> 7, col = threadIdx.x & 127;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kBwdWarps; ++i) sum += sums[kind][i][col];
  bp.part[static_cast<size_t>(blockIdx.x) * 2 * kD + threadIdx.x] = sum;
}

struct JoinParams {
  const float* part;
  float* dwq;
  float* dwk;
  int parts;
};

constexpr int kJoinCols = 8, kJoinThreads = 256, kJoinLanes = kJoinThreads / kJoinCols;

// 8 columns a block, 32 threads a column, each over every 32nd part; then in order.
__global__ void __launch_bounds__(kJoinThreads) attn_rope_join(const JoinParams p) {
  __shared__ float sums[kJoinLanes][kJoinCols];
  ptx::grid_dependency_wait();
  const int col = blockIdx.x * kJoinCols + (threadIdx.x & (kJoinCols - 1)), at = threadIdx.x / kJoinCols;
  float s = 0.f;
#pragma unroll 4
  for (int i = at; i < p.parts; i += kJoinLanes) s += p.part[static_cast<size_t>(i) * 2 * kD + col];
  sums[at][threadIdx.x & (kJoinCols - 1)] = s;
  __syncthreads();
  if (at != 0) return;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < kJoinLanes; ++i) s += sums[i][threadIdx.x];
  (col < kD ? p.dwq : p.dwk)[col & (kD - 1)] = s;
}

}  // namespace rope
}  // namespace attn
