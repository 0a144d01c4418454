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
// 8 lanes hold a row, 16 columns each: 8 l .. 8 l + 7 and 64 + 8 l .. in lane l, so that with
// rot = 128 both columns of a pair are in one lane, in either form, and a reduction is three
// shuffles. A warp takes one head of four tokens at a time; the angles of a token stay in its
// lanes' registers from head to head. (16 lanes a row and the same columns apart in two lanes took 82
// instructions a row instead of 37, and was bound by them.)
#pragma once
#include "attn_fwd_kernel.cuh"

namespace attn {
namespace rope {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kTokens = 4;   // of a warp, 8 lanes each
constexpr int kHeads = 4;    // of a chunk: a warp's loads in flight, 4 KiB

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
  int tokens;              // B * S
  int S, Hq, Hkv, max_pos, half, mode, layout;
  int page_size, n_slots;
  int q_chunks, kv_chunks, chunks;  // of a token's heads: queries', keys' (and values'), all
  int parts;               // warps that share four tokens, each every parts-th chunk
  float eps;
};

// A chunk of a token's heads: 0 queries, 1 keys, 2 values.
struct Chunk {
  int kind, h0, n;
};
template <int kHeadsOf>
__device__ __forceinline__ Chunk chunk_of(const Params& p, int c) {
  const int kind = c < p.q_chunks ? 0 : c < p.q_chunks + p.kv_chunks ? 1 : 2;
  const int h0 = (c - (kind == 0 ? 0 : kind == 1 ? p.q_chunks : p.q_chunks + p.kv_chunks)) * kHeadsOf;
  return {kind, h0, min(kHeadsOf, (kind == 0 ? p.Hq : p.Hkv) - h0)};
}

__device__ __forceinline__ uint4 load16(const uint16_t* p) { return *reinterpret_cast<const uint4*>(p); }

// Eight columns as four pairs of fp32, for two products or sums in one instruction.
struct F8 {
  uint64_t p[4];
};
__device__ __forceinline__ F8 unpack8(const uint4& x) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  F8 f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    f.p[i] = ptx::f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  return f;
}

__device__ __forceinline__ uint4 pack8(const F8& f, int mode) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    ptx::f2_unpack(f.p[i], lo, hi);
    w[i] = mode == 0 ? round_pair_bf16_rtne(lo, hi) : round_pair_bf16(lo, hi, mode == 1 ? 0x8000u : 0u);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ F8 both(float x) {
  F8 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) f.p[i] = ptx::f2_pack(x, x);
  return f;
}
__device__ __forceinline__ F8 mul(const F8& a, const F8& b) {
  F8 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) f.p[i] = ptx::f2_mul(a.p[i], b.p[i]);
  return f;
}
__device__ __forceinline__ F8 fma(const F8& a, const F8& b, const F8& c) {
  F8 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) f.p[i] = ptx::f2_fma(a.p[i], b.p[i], c.p[i]);
  return f;
}
// sum a_j b_j over the lane's 8 columns.
__device__ __forceinline__ float dot(const F8& a, const F8& b) {
  uint64_t s = ptx::f2_mul(a.p[0], b.p[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) s = ptx::f2_fma(a.p[i], b.p[i], s);
  float lo, hi;
  ptx::f2_unpack(s, lo, hi);
  return lo + hi;
}

// Sum over the 8 lanes of a row.
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int d = 4; d > 0; d >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
  return x;
}

// A lane's 16 columns of a row: 8 l .. and 64 + 8 l ..
struct Cols {
  uint4 x[2];
};
__device__ __forceinline__ Cols load_cols(const uint16_t* row) { return {{load16(row), load16(row + 64)}}; }
__device__ __forceinline__ void store_cols(uint16_t* row, const F8 (&f)[2], int mode) {
  *reinterpret_cast<uint4*>(row) = pack8(f[0], mode);
  *reinterpret_cast<uint4*>(row + 64) = pack8(f[1], mode);
}

// Where a column's other half of the pair is: kWhole: column i + 64 or i - 64, the lane's other eight;
// kNext: the neighbour (interleaved); kApart: i + rot / 2 or i - rot / 2 with rot < 128, in the
// eight `slot` of lane `src`.
enum Form : int { kWhole = 0, kNext = 1, kApart = 2 };

// What a lane knows of the rotation: cos and +-sin of its columns, such that y = u c + (the
// other half's u) s, and where the other halves are. Eights that are not turned have c = 1, s = -0, and
// zeros for the other half: what stands there, or in the neighbouring column, has no part in them, and an
// infinity times 0 would be a NaN. What is added is then -0, which leaves a zero its sign.
struct Turn {
  F8 c[2], s[2];
  int src[2], slot[2];
  uint32_t pick[2];  // kNext: of a word's bytes, the halves swapped or zeros; kApart: a mask
  __device__ __forceinline__ bool turned(int e) const { return (pick[e] & 2u) != 0; }  // in either
};

// Eight e of a lane: its other halves' eight.
__device__ __forceinline__ int other_eight(int eight, int half) {
  const int pairs = half / 8;  // eights of the pairs' first columns
  return eight < pairs ? eight + pairs : eight < 2 * pairs ? eight - pairs : eight;
}

template <int kForm>
__device__ __forceinline__ void turn_lane(int lane, int half, Turn& t) {
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int other = other_eight((lane & 7) + 8 * e, half);
    t.src[e] = (lane & 24) | (other & 7);
    t.slot[e] = other >> 3;
    const bool turned = 8 * (lane & 7) + 64 * e < 2 * half;
    t.pick[e] = kForm == kNext ? (turned ? 0x1032u : 0x4444u) : turned ? 0xFFFFFFFFu : 0u;
  }
}

// kBack: turned back, s of the other sign.
template <int kForm, bool kBack>
__device__ __forceinline__ void turn_load(const Params& p, int lane, int pos, Turn& t) {
  const size_t row = static_cast<size_t>(pos) * p.half;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int c0 = 8 * (lane & 7) + 64 * e;
    if (kForm == kWhole && e == 1) {  // the same angles, the other sign
      t.c[1] = t.c[0];
#pragma unroll
      for (int j = 0; j < 4; ++j) t.s[1].p[j] = ptx::f2_sub(0, t.s[0].p[j]);
    } else if (c0 >= 2 * p.half) {
      t.c[e] = both(1.f);
      t.s[e] = both(-0.f);
    } else if constexpr (kForm == kNext) {
      const float4 c = __ldg(reinterpret_cast<const float4*>(p.cos + row + c0 / 2));
      const float4 s = __ldg(reinterpret_cast<const float4*>(p.sin + row + c0 / 2));
      const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        t.c[e].p[j] = ptx::f2_pack(cc[j], cc[j]);
        t.s[e].p[j] = kBack ? ptx::f2_pack(ss[j], -ss[j]) : ptx::f2_pack(-ss[j], ss[j]);
      }
    } else {
      const bool first = c0 < p.half;
      const size_t at = row + (first ? c0 : c0 - p.half);
      const float sign = first != kBack ? -1.f : 1.f;
      const uint64_t sign2 = ptx::f2_pack(sign, sign);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float4 c = __ldg(reinterpret_cast<const float4*>(p.cos + at) + u);
        const float4 s = __ldg(reinterpret_cast<const float4*>(p.sin + at) + u);
        t.c[e].p[2 * u] = ptx::f2_pack(c.x, c.y);
        t.c[e].p[2 * u + 1] = ptx::f2_pack(c.z, c.w);
        t.s[e].p[2 * u] = ptx::f2_mul(ptx::f2_pack(s.x, s.y), sign2);
        t.s[e].p[2 * u + 1] = ptx::f2_mul(ptx::f2_pack(s.z, s.w), sign2);
      }
    }
  }
}

__device__ __forceinline__ uint4 halves_swapped(const uint4& x, uint32_t pick) {
  return make_uint4(__byte_perm(x.x, 0, pick), __byte_perm(x.y, 0, pick), __byte_perm(x.z, 0, pick),
                    __byte_perm(x.w, 0, pick));
}

// The other halves of a lane's columns; zeros where there is none.
template <int kForm>
__device__ __forceinline__ Cols others(const Cols& x, const Turn& t) {
  if constexpr (kForm == kWhole) {
    return {{x.x[1], x.x[0]}};
  } else if constexpr (kForm == kNext) {
    return {{halves_swapped(x.x[0], t.pick[0]), halves_swapped(x.x[1], t.pick[1])}};
  } else {
    Cols o;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t a[4] = {x.x[0].x, x.x[0].y, x.x[0].z, x.x[0].w}, b[4] = {x.x[1].x, x.x[1].y, x.x[1].z, x.x[1].w};
      uint32_t r[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t u = __shfl_sync(0xFFFFFFFFu, a[j], t.src[e]), v = __shfl_sync(0xFFFFFFFFu, b[j], t.src[e]);
        r[j] = (t.slot[e] ? v : u) & t.pick[e];
      }
      o.x[e] = make_uint4(r[0], r[1], r[2], r[3]);
    }
    return o;
  }
}

// A warp's token of this lane, and its rows.
struct Token {
  int tok, pos;
  long long b, s;
  bool there;  // one of the call's
};
__device__ __forceinline__ Token token_of(const Params& p, long long first, int lane) {
  const long long x = first + (lane >> 3);
  Token t;
  t.there = x < p.tokens;
  t.tok = static_cast<int>(t.there ? x : p.tokens - 1);
  t.pos = __ldg(p.positions + t.tok);
  t.b = t.tok / p.S;
  t.s = t.tok - t.b * p.S;
  return t;
}
__device__ __forceinline__ uint16_t* row_of(const Rows& r, const Token& t, int h, int lane) {
  return r.p + t.b * r.batch + t.s * r.token + h * r.head + 8 * (lane & 7);
}

// Five CTAs an SM are 20 warps, 80 KiB on their way (16384 tokens of 20 heads: 25.5 us, 28 with four and 33
// with six, which spill); the other forms need more registers.
template <int kForm>
constexpr int kFwdCtas = kForm == kWhole ? 5 : 4;

// One warp: chunks of four tokens' heads. Bound by HBM: 512 bytes a row.
template <int kForm, bool kPaged>
__global__ void __launch_bounds__(kThreads, kFwdCtas<kForm>) attn_rope_fwd(const Params p) {
  const int lane = threadIdx.x & 31;
  const long long first = (static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * kTokens;
  if (first >= p.tokens) return;
  const Token tk = token_of(p, first, lane);
  int slot = 0;
  if constexpr (kPaged) slot = __ldg(p.slots + tk.tok);
  bool ok = tk.pos >= 0 && tk.pos < p.max_pos;
  if constexpr (kPaged) ok = ok && slot >= -1 && slot < p.n_slots;
  if (!ok && tk.there && (lane & 7) == 0) atomicOr(&g_attn_status, 8u);
  ok = ok && tk.there;  // nothing of a token out of range is written
  long long page_at = 0;  // elements; of the slot's head 0
  if constexpr (kPaged) {
    const int at = ok ? max(slot, 0) : 0, page = at / p.page_size, i = at - page * p.page_size;
    page_at = page * p.page_stride + static_cast<long long>(p.layout == 0 ? i : i * p.Hkv) * kD;
  }
  Turn t;  // with the weights: w c and (the other half's w) s
  turn_lane<kForm>(lane, p.half, t);
  int kind = -1;
  for (int c = blockIdx.y; c < p.chunks; c += p.parts) {
    const Chunk ch = chunk_of<kHeads>(p, c);
    const Rows& in = ch.kind == 0 ? p.q : ch.kind == 1 ? p.k : p.v;
    const uint16_t* src = row_of(in, tk, ch.h0, lane);
    if (!dbg_ok(ch.n >= 1)) return;
    Cols x[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
      if (i < ch.n) x[i] = load_cols(src + i * in.head);
    uint16_t* dst;
    long long step;  // elements between heads
    bool to = ok;
    if (kPaged && ch.kind != 0) {
      step = p.layout == 0 ? static_cast<long long>(p.page_size) * kD : kD;
      dst = (ch.kind == 1 ? p.k_pages : p.v_pages) + page_at + ch.h0 * step + 8 * (lane & 7);
      to = ok && slot >= 0;
      if (ch.kind == 2) {
#pragma unroll
        for (int i = 0; i < kHeads; ++i)
          if (i < ch.n && to) {
            *reinterpret_cast<uint4*>(dst + i * step) = x[i].x[0];
            *reinterpret_cast<uint4*>(dst + i * step + 64) = x[i].x[1];
          }
        continue;
      }
    } else {
      const Rows& out = ch.kind == 0 ? p.q_out : p.k_out;
      dst = row_of(out, tk, ch.h0, lane);
      step = out.head;
    }
    if (kind != ch.kind) {
      kind = ch.kind;
      turn_load<kForm, false>(p, lane, ok ? tk.pos : 0, t);
      const Cols w = load_cols((kind == 0 ? p.wq : p.wk) + 8 * (lane & 7)), w_other = others<kForm>(w, t);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        t.c[e] = mul(t.c[e], unpack8(w.x[e]));
        t.s[e] = mul(t.s[e], unpack8(w_other.x[e]));
      }
    }
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      if (i >= ch.n) break;
      const Cols o = others<kForm>(x[i], t);
      F8 a[2] = {unpack8(x[i].x[0]), unpack8(x[i].x[1])};
      const float r = rsqrtf(fmaf(row_sum(dot(a[0], a[0]) + dot(a[1], a[1])), 1.f / kD, p.eps));
      F8 y[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) a[e] = mul(a[e], both(r));
#pragma unroll
      for (int e = 0; e < 2; ++e)
        y[e] = fma(kForm == kWhole ? a[1 - e] : mul(unpack8(o.x[e]), both(t.turned(e) ? r : 0.f)), t.s[e],
                   mul(a[e], t.c[e]));
      if (to) store_cols(dst + i * step, y, p.mode);
    }
  }
}

// ---------------------------------------------------------------- backward
struct BwdParams {
  Params f;                // q, k, weights, table and positions as in the forward call
  Rows dq_out, dk_out;     // the gradients of what it gave
  Rows dq, dk;
  float* part;             // [block][2][128]
};

// The forms whose columns' angles differ between a lane's two eights need more registers.
template <int kForm>
constexpr int kBwdCtas = kForm == kWhole ? 4 : 3;
constexpr int kStages = 4;                        // heads of four tokens in a warp's ring
constexpr int kStageBytes = 4 * 32 * 16;          // x and dy, two eights each, as the lanes read them
constexpr int kBwdSmem = kWarps * kStages * kStageBytes;

// Persistent blocks: a warp takes its tokens' heads one after another, first the queries', then the
// keys', and sums their terms of the weight's gradient in registers; a block's sums go to the
// workspace, where attn_rope_join adds them in a fixed order. x and dy come by way of shared
// memory, three heads ahead (a lane copies what it reads itself, so nothing is waited for but its own
// copies): 96 KiB on their way an SM, where one head ahead in registers had 32 (16384 tokens of 32 heads:
// 85 us). Bound by HBM: 768 bytes a row (x, dy, dx).
template <int kForm>
__global__ void __launch_bounds__(kThreads, kBwdCtas<kForm>) attn_rope_bwd(const BwdParams bp) {
  extern __shared__ __align__(16) uint8_t ring_bytes[];
  __shared__ float sums[2][kWarps][kD];
  const Params& p = bp.f;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int w = static_cast<int>(blockIdx.x) * kWarps + warp;
  const int groups = static_cast<int>(gridDim.x) * kWarps / p.parts;  // of four tokens, at once
  const int part = w % p.parts, group = w / p.parts;
  const uint32_t ring = ptx::smem_u32(ring_bytes) + warp * kStages * kStageBytes + 16 * lane;
  Turn t;
  turn_lane<kForm>(lane, p.half, t);
#pragma unroll 1
  for (int kind = 0; kind < 2; ++kind) {
    // This warp's part of the queries' and then the keys' heads: of one kind where there are many parts.
    const int all = p.Hq + p.Hkv, before = kind == 0 ? 0 : p.Hq;
    const int h_first = max(static_cast<int>(static_cast<long long>(all) * part / p.parts) - before, 0);
    const Rows& in = kind == 0 ? p.q : p.k;
    const Rows& gin = kind == 0 ? bp.dq_out : bp.dk_out;
    const Rows& out = kind == 0 ? bp.dq : bp.dk;
    const int H = min(static_cast<int>(static_cast<long long>(all) * (part + 1) / p.parts) - before, kind == 0 ? p.Hq : p.Hkv);
    const Cols weight = load_cols((kind == 0 ? p.wq : p.wk) + 8 * (lane & 7));
    F8 dw[2] = {both(0.f), both(0.f)};
    for (long long first = static_cast<long long>(group) * kTokens;
         h_first < H && group < groups && first < p.tokens; first += static_cast<long long>(groups) * kTokens) {
      const Token tk = token_of(p, first, lane);
      const uint16_t* px = row_of(in, tk, h_first, lane);
      const uint16_t* py = row_of(gin, tk, h_first, lane);
      uint16_t* pd = row_of(out, tk, h_first, lane);
      int h_load = h_first, s_load = 0;
      auto load = [&]() {  // the next head, if there is one, into the next stage
        if (h_load < H) {
          const uint32_t to = ring + s_load * kStageBytes;
          ptx::cp_async16(to, px);
          ptx::cp_async16(to + 512, px + 64);
          ptx::cp_async16(to + 1024, py);
          ptx::cp_async16(to + 1536, py + 64);
          px += in.head;
          py += gin.head;
          ++h_load;
          s_load = s_load + 1 == kStages ? 0 : s_load + 1;
        }
        ptx::cp_async_commit();
      };
#pragma unroll
      for (int i = 0; i < kStages - 1; ++i) load();
      bool ok = tk.pos >= 0 && tk.pos < p.max_pos;
      // The gradients of a token out of range are not written, and it adds none to the weights'.
      if (!ok && tk.there && (lane & 7) == 0) atomicOr(&g_attn_status, 8u);
      ok = ok && tk.there;
      turn_load<kForm, true>(p, lane, ok ? tk.pos : 0, t);
      int stage = 0;
      for (int h = h_first; h < H; ++h) {
        __syncwarp();  // what the stage held has been read
        load();
        ptx::cp_async_wait<kStages - 1>();
        const uint32_t from = ring + stage * kStageBytes;
        stage = stage + 1 == kStages ? 0 : stage + 1;
        const Cols x = {{ptx::ld_shared_v4(from), ptx::ld_shared_v4(from + 512)}};
        const Cols y = {{ptx::ld_shared_v4(from + 1024), ptx::ld_shared_v4(from + 1536)}};
        const Cols o = others<kForm>(y, t);
        F8 a[2], g[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          a[e] = unpack8(x.x[e]);
          g[e] = fma(unpack8(y.x[e]), t.c[e], mul(unpack8(o.x[e]), t.s[e]));  // du: turned back
        }
        const float r = rsqrtf(fmaf(row_sum(dot(a[0], a[0]) + dot(a[1], a[1])), 1.f / kD, p.eps));
        const F8 r8 = both(r);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          a[e] = mul(a[e], r8);  // x r
          if (ok) dw[e] = fma(g[e], a[e], dw[e]);
          g[e] = mul(g[e], unpack8(weight.x[e]));  // dn
        }
        const F8 m = both(row_sum(dot(g[0], a[0]) + dot(g[1], a[1])) * (-1.f / kD));
#pragma unroll
        for (int e = 0; e < 2; ++e) g[e] = mul(fma(a[e], m, g[e]), r8);
        if (ok) store_cols(pd, g, p.mode);
        pd += out.head;
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float lo, hi;
        ptx::f2_unpack(dw[e].p[j], lo, hi);
#pragma unroll
        for (int d = 8; d < 32; d <<= 1) {  // the warp's four rows
          lo += __shfl_xor_sync(0xFFFFFFFFu, lo, d);
          hi += __shfl_xor_sync(0xFFFFFFFFu, hi, d);
        }
        if (lane < 8) *reinterpret_cast<float2*>(&sums[kind][warp][64 * e + 8 * lane + 2 * j]) = make_float2(lo, hi);
      }
  }
  __syncthreads();
#pragma unroll
  for (int kind = 0; kind < 2; ++kind) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) sum += sums[kind][i][threadIdx.x];
    bp.part[(static_cast<size_t>(blockIdx.x) * 2 + kind) * kD + threadIdx.x] = sum;
  }
}
static_assert(kThreads == kD, "a thread a column");

struct JoinParams {
  const float* part;
  float* dwq;
  float* dwk;
  int parts;
};

constexpr int kJoinCols = 8, kJoinThreads = 256, kJoinLanes = kJoinThreads / kJoinCols,
              kJoinBatch = 20;

// 8 columns a block, 32 threads a column, each over every 32nd part; then in order.
__global__ void __launch_bounds__(kJoinThreads) attn_rope_join(const JoinParams p) {
  __shared__ float sums[kJoinLanes][kJoinCols];
  ptx::grid_dependency_wait();
  const int col = blockIdx.x * kJoinCols + (threadIdx.x & (kJoinCols - 1)), at = threadIdx.x / kJoinCols;
  float s = 0.f;
  for (int base = at; base < p.parts; base += kJoinBatch * kJoinLanes) {  // a batch on its way at once
    float x[kJoinBatch];
#pragma unroll
    for (int j = 0; j < kJoinBatch; ++j) {
      const int i = base + j * kJoinLanes;
      x[j] = i < p.parts ? p.part[static_cast<size_t>(i) * 2 * kD + col] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < kJoinBatch; ++j) s += x[j];
  }
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
