// host_common.h - what the library's translation units with kernels share on the
// host: the tensor-map encoder, argument checks, the status words.
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>
#include <utility>

#include "attn_fwd.h"

namespace attn_host {

constexpr unsigned long long kTimeoutNs = 2000000000ull;  // 2 s per wait
constexpr int kMaxDevices = 64;

inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  std::call_once(once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult qres;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &qres) == cudaSuccess &&
        qres == cudaDriverEntryPointSuccess)
      encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  return encode;
}

// 4-D map over a (B, H, S, 128) bf16 tensor in the given layout, box of
// 64 columns x box_rows rows, 128-byte swizzle, zero fill outside the tensor.
inline bool make_map(CUtensorMap* map, const void* ptr, int layout, int64_t B, int64_t H, int64_t S,
              uint32_t box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  if (!encode) return false;
  const cuuint64_t row = 128 * 2;
  cuuint64_t dims[4], strides[3];
  cuuint32_t box[4];
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  if (layout == ATTN_LAYOUT_BHSD) {
    dims[0] = 128; dims[1] = S; dims[2] = H; dims[3] = B;
    strides[0] = row; strides[1] = S * row; strides[2] = H * S * row;
    box[0] = 64; box[1] = box_rows; box[2] = 1; box[3] = 1;
  } else {
    dims[0] = 128; dims[1] = H; dims[2] = S; dims[3] = B;
    strides[0] = row; strides[1] = H * row; strides[2] = S * H * row;
    box[0] = 64; box[1] = 1; box[2] = box_rows; box[3] = 1;
  }
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims,
                            strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

inline bool overlaps(const void* a, uint64_t na, const void* b, uint64_t nb) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + nb && b0 < a0 + na;
}

// Causal schedule: heads whose tiles are launched longest first together, in groups of
// one size whose streamed tensors (`bytes` a head) take at most 80 MiB of the 126 MiB
// L2. A group's last tiles are short, so it fills the SMs that the next one's first
// tiles leave; a small last group would start its longest tiles at the very end.
inline int heads_together(int64_t heads, int64_t bytes) {
  int64_t most = (int64_t(80) << 20) / (bytes > 0 ? bytes : 1);
  if (most < 1) most = 1;
  const int64_t groups = (heads + most - 1) / most;
  return static_cast<int>((heads + groups - 1) / groups);
}

// Adds a translation unit's device status word of the current device to *s and
// clears it.
template <typename Word>
bool take_status(Word& word, unsigned int* s) {
  unsigned int x = 0;
  if (cudaMemcpyFromSymbol(&x, word, sizeof(x)) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  if (x != 0) {
    const unsigned int zero = 0;
    cudaMemcpyToSymbol(word, &zero, sizeof(zero));
    *s |= x;
  }
  return true;
}
bool bwd_take_status(unsigned int* s);     // attn_bwd.cu
bool prefix_take_status(unsigned int* s);  // attn_prefix.cu

// Streaming multiprocessors of the current device (152, a GB300's, where there is
// none: size queries work without one).
inline int sms_here() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) {
    cudaGetLastError();
    return 152;
  }
  return sms;
}

// A launch that, when `dependent`, may start while the kernel before it on the
// stream drains: its kernel waits on the device for what it reads.
template <typename... Params, typename... Args>
bool launch(void (*fn)(Params...), int64_t grid, int threads, int smem, cudaStream_t stream, bool dependent,
            Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = dependent ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, fn, std::forward<Args>(args)...) == cudaSuccess) return true;
  cudaGetLastError();
  return false;
}

// attn_fwd.cu: the split form of the fused kernel without its merge. Each of
// n_splits parts of the keys leaves unnormalised rows [split][b*H + h][sq_pad][128]
// and (reference, row sum) [split][b*H + h][sq_pad][2], sq_pad = Sq rounded up to
// 256. A programmatic dependent of the launch before it (which writes q): it reads q
// after that has finished. Arguments are checked by the caller; returns a status code.
int split_parts(const void* q, const void* k, const void* v, int layout, int64_t B, int64_t H, int64_t Sq,
                int64_t Sk, float scale, int n_splits, float* part_o, float* part_rl, cudaStream_t stream);

}  // namespace attn_host
