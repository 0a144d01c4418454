// packed_range.h - the check of a packed batch's offsets, for host and device.
#pragma once

#if defined(__CUDACC__)
#define ATTN_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define ATTN_HOST_DEVICE inline
#endif

namespace attn {

// Length of a sequence whose tokens are [base, end) of `total`, -1 unless they lie inside and
// are at most `longest`. For any two ints: nothing is subtracted or added before it is known
// to fit (2^31 - 1 and -2^31 as neighbours would pass for a sequence of one token otherwise).
ATTN_HOST_DEVICE int packed_len(int base, int end, int longest, int total) {
  if (base < 0 || end < base || end > total) return -1;
  return end - base <= longest ? end - base : -1;
}

}  // namespace attn
