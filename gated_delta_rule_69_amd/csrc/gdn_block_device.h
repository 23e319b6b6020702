// Device helpers of the operators of a block: lengths, sigmoids, sums of columns.
#pragma once

#include "gdn_layer_device.h"

namespace gdn {

__device__ __forceinline__ int64_t tokens_of(const int32_t* lens, int64_t b, int64_t T) {
  if (lens == nullptr) return T;
  const int64_t n = lens[b];
  return n < 0 ? 0 : n > T ? T : n;
}

// e^x. bf16 values take the one-instruction 2^x of x log2 e, off by |x| 2^-24; float32 expf.
template <typename E>
__device__ __forceinline__ float exp_of(float x) {
  return sizeof(E) == 2 ? __builtin_amdgcn_exp2f(1.44269504089f * x) : expf(x);
}

// The sigmoid s of z and 1 - s, both from e^-|z|, so that neither is a difference.
template <typename E>
__device__ __forceinline__ void sigmoids(float z, float* s, float* rest) {
  const float e = exp_of<E>(-fabsf(z));
  const float big = __builtin_amdgcn_rcpf(1.0f + e), small = e * big;
  *s = z < 0.0f ? small : big;
  *rest = z < 0.0f ? big : small;
}
// The sigmoid alone: the reciprocal of at least 1, 0 where e^-z overflows.
template <typename E>
__device__ __forceinline__ float sigmoid_of(float z) {
  return __builtin_amdgcn_rcpf(1.0f + exp_of<E>(-z));
}

// out[c] = sum over rows of partial[row][c] for c < cols, split over up to three arrays of n0,
// n1 and the remaining columns (NULL: dropped). The sums of out1 come times by1, and times by_also
// in `also` (NULL: times one). A block has 32 columns, 32 threads a column add up every 32nd row,
// then a tree of fixed order. Rows may be millions (one a sequence): a thread's sum is one of two floats,
// or 2^15 equal terms would be off by 10^-4 of it.
struct ColumnSum {
  const float* partial;
  int rows;
  int64_t cols, n0, n1;
  float *out0, *out1, *out2;
  float* also = nullptr;
  const float *by1 = nullptr, *by_also = nullptr;
};
static __global__ __launch_bounds__(1024) void column_sum_kernel(ColumnSum a) {
  const int64_t c = int64_t(blockIdx.x) * 32 + threadIdx.x % 32;
  float s = 0.0f, low = 0.0f;
  if (c < a.cols) {
#pragma unroll 4
    for (int r = threadIdx.x / 32; r < a.rows; r += 32) {
      const float x = a.partial[r * a.cols + c], sum = s + x, back = sum - s;
      low += (s - (sum - back)) + (x - back);
      s = sum;
    }
    if (low == low) s += low;   // not behind an infinity
  }
  __shared__ float part[1024];
  part[threadIdx.x] = s;
#pragma unroll
  for (int step = 512; step >= 32; step /= 2) {
    __syncthreads();
    if (threadIdx.x < step) part[threadIdx.x] += part[threadIdx.x + step];
  }
  if (threadIdx.x < 32 && c < a.cols) {
    const float sum = part[threadIdx.x];
    const int64_t c1 = c - a.n0;
    if (c1 < 0) {
      if (a.out0 != nullptr) a.out0[c] = sum;
    } else if (c1 < a.n1) {
      if (a.out1 != nullptr) a.out1[c1] = a.by1 != nullptr ? a.by1[c1] * sum : sum;
      if (a.also != nullptr) a.also[c1] = a.by_also != nullptr ? a.by_also[c1] * sum : sum;
    } else if (a.out2 != nullptr) {
      a.out2[c1 - a.n1] = sum;
    }
  }
}
inline int launch_column_sum(const ColumnSum& a, hipStream_t s) {
  column_sum_kernel<<<unsigned((a.cols + 31) / 32), 1024, 0, s>>>(a);
  return int(hipGetLastError());
}

}  // namespace gdn
