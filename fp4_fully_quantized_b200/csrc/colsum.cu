// colsum.cu -- the second half of the sums over rows (dweight, dbias): adds the
// row slices' partial sums, and the size helpers of these calls' buffers.
//
// out[c] = sum over the slices of partial[slice][c], slice order fixed.  The
// partials (at most 444 rows) were just written and are in L2; the kernel is
// bound by the latency of its loads, so 32 threads share a column's slices
// (at most 14 loads each, all in flight together) and join through shared
// memory; a CTA covers 32 columns, one 128-byte line of each slice.
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"

namespace fp4impl {
namespace {

constexpr int kColsPerCta = 32, kSlicesAtOnce = 32;

__global__ void __launch_bounds__(256)
colsum_kernel(const float* partial, int slices, int64_t cols, float* __restrict__ out) {
  __shared__ float4 acc[kSlicesAtOnce][8];
  wait_previous_launch();
  const int tx = threadIdx.x & 7, ty = threadIdx.x >> 3;
  const int64_t c = (int64_t)blockIdx.x * kColsPerCta + tx * 4;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < cols) {
#pragma unroll
    for (int i = 0; i < (kMaxSlices + kSlicesAtOnce - 1) / kSlicesAtOnce; ++i) {
      const int p = ty + i * kSlicesAtOnce;
      if (p < slices) {
        const float4 v = *reinterpret_cast<const float4*>(partial + p * cols + c);
        a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
      }
    }
  }
  acc[ty][tx] = a;
  allow_next_launch();
  __syncthreads();
  if (threadIdx.x < kColsPerCta) {
    const int64_t col = (int64_t)blockIdx.x * kColsPerCta + threadIdx.x;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kSlicesAtOnce; ++i) sum += reinterpret_cast<const float*>(acc[i])[threadIdx.x];
    if (col < cols) out[col] = sum;
  }
}

}  // namespace

cudaError_t launch_colsum(const float* partial, int64_t slices, int64_t cols, float* out,
                          cudaStream_t s) {
  return launch_overlapped(colsum_kernel, dim3((unsigned)((cols + kColsPerCta - 1) / kColsPerCta)), 256, 0, s,
                           partial, (int)slices, cols, out);
}

}  // namespace fp4impl

using namespace fp4impl;

extern "C" {

void fqt_ckpt8_sizes(int64_t rows, int64_t cols, size_t* codes_bytes, size_t* scales_bytes) {
  if (codes_bytes) *codes_bytes = (size_t)(rows * cols);
  if (scales_bytes) *scales_bytes = (size_t)(rows * (cols / 32));
}

size_t fqt_colsum_workspace_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0) return sizeof(DeviceStatus);
  return sizeof(DeviceStatus) + (size_t)(colsum_slices(rows) * cols) * sizeof(float);
}

}  // extern "C"
