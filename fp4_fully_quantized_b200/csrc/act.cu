// act.cu -- activations and gated activations with 8-bit checkpoints of their
// input: forward (with encoding), recomputation from a checkpoint, backward
// (with the bias gradient).
//
// Elementwise and bound by HBM: a thread owns eight columns (of both halves
// when gated) and walks down its rows, so the bias gradient sums in registers
// and needs no atomics.  A CTA has `lanes` threads side by side (8, 16 or 32: 64
// to 256 columns) and 256 / lanes rows at a time; a grid column covers the
// width, a grid row a slice of the rows.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "act_device.cuh"
#include "fp4_device.cuh"
#include "internal.h"

namespace fp4impl {
using namespace fp4dev;
namespace {

constexpr int kThreads = 256;

struct ActParams {
  const __nv_bfloat16* z; int64_t ldz;
  const uint8_t* codes; const uint8_t* scales;       // z from a checkpoint
  const __nv_bfloat16* dy; int64_t lddy;
  __nv_bfloat16* out; int64_t ldo;                   // y or dz
  uint8_t* codes_out; uint8_t* scales_out;
  int64_t rows, cols, zcols;
  float* partial; float* amax; uint32_t* status;
  int lanes;
};

// Eight values of z at (row, c).
template <bool CKPT>
__device__ __forceinline__ void load_z(const ActParams& p, int64_t row, int64_t c, float* v) {
  if constexpr (CKPT) {
    const int64_t at = row * p.zcols + c;
    const uint2 q = *reinterpret_cast<const uint2*>(p.codes + at);
    const float e = ckpt_scale(p.scales[at >> 5]);
    e4m3x4_to_f32(q.x, v);
    e4m3x4_to_f32(q.y, v + 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= e;
  } else {
    load8(p.z, row * p.ldz + c, false, v);
  }
}

__device__ __forceinline__ void max_to(float* dst, uint32_t amax) {
  if (dst == nullptr) return;
  amax = __reduce_max_sync(0xFFFFFFFFu, amax);
  if ((threadIdx.x & 31) == 0) atomicMax(reinterpret_cast<unsigned int*>(dst), amax);
}

template <int ACT, bool GATED, bool CKPT>
__global__ void __launch_bounds__(kThreads) act_fwd_kernel(const ActParams p) {
  const int lane = threadIdx.x % p.lanes, rows_at_once = kThreads / p.lanes;
  const int64_t c = ((int64_t)blockIdx.x * p.lanes + lane) * 8;
  const bool in = c < p.cols;
  uint32_t amax = 0;
  bool finite = true;
  for (int64_t base = (int64_t)blockIdx.y * rows_at_once; base < p.rows;
       base += (int64_t)gridDim.y * rows_at_once) {
    const int64_t row = base + threadIdx.x / p.lanes;
    const bool ok = in && row < p.rows;
    float g[8], u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = u[i] = 0.0f;
    if (ok) {
      load_z<CKPT>(p, row, c, g);
      if constexpr (GATED) load_z<CKPT>(p, row, p.cols + c, u);
    }
    if (p.out != nullptr && ok) {
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        y[i] = g[i];
        y[i + 1] = g[i + 1];
        act_value2<ACT>(y[i], y[i + 1]);
        if constexpr (GATED) { y[i] *= u[i]; y[i + 1] *= u[i + 1]; }
      }
      const uint4 packed = pack_bf16x8(y);
      *reinterpret_cast<uint4*>(p.out + row * p.ldo + c) = packed;
      amax = max(amax, amax_bits_bf16x8(packed));
    }
    if constexpr (!CKPT) {
      if (p.codes_out != nullptr) {
        const int64_t at = row * p.zcols + c;
        finite &= encode8(g, p.codes_out + at, p.scales_out + (at >> 5), ok);
        if constexpr (GATED)
          finite &= encode8(u, p.codes_out + at + p.cols, p.scales_out + ((at + p.cols) >> 5), ok);
      }
    }
  }
  max_to(p.amax, amax);
  if (!finite) set_status(p.status, FP4_ERR_NONFINITE, 7);
}

template <int ACT, bool GATED, bool CKPT>
__global__ void __launch_bounds__(kThreads) act_bwd_kernel(const ActParams p) {
  __shared__ float sums[kThreads * 8];
  const int lane = threadIdx.x % p.lanes, rows_at_once = kThreads / p.lanes;
  const int64_t c = ((int64_t)blockIdx.x * p.lanes + lane) * 8;
  const bool in = c < p.cols;
  uint32_t amax = 0;
  float db[GATED ? 16 : 8];
#pragma unroll
  for (int i = 0; i < (GATED ? 16 : 8); ++i) db[i] = 0.0f;
  for (int64_t row = (int64_t)blockIdx.y * rows_at_once + threadIdx.x / p.lanes; in && row < p.rows;
       row += (int64_t)gridDim.y * rows_at_once) {
    float g[8], dy[8], d[8];
    load_z<CKPT>(p, row, c, g);
    load8(p.dy, row * p.lddy + c, false, dy);
    if constexpr (GATED) {
      float u[8], du[8];
      load_z<CKPT>(p, row, p.cols + c, u);
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        float f[2], df[2];
        act_both2<ACT>(g[i], g[i + 1], f[0], f[1], df[0], df[1]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          d[i + j] = dy[i + j] * u[i + j] * df[j];
          du[i + j] = dy[i + j] * f[j];
          db[8 + i + j] += du[i + j];
        }
      }
      const uint4 packed = pack_bf16x8(du);
      *reinterpret_cast<uint4*>(p.out + row * p.ldo + p.cols + c) = packed;
      amax = max(amax, amax_bits_bf16x8(packed));
    } else {
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        float f[2], df[2];
        act_both2<ACT>(g[i], g[i + 1], f[0], f[1], df[0], df[1]);
        d[i] = dy[i] * df[0];
        d[i + 1] = dy[i + 1] * df[1];
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) db[i] += d[i];
    const uint4 packed = pack_bf16x8(d);
    *reinterpret_cast<uint4*>(p.out + row * p.ldo + c) = packed;
    amax = max(amax, amax_bits_bf16x8(packed));
  }
  max_to(p.amax, amax);
  if (p.partial == nullptr) return;
  // join the CTA's rows, half by half
  const int width = p.lanes * 8;
#pragma unroll
  for (int h = 0; h < (GATED ? 2 : 1); ++h) {
    __syncthreads();
    store8(sums, threadIdx.x * 8, true, db + 8 * h);
    __syncthreads();
    const int64_t col = (int64_t)blockIdx.x * width + threadIdx.x;
    if (threadIdx.x < width && col < p.cols) {
      float a = 0.0f;
      for (int k = 0; k < rows_at_once; ++k) a += sums[k * width + threadIdx.x];
      p.partial[(int64_t)blockIdx.y * p.zcols + h * p.cols + col] = a;
    }
  }
}

// Lanes side by side: as few of 8, 16, 32 as cover the width in one CTA.
int lanes_for(int64_t cols) { return cols <= 64 ? 8 : cols <= 128 ? 16 : 32; }

// Row slices of the grid: enough CTAs for every SM to hold eight, at most one
// per group of rows, at most kMaxSlices (the partial sums' bound).  The size of
// the part is a constant here, so that sums do not depend on the device.
dim3 act_grid(int64_t rows, int64_t cols, int lanes) {
  const int64_t gx = (cols + lanes * 8 - 1) / (lanes * 8);
  const int64_t most = (rows + kThreads / lanes - 1) / (kThreads / lanes);
  int64_t gy = (148 * 8 + gx - 1) / gx;
  gy = gy < most ? gy : most;
  gy = gy < kMaxSlices ? gy : kMaxSlices;
  return dim3((unsigned)gx, (unsigned)gy);
}

template <bool FWD, int ACT, bool GATED, bool CKPT>
void launch_one(const ActParams& p, dim3 grid, cudaStream_t s) {
  if constexpr (FWD) act_fwd_kernel<ACT, GATED, CKPT><<<grid, kThreads, 0, s>>>(p);
  else act_bwd_kernel<ACT, GATED, CKPT><<<grid, kThreads, 0, s>>>(p);
}

template <bool FWD, int ACT>
void launch_act(const ActParams& p, bool gated, bool ckpt, dim3 grid, cudaStream_t s) {
  if (gated && ckpt) launch_one<FWD, ACT, true, true>(p, grid, s);
  else if (gated) launch_one<FWD, ACT, true, false>(p, grid, s);
  else if (ckpt) launch_one<FWD, ACT, false, true>(p, grid, s);
  else launch_one<FWD, ACT, false, false>(p, grid, s);
}

template <bool FWD>
cudaError_t launch(ActParams& p, int act, bool gated, unsigned& slices, cudaStream_t s) {
  p.lanes = lanes_for(p.cols);
  const dim3 grid = act_grid(p.rows, p.cols, p.lanes);
  slices = grid.y;
  switch (act) {
    case FQT_ACT_RELU: launch_act<FWD, FQT_ACT_RELU>(p, gated, p.codes != nullptr, grid, s); break;
    case FQT_ACT_GELU: launch_act<FWD, FQT_ACT_GELU>(p, gated, p.codes != nullptr, grid, s); break;
    case FQT_ACT_GELU_TANH: launch_act<FWD, FQT_ACT_GELU_TANH>(p, gated, p.codes != nullptr, grid, s); break;
    case FQT_ACT_SILU: launch_act<FWD, FQT_ACT_SILU>(p, gated, p.codes != nullptr, grid, s); break;
    default: launch_act<FWD, FQT_ACT_NONE>(p, gated, p.codes != nullptr, grid, s); break;
  }
  count_launches(1);
  return cudaGetLastError();
}

// The checks that both directions make of their shape and of z.
fp4_status check_act(const void* z, int64_t ldz, const fqt_ckpt8* z8, int32_t act, int64_t rows,
                     int64_t cols, int64_t zcols, const void* ws, size_t ws_bytes) {
  if (!known_act(act)) return FP4_ERR_FORMAT;
  if (rows < 0 || cols <= 0 || cols % 8 || zcols > ((int64_t)1 << 30)) return FP4_ERR_SHAPE;
  if (ws != nullptr && ws_bytes < sizeof(DeviceStatus)) return FP4_ERR_WORKSPACE;
  if (z8 != nullptr) {
    if (z != nullptr) return FP4_ERR_FORMAT;
    if (cols % 32) return FP4_ERR_SHAPE;      // a block lies in one half
    return check_ckpt8(z8, rows, zcols);
  }
  return rows > 0 ? check_matrix(z, zcols, ldz) : FP4_OK;
}

}  // namespace
}  // namespace fp4impl

using namespace fp4impl;

extern "C" {

fp4_status fqt_act_fwd(const void* z, int64_t ldz, const fqt_ckpt8* z8_in, int32_t act, int32_t gated,
                       int64_t rows, int64_t cols, void* y, int64_t ldy, const fqt_ckpt8* z8_out,
                       float* y_amax, void* ws, size_t ws_bytes, void* stream) {
  const int64_t zcols = gated ? 2 * cols : cols;
  fp4_status st = check_act(z, ldz, z8_in, act, rows, cols, zcols, ws, ws_bytes);
  if (st != FP4_OK) return st;
  if (rows > 0 && y == nullptr && (z8_out == nullptr || y_amax != nullptr)) return FP4_ERR_NULL;
  if (z8_in != nullptr && z8_out != nullptr) return FP4_ERR_FORMAT;
  if (y != nullptr && rows > 0 && (st = check_matrix(y, cols, ldy)) != FP4_OK) return st;
  if (z8_out != nullptr) {
    if (cols % 32) return FP4_ERR_SHAPE;
    if ((st = check_ckpt8(z8_out, rows, zcols)) != FP4_OK) return st;
  }
  if (!ptr_aligned(y_amax, 4)) return FP4_ERR_ALIGN;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (y_amax != nullptr && cudaMemsetAsync(y_amax, 0, sizeof(float), s) != cudaSuccess) return FP4_ERR_CUDA;
  if (rows == 0) return FP4_OK;
  ActParams p{};
  p.z = static_cast<const __nv_bfloat16*>(z); p.ldz = ldz;
  if (z8_in != nullptr) { p.codes = z8_in->codes; p.scales = z8_in->scales; }
  p.out = static_cast<__nv_bfloat16*>(y); p.ldo = ldy;
  if (z8_out != nullptr) { p.codes_out = z8_out->codes; p.scales_out = z8_out->scales; }
  p.rows = rows; p.cols = cols; p.zcols = zcols;
  p.amax = y_amax; p.status = static_cast<uint32_t*>(ws);
  unsigned slices = 0;
  return launch<true>(p, act, gated != 0, slices, s) == cudaSuccess ? FP4_OK : FP4_ERR_CUDA;
}

fp4_status fqt_act_bwd(const void* dy, int64_t lddy, const void* z, int64_t ldz, const fqt_ckpt8* z8,
                       int32_t act, int32_t gated, int64_t rows, int64_t cols, void* dz, int64_t lddz,
                       float* dbias, float* dz_amax, void* ws, size_t ws_bytes, void* stream) {
  const int64_t zcols = gated ? 2 * cols : cols;
  fp4_status st = check_act(z, ldz, z8, act, rows, cols, zcols, ws, ws_bytes);
  if (st != FP4_OK) return st;
  if (rows > 0 && ((st = check_matrix(dy, cols, lddy)) != FP4_OK ||
                   (st = check_matrix(dz, zcols, lddz)) != FP4_OK))
    return st;
  if (!ptr_aligned(dbias, 4) || !ptr_aligned(dz_amax, 4) || !ptr_aligned(ws, 16)) return FP4_ERR_ALIGN;
  if (dbias != nullptr && (ws == nullptr || ws_bytes < fqt_colsum_workspace_bytes(rows, zcols)))
    return FP4_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dz_amax != nullptr && cudaMemsetAsync(dz_amax, 0, sizeof(float), s) != cudaSuccess) return FP4_ERR_CUDA;
  if (rows == 0) {
    if (dbias != nullptr && cudaMemsetAsync(dbias, 0, zcols * sizeof(float), s) != cudaSuccess)
      return FP4_ERR_CUDA;
    return FP4_OK;
  }
  ActParams p{};
  p.z = static_cast<const __nv_bfloat16*>(z); p.ldz = ldz;
  if (z8 != nullptr) { p.codes = z8->codes; p.scales = z8->scales; }
  p.dy = static_cast<const __nv_bfloat16*>(dy); p.lddy = lddy;
  p.out = static_cast<__nv_bfloat16*>(dz); p.ldo = lddz;
  p.rows = rows; p.cols = cols; p.zcols = zcols;
  p.partial = dbias != nullptr ? colsum_partials(ws) : nullptr;
  p.amax = dz_amax; p.status = static_cast<uint32_t*>(ws);
  unsigned slices = 0;
  cudaError_t e = launch<false>(p, act, gated != 0, slices, s);
  if (e == cudaSuccess && dbias != nullptr) e = launch_colsum(p.partial, slices, zcols, dbias, s);
  return e == cudaSuccess ? FP4_OK : FP4_ERR_CUDA;
}

}  // extern "C"
