// rmsnorm.cu -- RMS norm with the residual's addition and an 8-bit output, and
// its backward.
//
// Forward, per row: s = x + residual, rstd = (mean s^2 + eps)^(-1/2),
// y = s * rstd * weight; the row stays in registers between the statistics and
// the outputs, so each input is read once and each output written once.
// Backward, per row, with g = dy * weight: dx = rstd (g - xhat mean(g xhat)) +
// dres; dweight sums dy * xhat over the rows in registers, one partial row per
// CTA, joined by colsum.cu.
//
// A row belongs to a group of threads, each of which holds V chunks of eight
// consecutive columns, the group's threads side by side: 8, 16 or 32 lanes of
// a warp for rows of up to 1024 columns (several rows per CTA, no barrier), a
// CTA for longer ones.  Both kernels are bound by HBM.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>

#include "act_device.cuh"
#include "fp4_device.cuh"
#include "internal.h"

namespace fp4impl {
using namespace fp4dev;
namespace {

constexpr int kMaxCols = 32768;      // 1024 threads x 4 chunks of 8
constexpr int kGroupThreads = 256;   // CTA of the lane-group kernels

struct FwdParams {
  const __nv_bfloat16* x; int64_t ldx;
  const void* res; int64_t ldr;
  void* res_out; int64_t ldo;
  const void* w; bool w_f32;
  float eps; int64_t rows; int cols;
  __nv_bfloat16* y; int64_t ldy;
  uint8_t* codes; uint8_t* scales; bool q_xhat;
  float* rstd; float* y_amax; uint32_t* status;
};

struct BwdParams {
  const __nv_bfloat16* dy; int64_t lddy;
  const void* s; int64_t lds;
  const uint8_t* codes; const uint8_t* scales;
  const float* rstd; const void* w; bool w_f32;
  const void* dres; int64_t lddres;
  void* dx; int64_t lddx; bool grad_f32;
  int64_t rows; int cols;
  float* partial;
};

// Sum over the group: G lanes of the warp, or (G == 0) the CTA through `slot`
// (one float per warp; the caller alternates between two slots, so one barrier
// per sum is enough).  Every thread gets the same value, added in a fixed order.
template <int G>
__device__ __forceinline__ float group_sum(float v, float* slot) {
  constexpr int W = G == 0 ? 32 : G;
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if constexpr (G == 0) {
    if ((threadIdx.x & 31) == 0) slot[threadIdx.x >> 5] = v;
    __syncthreads();
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    v = lane < warps ? slot[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  }
  return v;
}

// RES: 0 no residual, 1 BF16, 2 FP32.
template <int G, int V, int RES>
__global__ void __launch_bounds__(G ? kGroupThreads : 1024)
rmsnorm_fwd_kernel(const FwdParams p) {
  __shared__ float slots[2][32];
  const int T = G ? G : blockDim.x;
  const int gl = G ? threadIdx.x % T : threadIdx.x;
  const int per_cta = G ? kGroupThreads / T : 1;
  const int64_t S = p.cols >> 5;
  uint32_t amax = 0;
  bool finite = true;
  int flip = 0;
  for (int64_t base = (int64_t)blockIdx.x * per_cta; base < p.rows;
       base += (int64_t)gridDim.x * per_cta, flip ^= 1) {
    const int64_t row = base + (G ? threadIdx.x / T : 0);
    float s[V][8];
    float ss = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (gl + v * T) * 8;
      const bool ok = row < p.rows && c < p.cols;
#pragma unroll
      for (int i = 0; i < 8; ++i) s[v][i] = 0.0f;
      if (ok) {
        load8(p.x, row * p.ldx + c, false, s[v]);
        if constexpr (RES != 0) {
          float r[8];
          load8(p.res, row * p.ldr + c, RES == 2, r);
#pragma unroll
          for (int i = 0; i < 8; ++i) s[v][i] += r[i];
          store8(p.res_out, row * p.ldo + c, RES == 2, s[v]);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += s[v][i] * s[v][i];
    }
    ss = group_sum<G>(ss, slots[flip]);
    const float rstd = rsqrtf(ss / (float)p.cols + p.eps);
    if (p.rstd != nullptr && gl == 0 && row < p.rows) p.rstd[row] = rstd;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (gl + v * T) * 8;
      const bool ok = row < p.rows && c < p.cols;
      float w[8], y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = 0.0f;
      if (ok) load8(p.w, c, p.w_f32, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) { s[v][i] *= rstd; y[i] = s[v][i] * w[i]; }
      if (p.y != nullptr && ok) {
        const uint4 packed = pack_bf16x8(y);
        *reinterpret_cast<uint4*>(p.y + row * p.ldy + c) = packed;
        amax = max(amax, amax_bits_bf16x8(packed));
      } else if (ok) {
        amax = max(amax, amax_bits_bf16x8(pack_bf16x8(y)));
      }
      if (p.codes != nullptr)
        finite &= encode8(p.q_xhat ? s[v] : y, p.codes + row * p.cols + c, p.scales + row * S + (c >> 5), ok);
    }
  }
  if (p.y_amax != nullptr) {
    amax = __reduce_max_sync(0xFFFFFFFFu, amax);
    if ((threadIdx.x & 31) == 0) atomicMax(reinterpret_cast<unsigned int*>(p.y_amax), amax);
  }
  if (!finite) set_status(p.status, FP4_ERR_NONFINITE, 6);
}

// SRC: 0 the stored sum in BF16, 1 in FP32, 2 the 8-bit checkpoint of xhat.
template <int G, int V, int SRC>
__global__ void __launch_bounds__(G ? kGroupThreads : 1024)
rmsnorm_bwd_kernel(const BwdParams p) {
  __shared__ float slots[2][32];
  extern __shared__ float sums[];        // lane groups: [groups][cols]
  const int T = G ? G : blockDim.x;
  const int gl = G ? threadIdx.x % T : threadIdx.x;
  const int per_cta = G ? kGroupThreads / T : 1;
  const int64_t S = p.cols >> 5;
  const float inv_cols = 1.0f / (float)p.cols;
  float dw[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[v][i] = 0.0f;
  int flip = 0;
  for (int64_t base = (int64_t)blockIdx.x * per_cta; base < p.rows;
       base += (int64_t)gridDim.x * per_cta, flip ^= 1) {
    const int64_t row = base + (G ? threadIdx.x / T : 0);
    const float rstd = row < p.rows ? p.rstd[row] : 0.0f;
    float xh[V][8], g[V][8];
    float dot = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (gl + v * T) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) xh[v][i] = g[v][i] = 0.0f;
      if (row < p.rows && c < p.cols) {
        if constexpr (SRC == 2) {
          const uint2 q = *reinterpret_cast<const uint2*>(p.codes + row * p.cols + c);
          const float e = ckpt_scale(p.scales[row * S + (c >> 5)]);
          e4m3x4_to_f32(q.x, xh[v]);
          e4m3x4_to_f32(q.y, xh[v] + 4);
#pragma unroll
          for (int i = 0; i < 8; ++i) xh[v][i] *= e;
        } else {
          load8(p.s, row * p.lds + c, SRC == 1, xh[v]);
#pragma unroll
          for (int i = 0; i < 8; ++i) xh[v][i] *= rstd;
        }
        float dy[8], w[8];
        load8(p.dy, row * p.lddy + c, false, dy);
        load8(p.w, c, p.w_f32, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          g[v][i] = dy[i] * w[i];
          dw[v][i] += dy[i] * xh[v][i];
          dot += g[v][i] * xh[v][i];
        }
      }
    }
    const float m = group_sum<G>(dot, slots[flip]) * inv_cols;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (gl + v * T) * 8;
      if (row < p.rows && c < p.cols) {
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = rstd * (g[v][i] - xh[v][i] * m);
        if (p.dres != nullptr) {
          float r[8];
          load8(p.dres, row * p.lddres + c, p.grad_f32, r);
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] += r[i];
        }
        store8(p.dx, row * p.lddx + c, p.grad_f32, o);
      }
    }
  }
  if (p.partial == nullptr) return;
  float* out = p.partial + (int64_t)blockIdx.x * p.cols;
  if constexpr (G == 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (gl + v * T) * 8;
      if (c < p.cols) store8(out, c, true, dw[v]);
    }
  } else {
    const int grp = threadIdx.x / T;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (gl + v * T) * 8;
      if (c < p.cols) store8(sums + grp * p.cols, c, true, dw[v]);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.cols; c += kGroupThreads) {
      float a = 0.0f;
      for (int k = 0; k < per_cta; ++k) a += sums[k * p.cols + c];
      out[c] = a;
    }
  }
}

// Lanes per row (0: the CTA), chunks per thread and threads of the CTA for a row
// of `cols`: as few lanes as hold the row in one chunk each, then more chunks.
struct RowPlan { int lanes, chunks, threads; };
RowPlan row_plan(int64_t cols) {
  const int64_t n = cols / 8;
  if (n <= 8) return {8, 1, kGroupThreads};
  if (n <= 16) return {16, 1, kGroupThreads};
  if (n <= 32) return {32, 1, kGroupThreads};
  if (n <= 64) return {32, 2, kGroupThreads};
  if (n <= 128) return {32, 4, kGroupThreads};
  const int chunks = n <= 512 ? 1 : n <= 1024 ? 2 : 4;
  const int64_t t = (n + chunks - 1) / chunks;
  return {0, chunks, (int)((t + 31) / 32 * 32)};
}

template <int RES>
cudaError_t launch_fwd(const FwdParams& p, cudaStream_t s) {
  const RowPlan r = row_plan(p.cols);
  const int per_cta = r.lanes ? kGroupThreads / r.lanes : 1;
  const int64_t want = (p.rows + per_cta - 1) / per_cta;
  const int64_t slots = (int64_t)sm_count() * (2048 / r.threads);
  const int grid = (int)(want < slots ? want : slots);
#define FP4_NORM_FWD(G, V) rmsnorm_fwd_kernel<G, V, RES><<<grid, r.threads, 0, s>>>(p)
  if (r.lanes == 8) FP4_NORM_FWD(8, 1);
  else if (r.lanes == 16) FP4_NORM_FWD(16, 1);
  else if (r.lanes == 32 && r.chunks == 1) FP4_NORM_FWD(32, 1);
  else if (r.lanes == 32 && r.chunks == 2) FP4_NORM_FWD(32, 2);
  else if (r.lanes == 32) FP4_NORM_FWD(32, 4);
  else if (r.chunks == 1) FP4_NORM_FWD(0, 1);
  else if (r.chunks == 2) FP4_NORM_FWD(0, 2);
  else FP4_NORM_FWD(0, 4);
#undef FP4_NORM_FWD
  count_launches(1);
  return cudaGetLastError();
}

template <int SRC>
cudaError_t launch_bwd(const BwdParams& p, int& grid, cudaStream_t s) {
  const RowPlan r = row_plan(p.cols);
  const int per_cta = r.lanes ? kGroupThreads / r.lanes : 1;
  const int64_t want = (p.rows + per_cta - 1) / per_cta;
  grid = (int)(want < kMaxSlices ? want : kMaxSlices);
  const size_t smem = r.lanes && p.partial ? (size_t)per_cta * p.cols * sizeof(float) : 0;   // <= 32 KB
#define FP4_NORM_BWD(G, V) rmsnorm_bwd_kernel<G, V, SRC><<<grid, r.threads, smem, s>>>(p)
  if (r.lanes == 8) FP4_NORM_BWD(8, 1);
  else if (r.lanes == 16) FP4_NORM_BWD(16, 1);
  else if (r.lanes == 32 && r.chunks == 1) FP4_NORM_BWD(32, 1);
  else if (r.lanes == 32 && r.chunks == 2) FP4_NORM_BWD(32, 2);
  else if (r.lanes == 32) FP4_NORM_BWD(32, 4);
  else if (r.chunks == 1) FP4_NORM_BWD(0, 1);
  else if (r.chunks == 2) FP4_NORM_BWD(0, 2);
  else FP4_NORM_BWD(0, 4);
#undef FP4_NORM_BWD
  count_launches(1);
  return cudaGetLastError();
}

fp4_status check_norm(int64_t rows, int64_t cols, const void* weight, int32_t w_dtype, const void* ws,
                      size_t ws_bytes) {
  if (weight == nullptr) return FP4_ERR_NULL;
  if (!known_dtype(w_dtype)) return FP4_ERR_FORMAT;
  if (rows < 0 || cols <= 0 || cols > kMaxCols || cols % 8) return FP4_ERR_SHAPE;
  if (!ptr_aligned(weight, 16)) return FP4_ERR_ALIGN;
  if (ws != nullptr && ws_bytes < sizeof(DeviceStatus)) return FP4_ERR_WORKSPACE;
  return FP4_OK;
}

}  // namespace
}  // namespace fp4impl

using namespace fp4impl;

extern "C" {

fp4_status fqt_rmsnorm_fwd(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                           void* res_out, int64_t ldo, int32_t res_dtype, const void* weight,
                           int32_t w_dtype, float eps, int64_t rows, int64_t cols, void* y,
                           int64_t ldy, const fqt_ckpt8* q8, int32_t q8_of, float* rstd,
                           float* y_amax, void* ws, size_t ws_bytes, void* stream) {
  fp4_status st = check_norm(rows, cols, weight, w_dtype, ws, ws_bytes);
  if (st != FP4_OK) return st;
  if (y == nullptr && q8 == nullptr && rows > 0) return FP4_ERR_NULL;
  if ((residual == nullptr) != (res_out == nullptr) && rows > 0) return FP4_ERR_NULL;
  if (!(eps > 0.0f) || !(eps <= FLT_MAX)) return FP4_ERR_FORMAT;
  if (residual != nullptr && !known_dtype(res_dtype)) return FP4_ERR_FORMAT;
  if (q8 != nullptr && q8_of != FQT_RMS_Y && q8_of != FQT_RMS_XHAT) return FP4_ERR_FORMAT;
  if (rows > 0) {
    if ((st = check_matrix(x, cols, ldx)) != FP4_OK) return st;
    if (residual != nullptr && ((st = check_matrix(residual, cols, ldr)) != FP4_OK ||
                                (st = check_matrix(res_out, cols, ldo)) != FP4_OK))
      return st;
    if (y != nullptr && (st = check_matrix(y, cols, ldy)) != FP4_OK) return st;
  }
  if (q8 != nullptr && (st = check_ckpt8(q8, rows, cols)) != FP4_OK) return st;
  if (!ptr_aligned(rstd, 4) || !ptr_aligned(y_amax, 4)) return FP4_ERR_ALIGN;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (y_amax != nullptr && cudaMemsetAsync(y_amax, 0, sizeof(float), s) != cudaSuccess) return FP4_ERR_CUDA;
  if (rows == 0) return FP4_OK;
  FwdParams p{};
  p.x = static_cast<const __nv_bfloat16*>(x); p.ldx = ldx;
  p.res = residual; p.ldr = ldr; p.res_out = res_out; p.ldo = ldo;
  p.w = weight; p.w_f32 = w_dtype == FP4_OUT_F32;
  p.eps = eps; p.rows = rows; p.cols = (int)cols;
  p.y = static_cast<__nv_bfloat16*>(y); p.ldy = ldy;
  if (q8 != nullptr) { p.codes = q8->codes; p.scales = q8->scales; p.q_xhat = q8_of == FQT_RMS_XHAT; }
  p.rstd = rstd; p.y_amax = y_amax; p.status = static_cast<uint32_t*>(ws);
  const cudaError_t e = residual == nullptr       ? launch_fwd<0>(p, s)
                        : res_dtype == FP4_OUT_F32 ? launch_fwd<2>(p, s)
                                                   : launch_fwd<1>(p, s);
  return e == cudaSuccess ? FP4_OK : FP4_ERR_CUDA;
}

fp4_status fqt_rmsnorm_bwd(const void* dy, int64_t lddy, const void* sum, int64_t lds, int32_t s_dtype,
                           const fqt_ckpt8* xhat8, const float* rstd, const void* weight,
                           int32_t w_dtype, const void* dres, int64_t lddres, void* dx, int64_t lddx,
                           int32_t grad_dtype, int64_t rows, int64_t cols, float* dweight, void* ws,
                           size_t ws_bytes, void* stream) {
  fp4_status st = check_norm(rows, cols, weight, w_dtype, ws, ws_bytes);
  if (st != FP4_OK) return st;
  if (!known_dtype(grad_dtype)) return FP4_ERR_FORMAT;
  if (xhat8 != nullptr) {
    if (sum != nullptr) return FP4_ERR_FORMAT;
    if ((st = check_ckpt8(xhat8, rows, cols)) != FP4_OK) return st;
  } else if (!known_dtype(s_dtype)) {
    return FP4_ERR_FORMAT;
  }
  if (rows > 0) {
    if (rstd == nullptr) return FP4_ERR_NULL;
    if ((st = check_matrix(dy, cols, lddy)) != FP4_OK) return st;
    if (xhat8 == nullptr && (st = check_matrix(sum, cols, lds)) != FP4_OK) return st;
    if (dres != nullptr && (st = check_matrix(dres, cols, lddres)) != FP4_OK) return st;
    if ((st = check_matrix(dx, cols, lddx)) != FP4_OK) return st;
  }
  if (!ptr_aligned(rstd, 4) || !ptr_aligned(dweight, 4) || !ptr_aligned(ws, 16)) return FP4_ERR_ALIGN;
  if (dweight != nullptr && (ws == nullptr || ws_bytes < fqt_colsum_workspace_bytes(rows, cols)))
    return FP4_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    if (dweight != nullptr && cudaMemsetAsync(dweight, 0, cols * sizeof(float), s) != cudaSuccess)
      return FP4_ERR_CUDA;
    return FP4_OK;
  }
  BwdParams p{};
  p.dy = static_cast<const __nv_bfloat16*>(dy); p.lddy = lddy;
  p.s = sum; p.lds = lds;
  if (xhat8 != nullptr) { p.codes = xhat8->codes; p.scales = xhat8->scales; }
  p.rstd = rstd; p.w = weight; p.w_f32 = w_dtype == FP4_OUT_F32;
  p.dres = dres; p.lddres = lddres; p.dx = dx; p.lddx = lddx; p.grad_f32 = grad_dtype == FP4_OUT_F32;
  p.rows = rows; p.cols = (int)cols;
  p.partial = dweight != nullptr ? colsum_partials(ws) : nullptr;
  int grid = 0;
  cudaError_t e = xhat8 != nullptr          ? launch_bwd<2>(p, grid, s)
                  : s_dtype == FP4_OUT_F32 ? launch_bwd<1>(p, grid, s)
                                           : launch_bwd<0>(p, grid, s);
  if (e == cudaSuccess && dweight != nullptr) e = launch_colsum(p.partial, grid, cols, dweight, s);
  return e == cudaSuccess ? FP4_OK : FP4_ERR_CUDA;
}

}  // extern "C"
