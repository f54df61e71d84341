// act.cu -- activations and gated activations with 8-bit checkpoints of their
// input: forward (with encoding), recomputation from a checkpoint, backward
// (with the bias gradient).
//
// Elementwise and bound by HBM, so the loads of two rows are issued before the
// arithmetic of either, and the arithmetic runs on pairs (act_device.cuh).  A
// thread owns eight columns (of both halves when gated) and walks down its rows:
// the bias gradient sums in registers and needs no atomics.  A CTA has `lanes`
// threads side by side (8, 16 or 32: 64 to 256 columns) and 256 / lanes rows at a
// time; a grid column covers the width, a grid row a slice of the rows.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

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

// Where a thread's eight values of z are, row by row (`off` columns on: the second
// half's), and the values of one row as they are stored.
template <bool CKPT>
struct Stored;
template <>
struct Stored<false> {
  struct At {
    const __nv_bfloat16* z; int64_t step;
    __device__ __forceinline__ At(const ActParams& p, int64_t row, int64_t c, int64_t rows)
        : z(p.z + row * p.ldz + c), step(rows * p.ldz) {}
    __device__ __forceinline__ void next() { z += step; }
  };
  uint4 q;
  __device__ __forceinline__ void load(const At& at, int64_t off) { q = ld_stream(at.z + off); }
  __device__ __forceinline__ F8 values() const { return bf16x8(q); }
};
template <>
struct Stored<true> {
  struct At {
    const uint8_t* codes; const uint8_t* scales; int64_t step;
    __device__ __forceinline__ At(const ActParams& p, int64_t row, int64_t c, int64_t rows)
        : codes(p.codes + row * p.zcols + c), scales(p.scales + ((row * p.zcols + c) >> 5)),
          step(rows * p.zcols) {}
    __device__ __forceinline__ void next() { codes += step; scales += step >> 5; }
  };
  uint2 q;
  uint32_t byte;
  __device__ __forceinline__ void load(const At& at, int64_t off) {
    q = ld_stream2(at.codes + off);
    byte = at.scales[off >> 5];
  }
  __device__ __forceinline__ F8 values() const { return scaled8(e4m3x8(q), ckpt_scale(byte)); }
};

// Rows whose loads are in flight together: about 40 KB an SM cover the memory's
// latency, and a row of a checkpoint is half a row of BF16 (recomputing ReLU with
// two rows: 0.77 of the copy rate, with four 0.90; gated, four spill up to 12 bytes
// in the activations other than GELU).
constexpr int kRows = 2, kCkptFwdRows = 4;

template <int ACT, bool GATED, bool CKPT>
__global__ void __launch_bounds__(kThreads, 4) act_fwd_kernel(const ActParams p) {
  wait_previous_launch();
  const int lane = threadIdx.x % p.lanes, rows_at_once = kThreads / p.lanes;
  const int64_t c = ((int64_t)blockIdx.x * p.lanes + lane) * 8;
  const int64_t step = (int64_t)gridDim.y * rows_at_once;
  AmaxBf16 amax;
  bool finite = true;
  if (c < p.cols) {
    int64_t row = (int64_t)blockIdx.y * rows_at_once + threadIdx.x / p.lanes;
    typename Stored<CKPT>::At at(p, row, c, step);
    __nv_bfloat16* out = p.out + row * p.ldo + c;
    uint8_t* codes = p.codes_out + row * p.zcols + c;
    uint8_t* scales = p.scales_out + ((row * p.zcols + c) >> 5);
    const int64_t out_step = step * p.ldo, z_step = step * p.zcols;
    auto body = [&](auto rows) {
      constexpr int N = decltype(rows)::value;
      Stored<CKPT> gs[N], us[N];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        gs[k].load(at, 0);
        if constexpr (GATED) us[k].load(at, p.cols);
        at.next();
      }
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const F8 g = gs[k].values();
        F8 u;
        if constexpr (GATED) u = us[k].values();
        if constexpr (!CKPT) {
          if (p.codes_out != nullptr) {
            finite &= encode8(g, codes, scales, true);
            if constexpr (GATED) finite &= encode8(u, codes + p.cols, scales + (p.cols >> 5), true);
            codes += z_step;
            scales += z_step >> 5;
          }
        }
        if (p.out != nullptr) {
          F8 y;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            y.p[i] = act_value2<ACT>(g.p[i]);
            if constexpr (GATED) y.p[i] = mul2(y.p[i], u.p[i]);
          }
          const uint4 packed = pack_bf16x8(y);
          *reinterpret_cast<uint4*>(out) = packed;
          out += out_step;
          if (p.amax != nullptr) amax.add(packed);
        }
      }
    };
    constexpr int R = CKPT ? kCkptFwdRows : kRows;
    for (; row + (R - 1) * step < p.rows; row += R * step) body(std::integral_constant<int, R>{});
    for (; row < p.rows; row += step) body(std::integral_constant<int, 1>{});
  }
  if (threadIdx.x == 0) allow_next_launch();       // its column and first row are always there
  __syncwarp();
  amax.to(p.amax);
  if (!finite) set_status(p.status, FP4_ERR_NONFINITE, 7);
}

// The backward's CTAs to an SM: as many as have registers for two rows each with
// no spills for SwiGLU (16384x8192 from a checkpoint: 0.90 of the copy rate with
// three, 0.89 with four, 0.86 with five of one row; with dbias from BF16 0.90 with
// two, 0.83 with three).  The rule does not look at the activation: without dbias
// others spill a few bytes (-Xptxas -v: gated GELU_TANH from BF16 24 stored and 36
// loaded, at most 12 elsewhere), and SiLU with dbias, not gated, from BF16 8 and 12.
// They run at 0.96 (that GELU_TANH), 0.90-0.92 (gated GELU and ReLU from BF16, ReLU
// from a checkpoint) and 0.89 of the copy rate at 16384x8192.
constexpr int bwd_ctas(bool gated, bool ckpt, bool dbias) { return gated && dbias ? 2 : gated && ckpt ? 3 : 4; }

template <int ACT, bool GATED, bool CKPT, bool DBIAS>
__global__ void __launch_bounds__(kThreads, bwd_ctas(GATED, CKPT, DBIAS)) act_bwd_kernel(const ActParams p) {
  wait_previous_launch();
  const int lane = threadIdx.x % p.lanes, rows_at_once = kThreads / p.lanes;
  const int64_t c = ((int64_t)blockIdx.x * p.lanes + lane) * 8;
  const int64_t step = (int64_t)gridDim.y * rows_at_once;
  AmaxBf16 amax;
  F8 db = zero8(), dbu = zero8();
  if (c < p.cols) {
    int64_t row = (int64_t)blockIdx.y * rows_at_once + threadIdx.x / p.lanes;
    typename Stored<CKPT>::At at(p, row, c, step);
    const __nv_bfloat16* dy_at = p.dy + row * p.lddy + c;
    __nv_bfloat16* out = p.out + row * p.ldo + c;
    const int64_t dy_step = step * p.lddy, out_step = step * p.ldo;
    auto body = [&](auto rows) {
      constexpr int N = decltype(rows)::value;
      Stored<CKPT> gs[N], us[N];
      uint4 dys[N];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        gs[k].load(at, 0);
        if constexpr (GATED) us[k].load(at, p.cols);
        at.next();
        dys[k] = ld_stream(dy_at);
        dy_at += dy_step;
      }
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const F8 g = gs[k].values(), dy = bf16x8(dys[k]);
        F8 d;
        if constexpr (GATED) {
          const F8 u = us[k].values();
          F8 du;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            f32x2 f, df;
            act_both2<ACT>(g.p[i], f, df);
            d.p[i] = mul2(mul2(dy.p[i], u.p[i]), df);
            du.p[i] = mul2(dy.p[i], f);
            if constexpr (DBIAS) dbu.p[i] = add2(dbu.p[i], du.p[i]);
          }
          const uint4 packed = pack_bf16x8(du);
          *reinterpret_cast<uint4*>(out + p.cols) = packed;
          if (p.amax != nullptr) amax.add(packed);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            f32x2 f, df;
            act_both2<ACT>(g.p[i], f, df);
            d.p[i] = mul2(dy.p[i], df);
          }
        }
        if constexpr (DBIAS)
#pragma unroll
          for (int i = 0; i < 4; ++i) db.p[i] = add2(db.p[i], d.p[i]);
        const uint4 packed = pack_bf16x8(d);
        *reinterpret_cast<uint4*>(out) = packed;
        out += out_step;
        if (p.amax != nullptr) amax.add(packed);
      }
    };
    for (; row + (kRows - 1) * step < p.rows; row += kRows * step) body(std::integral_constant<int, kRows>{});
    for (; row < p.rows; row += step) body(std::integral_constant<int, 1>{});
  }
  if (threadIdx.x == 0) allow_next_launch();       // its column and first row are always there
  __syncwarp();
  amax.to(p.amax);
  if constexpr (DBIAS) {
    // join the CTA's rows, half by half
    __shared__ float sums[kThreads * 8];
    const int width = p.lanes * 8;
#pragma unroll
    for (int h = 0; h < (GATED ? 2 : 1); ++h) {
      __syncthreads();
      put8<true>(sums, threadIdx.x * 8, h == 0 ? db : dbu);
      __syncthreads();
      const int64_t col = (int64_t)blockIdx.x * width + threadIdx.x;
      if (threadIdx.x < width && col < p.cols) {
        float a = 0.0f;
        for (int k = 0; k < rows_at_once; ++k) a += sums[k * width + threadIdx.x];
        p.partial[(int64_t)blockIdx.y * p.zcols + h * p.cols + col] = a;
      }
    }
  }
}

// Lanes side by side: as few of 8, 16, 32 as cover the width in one CTA.
int lanes_for(int64_t cols) { return cols <= 64 ? 8 : cols <= 128 ? 16 : 32; }

// Row slices of the grid, for a part of 148 SMs with `per_sm` CTAs each at a time:
// the fewest (of up to 64, and no more than there are groups of rows) that fill
// their waves to 0.96, else those that fill them best; a CTA then has many rows,
// and there are few partial sums.  148 is a constant here, so that
// sums do not depend on the device.  The limit of kMaxSlices, which the partial
// sums have, holds for all calls: where one CTA covers the width, three fit an SM.
dim3 act_grid(int64_t rows, int64_t cols, int lanes, int per_sm) {
  const int64_t wave = 148 * per_sm;
  const int64_t gx = (cols + lanes * 8 - 1) / (lanes * 8);
  const int64_t groups = (rows + kThreads / lanes - 1) / (kThreads / lanes);
  const int64_t least = gx >= wave ? 1 : wave / gx;              // one wave, or just under
  int64_t best = least;
  double full = -1.0;
  for (int64_t gy = least; gy <= 64 && full < 0.96; ++gy) {
    const int64_t n = gx * gy, waves = (n + wave - 1) / wave;
    const double f = (double)n / (double)(waves * wave);
    if (f > full) { full = f; best = gy; }
  }
  if (best > groups) best = groups;
  return dim3((unsigned)gx, (unsigned)(best < kMaxSlices ? best : kMaxSlices));
}

template <bool FWD, int ACT, bool GATED, bool CKPT>
cudaError_t launch_one(const ActParams& p, dim3 grid, cudaStream_t s) {
  if constexpr (FWD) return launch_overlapped(act_fwd_kernel<ACT, GATED, CKPT>, grid, kThreads, 0, s, p);
  else if (p.partial != nullptr)
    return launch_overlapped(act_bwd_kernel<ACT, GATED, CKPT, true>, grid, kThreads, 0, s, p);
  else return launch_overlapped(act_bwd_kernel<ACT, GATED, CKPT, false>, grid, kThreads, 0, s, p);
}

template <bool FWD, int ACT>
cudaError_t launch_act(const ActParams& p, bool gated, bool ckpt, dim3 grid, cudaStream_t s) {
  if (gated && ckpt) return launch_one<FWD, ACT, true, true>(p, grid, s);
  if (gated) return launch_one<FWD, ACT, true, false>(p, grid, s);
  if (ckpt) return launch_one<FWD, ACT, false, true>(p, grid, s);
  return launch_one<FWD, ACT, false, false>(p, grid, s);
}

template <bool FWD>
cudaError_t launch(ActParams& p, int act, bool gated, unsigned& slices, cudaStream_t s) {
  const bool ckpt = p.codes != nullptr;
  p.lanes = lanes_for(p.cols);
  const dim3 grid = act_grid(p.rows, p.cols, p.lanes, FWD ? 4 : bwd_ctas(gated, ckpt, p.partial != nullptr));
  slices = grid.y;
  switch (act) {
    case FQT_ACT_RELU: return launch_act<FWD, FQT_ACT_RELU>(p, gated, ckpt, grid, s);
    case FQT_ACT_GELU: return launch_act<FWD, FQT_ACT_GELU>(p, gated, ckpt, grid, s);
    case FQT_ACT_GELU_TANH: return launch_act<FWD, FQT_ACT_GELU_TANH>(p, gated, ckpt, grid, s);
    case FQT_ACT_SILU: return launch_act<FWD, FQT_ACT_SILU>(p, gated, ckpt, grid, s);
    default: return launch_act<FWD, FQT_ACT_NONE>(p, gated, ckpt, grid, s);
  }
}

// The checks that both directions make of their shape and of z; z's row length.
constexpr int64_t kMaxZCols = (int64_t)1 << 30;
fp4_status check_act(const void* z, int64_t ldz, const fqt_ckpt8* z8, int32_t act, int32_t gated,
                     int64_t rows, int64_t cols, const void* ws, size_t ws_bytes, int64_t& zcols) {
  if (!known_act(act)) return FP4_ERR_FORMAT;
  if (rows < 0 || cols <= 0 || cols % 8 || cols > (gated ? kMaxZCols / 2 : kMaxZCols)) return FP4_ERR_SHAPE;
  zcols = gated ? 2 * cols : cols;
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

fp4_status fqt_act_fwd(const fqt_act_fwd_args* args, void* ws, size_t ws_bytes, void* stream) {
  if (args == nullptr) return FP4_ERR_NULL;
  const auto& [z, ldz, z8_in, y, ldy, z8_out, y_amax, rows, cols, act, gated] = *args;
  int64_t zcols = 0;
  fp4_status st = check_act(z, ldz, z8_in, act, gated, rows, cols, ws, ws_bytes, zcols);
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

fp4_status fqt_act_bwd(const fqt_act_bwd_args* args, void* ws, size_t ws_bytes, void* stream) {
  if (args == nullptr) return FP4_ERR_NULL;
  const auto& [dy, lddy, z, ldz, z8, dz, lddz, dbias, dz_amax, rows, cols, act, gated] = *args;
  int64_t zcols = 0;
  fp4_status st = check_act(z, ldz, z8, act, gated, rows, cols, ws, ws_bytes, zcols);
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
