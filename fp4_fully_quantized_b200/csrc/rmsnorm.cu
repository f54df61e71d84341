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
// Both kernels are bound by HBM.  What that takes is bytes in flight while a
// row's two phases (sum, then outputs) run, and few instructions a value:
//  - persistent CTAs of independent thread groups, a row (or, below 33 threads,
//    a few) to a group at a time, up to four chunks of eight columns to a thread
//    (one chunk and four times the threads spent 1.4 us a row of 4096 on issue);
//  - a group has a ring of bulk copies (cp.async.bulk onto an mbarrier) that
//    brings its next rows to shared memory, and a barrier of its own, so that
//    the groups of an SM are in different phases;
//  - rows that fill their threads' chunks take a path without bounds.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cfloat>
#include <cstdint>
#include <type_traits>

#include "act_device.cuh"
#include "fp4_device.cuh"
#include "internal.h"
#include "sm100_ptx.cuh"

namespace fp4impl {
using namespace fp4dev;
namespace {

constexpr int kMaxCols = 16384;      // 512 threads x 4 chunks of 8
constexpr int kMaxStages = 8;

struct FwdParams {
  const __nv_bfloat16* x; int64_t ldx;
  const void* res; int64_t ldr;
  void* res_out; int64_t ldo;
  const void* w; bool w_f32;
  float eps; int64_t rows; int cols;
  __nv_bfloat16* y; int64_t ldy;
  uint8_t* codes; uint8_t* scales; bool q_xhat;
  float* rstd; float* y_amax; uint32_t* status;
  int T, stages;
};

struct BwdParams {
  const __nv_bfloat16* dy; int64_t lddy;
  const void* s; int64_t lds;
  const uint8_t* codes; const uint8_t* scales;
  const float* rstd; const void* w; bool w_f32;
  const void* dres; int64_t lddres;
  void* dx; int64_t lddx; bool grad_f32;
  int64_t rows; int cols;
  float* partial; uint32_t* status;
  int T, stages;
};

// A group's ring: `stages` slots, each with up to three sources' rows of one
// tile (the rows a group takes at a time).  Tile t of the group's sequence uses
// slot t % stages.
struct Source { const char* base; int64_t pitch; int row_bytes; };   // pitch in bytes

template <int N>
struct Ring {
  Source src[N];
  uint32_t bars, data;           // shared-memory addresses
  int stages, stage_bytes, rows_per_tile;
  int64_t rows;

  // Called by the group's first warp: copies the rows of `tile` into `slot`.
  // Rows that lie side by side in memory are one copy, others one each.
  __device__ __forceinline__ void fetch(int64_t tile, int slot) const {
    const int lane = threadIdx.x & 31;
    const int64_t row0 = tile * rows_per_tile;
    const int n = (int)(rows - row0 < rows_per_tile ? rows - row0 : rows_per_tile);
    const uint32_t bar = bars + 8 * slot;
    if (lane == 0) {
      uint32_t bytes = 0;
#pragma unroll
      for (int j = 0; j < N; ++j) bytes += (uint32_t)(n * src[j].row_bytes);
      ptx::mbar_arrive_expect_tx(bar, bytes);
    }
    __syncwarp();
    uint32_t dst = data + slot * stage_bytes;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int bytes = src[j].row_bytes;
      if (bytes != 0) {
        const char* from = src[j].base + row0 * src[j].pitch;
        if (src[j].pitch == bytes || rows_per_tile == 1) {
          if (lane == 0) ptx::bulk_load(dst, from, (uint32_t)(n * bytes), bar);
        } else {
          for (int r = lane; r < n; r += 32)
            ptx::bulk_load(dst + r * bytes, from + r * src[j].pitch, (uint32_t)bytes, bar);
        }
        dst += bytes * rows_per_tile;
      }
    }
  }
  // Bounded wait for a slot's copies.
  __device__ __forceinline__ bool wait(int slot, uint32_t parity) const {
    if (ptx::mbar_try_wait(bars + 8 * slot, parity)) return true;
    const uint64_t t0 = ptx::globaltimer();
    while (!ptx::mbar_try_wait_sleep(bars + 8 * slot, parity))
      if (ptx::globaltimer() - t0 > ptx::kWaitNs) return false;
    return true;
  }
};

// The group's barrier, with the OR of `flag` over its threads.
__device__ __forceinline__ bool group_sync_or(int group, int threads, bool flag) {
  if (threads == 32) {
    __syncwarp();
    return __any_sync(0xFFFFFFFFu, flag);
  }
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %3, 0;\n\t"
      "barrier.cta.red.or.pred p, %1, %2, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(any) : "r"(group + 1), "r"(threads), "r"((uint32_t)flag) : "memory");
  return any != 0;
}

// Sum over the T threads of a row: W lanes of a warp (all of a row of up to 32
// threads), then the row's warps through `slot`, one float a warp.  The group's
// barrier is in here, whatever T is.  Every thread of the row gets the same
// value, added in a fixed order.
template <int W>
__device__ __forceinline__ float row_sum(float v, float* slot, int T, int group, bool& failed) {
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if (W < 32 || T == 32) {
    failed = group_sync_or(group, 32, failed);
  } else {
    const int warps = T >> 5, lane = threadIdx.x & 31, i = lane & 15;     // at most 16 warps
    if (lane == 0) slot[threadIdx.x >> 5] = v;
    failed = group_sync_or(group, T, failed);
    v = i < warps ? slot[group * warps + i] : 0.0f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  }
  return v;
}

// What both kernels set up: the barriers, each group's first copies, and the
// weights as FP32 behind the rings.
template <int N>
__device__ __forceinline__ void ring_start(Ring<N>& ring, uint8_t* smem, uint64_t* bars, int stages,
                                           int group, int groups, bool first_warp, int64_t tile0,
                                           int64_t step, int64_t tiles, int cols, const void* w,
                                           bool w_f32) {
  ring.bars = ptx::smem_u32(bars + group * stages);
  ring.data = ptx::smem_u32(smem) + group * stages * ring.stage_bytes;
  ring.stages = stages;
  if (threadIdx.x == 0) {
    for (int i = 0; i < groups * stages; ++i) ptx::mbar_init(ptx::smem_u32(bars) + 8 * i, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  wait_previous_launch();
  __syncthreads();
  if (first_warp)
    for (int i = 0; i < stages; ++i)
      if (tile0 + i * step < tiles) ring.fetch(tile0 + i * step, i);
  float* const ws = reinterpret_cast<float*>(smem + groups * stages * ring.stage_bytes);
  for (int c = threadIdx.x * 8; c < cols; c += blockDim.x * 8) {
    float v[8];
    load8(w, c, w_f32, v);
    store8(ws, c, true, v);
  }
  __syncthreads();
}

// After a copy that did not arrive in time: wait for those still on their way,
// so that none writes to shared memory that is no longer this CTA's.
template <int N>
__device__ __forceinline__ void ring_give_up(const Ring<N>& ring, int slot, uint32_t phase,
                                             uint32_t* status, uint32_t where) {
  set_status(status, FP4_ERR_TIMEOUT, where);
  for (int i = 0; i < ring.stages; ++i) ring.wait(i, i < slot ? phase ^ 1u : phase);
}

// The place of a thread: T threads to a row, groups of max(T, 32) threads.
struct Place {
  int T, group_threads, group, groups, rows_per_tile, gl, rl;
  bool first_warp;
  __device__ __forceinline__ Place(int t)
      : T(t), group_threads(t < 32 ? 32 : t), group(threadIdx.x / group_threads),
        groups(blockDim.x / group_threads), rows_per_tile(group_threads / t), gl(threadIdx.x % t),
        rl(threadIdx.x % group_threads / t), first_warp(threadIdx.x % group_threads < 32) {}
};

constexpr int kMaxBars = 8 * kMaxStages;

// RES: 0 no residual, 1 BF16, 2 FP32.  W: lanes of a warp that share a row; V:
// chunks of a thread, T * (V - 1) < cols / 8 <= T * V.
template <int W, int V, int RES, int THREADS>
__global__ void __launch_bounds__(THREADS, V <= 2 ? 3 : 512 / THREADS)
rmsnorm_fwd_kernel(const FwdParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float slots[2][16];
  __shared__ __align__(8) uint64_t bars[kMaxBars];
  constexpr int RSZ = RES == 2 ? 4 : 2;
  const Place at(W < 32 ? W : p.T);
  const int T = at.T;
  const int64_t tiles = (p.rows + at.rows_per_tile - 1) / at.rows_per_tile;
  const int64_t tile0 = (int64_t)blockIdx.x * at.groups + at.group, step = (int64_t)gridDim.x * at.groups;
  const float inv_cols = 1.0f / (float)p.cols;
  Ring<RES ? 2 : 1> ring;
  ring.src[0] = {reinterpret_cast<const char*>(p.x), p.ldx * 2, p.cols * 2};
  if constexpr (RES != 0) ring.src[1] = {static_cast<const char*>(p.res), p.ldr * RSZ, p.cols * RSZ};
  ring.rows_per_tile = at.rows_per_tile;
  ring.stage_bytes = at.rows_per_tile * p.cols * (2 + (RES ? RSZ : 0));
  ring.rows = p.rows;
  ring_start(ring, smem, bars, p.stages, at.group, at.groups, at.first_warp, tile0, step, tiles, p.cols,
             p.w, p.w_f32);
  const uint8_t* const data = smem + at.group * p.stages * ring.stage_bytes;
  const int c0 = at.gl * 8, x_at = at.rl * p.cols + c0, r_at = at.rows_per_tile * p.cols * 2;
  const float* const ws = reinterpret_cast<const float*>(smem + at.groups * p.stages * ring.stage_bytes) + c0;
  const bool last = c0 + (V - 1) * T * 8 < p.cols;      // the last chunk exists
  AmaxBf16 amax;
  uint32_t phase = 0;
  bool finite = true, failed = false;
  int slot = 0, flip = 0;
  // this thread's first column in the outputs' rows, a step of tiles at a time
  int64_t row = tile0 * at.rows_per_tile + at.rl;
  const int64_t row_step = step * at.rows_per_tile;
  __nv_bfloat16* y = p.y + row * p.ldy + c0;
  uint8_t* codes = p.codes + row * p.cols + c0;
  uint8_t* scales = p.scales + row * (p.cols >> 5) + (c0 >> 5);
  char* res_out = static_cast<char*>(p.res_out) + (row * p.ldo + c0) * RSZ;
  const int64_t y_step = row_step * p.ldy, q_step = row_step * p.cols, o_step = row_step * p.ldo * RSZ;

  auto body = [&](int64_t tile, auto full) {
    constexpr bool FULL = decltype(full)::value;
    const bool row_ok = FULL || row < p.rows;
    failed = !ring.wait(slot, phase);
    const uint8_t* in = data + slot * ring.stage_bytes;
    F8 s[V];
    f32x2 sq = 0ull;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      s[v] = zero8();
      if (FULL || (row_ok && (v < V - 1 || last))) {
        s[v] = get8<false>(in, x_at + v * T * 8);
        if constexpr (RES != 0) {
          const F8 r = get8<RES == 2>(in + r_at, x_at + v * T * 8);
#pragma unroll
          for (int i = 0; i < 4; ++i) s[v].p[i] = add2(s[v].p[i], r.p[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) sq = fma2(s[v].p[i], s[v].p[i], sq);
    }
    float ss = unpair(sq).x + unpair(sq).y;
    ss = row_sum<W>(ss, slots[flip], T, at.group, failed);
    if (failed) return;
    // every thread has its part of the tile in registers: the slot is free
    const int64_t next = tile + p.stages * step;
    if (at.first_warp && next < tiles) ring.fetch(next, slot);
    if (++slot == p.stages) { slot = 0; phase ^= 1u; }
    const float rstd = rsqrtf(ss * inv_cols + p.eps);
    if (p.rstd != nullptr && at.gl == 0 && row_ok) p.rstd[row] = rstd;
    auto encode = [&] {
#pragma unroll
      for (int v = 0; v < V; ++v)
        finite &= encode8(s[v], codes + v * T * 8, scales + v * T / 4, FULL || (row_ok && (v < V - 1 || last)));
    };
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (RES != 0 && (FULL || (row_ok && (v < V - 1 || last)))) put8<RES == 2>(res_out, v * T * 8, s[v]);
      s[v] = scaled8(s[v], rstd);
    }
    if (p.codes != nullptr && p.q_xhat) encode();
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (FULL || v < V - 1 || last) {
        const F8 w = get8<true>(ws, v * T * 8);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[v].p[i] = mul2(s[v].p[i], w.p[i]);
      }
    if (p.codes != nullptr && !p.q_xhat) encode();
    if (p.y != nullptr || p.y_amax != nullptr) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (FULL || (row_ok && (v < V - 1 || last))) {
          const uint4 packed = pack_bf16x8(s[v]);
          if (p.y != nullptr) *reinterpret_cast<uint4*>(y + v * T * 8) = packed;
          if (p.y_amax != nullptr) amax.add(packed);
        }
    }
    row += row_step;
    y += y_step;
    codes += q_step;
    scales += q_step >> 5;
    res_out += o_step;
  };
  const bool whole = V * T * 8 == p.cols;
  for (int64_t tile = tile0; tile < tiles && !failed; tile += step, flip ^= 1) {
    if (whole && (tile + 1) * at.rows_per_tile <= p.rows) body(tile, std::true_type{});
    else body(tile, std::false_type{});
  }
  if (tile0 < tiles) allow_next_launch();      // the CTA's first group always has a tile
  if (failed && at.first_warp) ring_give_up(ring, slot, phase, p.status, 0x4100);
  __syncwarp();
  amax.to(p.y_amax);
  if (!finite) set_status(p.status, FP4_ERR_NONFINITE, 6);
}

// SRC: 0 the stored sum in BF16, 1 in FP32, 2 the 8-bit checkpoint of xhat.
// GF32: dres and dx in FP32.  Of the forms with four chunks the FP32 sum with BF16
// gradients spills (48 bytes stored, 92 loaded; 32768x4096 with dres 252 us, 0.81
// of the copy rate, against 303 us, 0.95, with FP32 gradients), the checkpoint with
// BF16 ones 8 bytes.
template <int W, int V, int SRC, bool GF32, int THREADS>
__global__ void __launch_bounds__(THREADS, V <= 2 ? 3 : 512 / THREADS)
rmsnorm_bwd_kernel(const BwdParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float slots[2][16];
  __shared__ __align__(8) uint64_t bars[kMaxBars];
  constexpr int SSZ = SRC == 2 ? 1 : SRC == 1 ? 4 : 2, GSZ = GF32 ? 4 : 2;
  const Place at(W < 32 ? W : p.T);
  const int T = at.T;
  const int64_t tiles = (p.rows + at.rows_per_tile - 1) / at.rows_per_tile;
  const int64_t tile0 = (int64_t)blockIdx.x * at.groups + at.group, step = (int64_t)gridDim.x * at.groups;
  const float inv_cols = 1.0f / (float)p.cols;
  const bool has_dres = p.dres != nullptr;
  Ring<3> ring;
  ring.src[0] = {reinterpret_cast<const char*>(p.dy), p.lddy * 2, p.cols * 2};
  if constexpr (SRC == 2) ring.src[1] = {reinterpret_cast<const char*>(p.codes), p.cols, p.cols};
  else ring.src[1] = {static_cast<const char*>(p.s), p.lds * SSZ, p.cols * SSZ};
  ring.src[2] = {static_cast<const char*>(p.dres), p.lddres * GSZ, has_dres ? p.cols * GSZ : 0};
  ring.rows_per_tile = at.rows_per_tile;
  ring.stage_bytes = at.rows_per_tile * (p.cols * (2 + SSZ) + ring.src[2].row_bytes);
  ring.rows = p.rows;
  ring_start(ring, smem, bars, p.stages, at.group, at.groups, at.first_warp, tile0, step, tiles, p.cols,
             p.w, p.w_f32);
  const uint8_t* const data = smem + at.group * p.stages * ring.stage_bytes;
  const int c0 = at.gl * 8, x_at = at.rl * p.cols + c0;
  const int s_at = at.rows_per_tile * p.cols * 2, r_at = at.rows_per_tile * p.cols * (2 + SSZ);
  const float* const ws = reinterpret_cast<const float*>(smem + at.groups * p.stages * ring.stage_bytes) + c0;
  const bool last = c0 + (V - 1) * T * 8 < p.cols;
  F8 dw[V];
#pragma unroll
  for (int v = 0; v < V; ++v) dw[v] = zero8();
  bool failed = false;
  uint32_t phase = 0;
  int slot = 0, flip = 0;
  int64_t row = tile0 * at.rows_per_tile + at.rl;
  const int64_t row_step = step * at.rows_per_tile;
  char* dx = static_cast<char*>(p.dx) + (row * p.lddx + c0) * GSZ;
  const int64_t dx_step = row_step * p.lddx * GSZ;
  // rstd and the checkpoint's scales come straight from memory, a tile ahead
  const uint8_t* scales = p.scales + ((row * p.cols + c0) >> 5);
  const int64_t scales_step = row_step * p.cols >> 5;
  float rstd_next = 0.0f;
  uint32_t scale_next[V];
  auto ahead = [&](int64_t r) {
    const bool row_ok = r < p.rows;
    rstd_next = row_ok ? p.rstd[r] : 0.0f;
    if constexpr (SRC == 2) {
#pragma unroll
      for (int v = 0; v < V; ++v) scale_next[v] = row_ok && (v < V - 1 || last) ? scales[v * T / 4] : 0u;
      scales += scales_step;
    }
  };
  ahead(row);

  auto body = [&](int64_t tile, auto full) {
    constexpr bool FULL = decltype(full)::value;
    const bool row_ok = FULL || row < p.rows;
    const float rstd = rstd_next;
    float e[V];                            // xhat = e * what is stored
#pragma unroll
    for (int v = 0; v < V; ++v) e[v] = SRC == 2 ? ckpt_scale(scale_next[v]) : rstd;
    ahead(row + row_step);
    failed = !ring.wait(slot, phase);
    const uint8_t* in = data + slot * ring.stage_bytes;
    // Both passes read the row from shared memory: between them a thread holds
    // its weight sums and little else, so that two CTAs fit an SM.
    auto stored = [&](int v) {
      if constexpr (SRC == 2) return e4m3x8(*reinterpret_cast<const uint2*>(in + s_at + x_at + v * T * 8));
      else return get8<SRC == 1>(in + s_at, x_at + v * T * 8);
    };
    float dot = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (FULL || (row_ok && (v < V - 1 || last))) {
        const F8 q = stored(v), d = get8<false>(in, x_at + v * T * 8), w = get8<true>(ws, v * T * 8);
        const f32x2 ee = pair(e[v], e[v]);
        f32x2 part = 0ull;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x2 t = mul2(mul2(q.p[i], ee), d.p[i]);      // dy * xhat
          dw[v].p[i] = add2(dw[v].p[i], t);
          part = fma2(t, w.p[i], part);
        }
        dot += unpair(part).x + unpair(part).y;
      }
    const float k = row_sum<W>(dot, slots[flip], T, at.group, failed) * inv_cols * -rstd;
    if (failed) return;
    // every thread is done with the tile before this one: its slot is free
    if (p.stages > 1 && tile != tile0) {
      const int64_t next = tile + (p.stages - 1) * step;
      if (at.first_warp && next < tiles) ring.fetch(next, slot == 0 ? p.stages - 1 : slot - 1);
    }
    const f32x2 rr = pair(rstd, rstd);
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (FULL || (row_ok && (v < V - 1 || last))) {
        const F8 q = stored(v), d = get8<false>(in, x_at + v * T * 8), w = get8<true>(ws, v * T * 8);
        F8 o = scaled8(q, k * e[v]);
        if (has_dres) {
          const F8 r = get8<GF32>(in + r_at, x_at + v * T * 8);
#pragma unroll
          for (int i = 0; i < 4; ++i) o.p[i] = add2(o.p[i], r.p[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) o.p[i] = fma2(mul2(d.p[i], w.p[i]), rr, o.p[i]);
        put8<GF32>(dx, v * T * 8, o);
      }
    if (p.stages == 1) {
      group_sync_or(at.group, at.group_threads, false);
      if (at.first_warp && tile + step < tiles) ring.fetch(tile + step, 0);
    }
    if (++slot == p.stages) { slot = 0; phase ^= 1u; }
    row += row_step;
    dx += dx_step;
  };
  const bool whole = V * T * 8 == p.cols;
  for (int64_t tile = tile0; tile < tiles && !failed; tile += step, flip ^= 1) {
    if (whole && (tile + 1) * at.rows_per_tile <= p.rows) body(tile, std::true_type{});
    else body(tile, std::false_type{});
  }
  if (tile0 < tiles) allow_next_launch();      // the CTA's first group always has a tile
  if (failed && at.first_warp) ring_give_up(ring, slot, phase, p.status, 0x4200);
  if (p.partial == nullptr) return;
  // join the CTA's rows through shared memory (no copies are on their way: every
  // one that was issued has been waited for)
  const int rows_held = at.groups * at.rows_per_tile;
  float* out = p.partial + (int64_t)blockIdx.x * p.cols;
  __syncthreads();
  float* sums = rows_held == 1 ? out + c0
                               : reinterpret_cast<float*>(smem) + (at.group * at.rows_per_tile + at.rl) * p.cols + c0;
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (v < V - 1 || last) put8<true>(sums, v * T * 8, dw[v]);
  if (rows_held == 1) return;
  __syncthreads();
  for (int c = threadIdx.x; c < p.cols; c += blockDim.x) {
    float a = 0.0f;
    for (int i = 0; i < rows_held; ++i) a += reinterpret_cast<const float*>(smem)[i * p.cols + c];
    out[c] = a;
  }
}

// T threads to a row with at most four chunks of eight columns each: 8 or 16 for
// short rows, else whole warps.  An SM gets about 512 threads (at 128 registers),
// as two or three CTAs where the weights' copies leave each ring two stages, else
// as one CTA (one stage, in the backward of 8192 columns: 0.67 of the copy rate
// against 0.85).  A forward that moves nine bytes a value or more gets 256
// threads: fewer rows at a time are in flight then, and the memory's mix of reads
// and writes mostly runs better.  Both sides in turn on one GPU, shares of the copy
// rate at 134 million values, rows of 512, 1024, 2048, 4096 and 8192: BF16 residual
// and checkpoint (9 bytes) 0.97, 0.93, 0.87, 0.84, 0.86 against 0.85, 0.84, 0.84,
// 0.83, 0.83; FP32 residual (12) 0.84, 0.84, 0.85, 0.87, 0.99 against 0.86, 0.88,
// 0.81, 0.83, 0.87; with a checkpoint too (13) 0.85-0.86 against 0.85-0.87.  Below
// nine, 256 threads do not issue fast enough (4 bytes: 0.69 against 0.94; 8 bytes:
// 0.86 against 0.88).  Short rows (two chunks a thread at most, 80
// registers) run three CTAs of 256 threads (40001x128: 7.4 us against 8.1 with two).
struct RowPlan { int T, chunks, threads, rows_per_cta, stages, smem, per_sm; };
RowPlan row_plan(int64_t cols, int bytes_per_value, bool row_sums, bool few) {
  const int64_t n = cols / 8;
  RowPlan r{8, 0, 0, 0, 0, 0, 0};
  if (n > 32) r.T = 16;
  if (n > 64) r.T = (int)((n + 127) / 128) * 32;
  r.chunks = (int)((n + r.T - 1) / r.T);
  const int group = r.T < 32 ? 32 : r.T;
  const int64_t weights = 4 * cols;
  // stages that fit when the SM's 228 KB (1 KB of them and the static part of
  // each CTA taken off) are shared by per_sm CTAs of `groups` groups
  auto fit = [&](int groups, int per_sm) {
    const int64_t stage = (int64_t)(groups * group / r.T) * cols * bytes_per_value;
    const int64_t s = (228 * 1024 / per_sm - 2048 - weights) / stage;
    r.threads = groups * group;
    r.rows_per_cta = r.threads / r.T;
    r.per_sm = per_sm;
    r.stages = (int)(s < 1 ? 1 : s < kMaxStages ? s : kMaxStages);
    r.smem = (int)(r.stages * stage + weights);
    return s;
  };
  const int small = group > 256 ? 1 : 256 / group;
  int64_t stages = few && group <= 256 ? fit((256 + group - 1) / group, 1) : 0;
  for (int per_sm = r.chunks <= 2 ? 3 : 512 / (small * group); per_sm >= 2 && stages < 2; --per_sm) stages = fit(small, per_sm);
  for (int groups = (r.T < 32 ? 256 : 512) / group; groups >= 1 && stages < 2; --groups) stages = fit(groups, 1);
  const int sums = row_sums ? r.threads * r.chunks * 8 * 4 : 0;     // the rows' weight sums at the end
  if (r.smem < sums) r.smem = sums;
  return r;
}

// Lets a kernel take all of an SM's shared memory, once per device (a bit each
// of `allowed`): half a microsecond of a small call otherwise.
cudaError_t allow_shared(const void* kernel, std::atomic<uint64_t>& allowed) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
  if (bit != 0 && (allowed.load(std::memory_order_relaxed) & bit) != 0) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024 - 1024);
  if (e == cudaSuccess) allowed.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

template <typename P>
cudaError_t launch_rows(void (*kernel)(const P), std::atomic<uint64_t>& allowed, P& p, const RowPlan& r,
                        int grid, cudaStream_t s) {
  p.T = r.T;
  p.stages = r.stages;
  if (const cudaError_t e = allow_shared(reinterpret_cast<const void*>(kernel), allowed); e != cudaSuccess)
    return e;
  return launch_overlapped(kernel, dim3((unsigned)grid), r.threads, (size_t)r.smem, s, p);
}

template <int RES>
cudaError_t launch_fwd(FwdParams& p, cudaStream_t s) {
  const int in = 2 + (RES == 2 ? 4 : RES == 1 ? 2 : 0), out = in - 2 + (p.y ? 2 : 0) + (p.codes ? 1 : 0);
  const RowPlan r = row_plan(p.cols, in, false, in + out >= 9);
  const int64_t want = (p.rows + r.rows_per_cta - 1) / r.rows_per_cta;
  const int64_t room = (int64_t)sm_count() * r.per_sm;
  const int grid = (int)(want < room ? want : room);
#define FP4_FWD(W, V, THREADS)                                                        \
  do {                                                                                \
    static std::atomic<uint64_t> allowed{0};                                          \
    return launch_rows(rmsnorm_fwd_kernel<W, V, RES, THREADS>, allowed, p, r, grid, s); \
  } while (0)
  if (r.T == 8) {
    if (r.chunks == 1) FP4_FWD(8, 1, 256);
    if (r.chunks == 2) FP4_FWD(8, 2, 256);
    if (r.chunks == 3) FP4_FWD(8, 3, 256);
    FP4_FWD(8, 4, 256);
  }
  if (r.T == 16) {
    if (r.chunks == 3) FP4_FWD(16, 3, 256);
    FP4_FWD(16, 4, 256);
  }
  if (r.threads > 256) {
    if (r.chunks == 3) FP4_FWD(32, 3, 512);
    FP4_FWD(32, 4, 512);
  }
  if (r.chunks == 3) FP4_FWD(32, 3, 256);
  FP4_FWD(32, 4, 256);
#undef FP4_FWD
}

template <int SRC, bool GF32>
cudaError_t launch_bwd(BwdParams& p, int& grid, cudaStream_t s) {
  const int dres = p.dres == nullptr ? 0 : GF32 ? 4 : 2;
  const RowPlan r = row_plan(p.cols, 2 + (SRC == 2 ? 1 : SRC == 1 ? 4 : 2) + dres, p.partial != nullptr, false);
  const int64_t want = (p.rows + r.rows_per_cta - 1) / r.rows_per_cta;
  const int64_t room = kMaxSlices / 3 * r.per_sm;
  grid = (int)(want < room ? want : room);
#define FP4_BWD(W, V, THREADS)                                                              \
  do {                                                                                      \
    static std::atomic<uint64_t> allowed{0};                                                \
    return launch_rows(rmsnorm_bwd_kernel<W, V, SRC, GF32, THREADS>, allowed, p, r, grid, s); \
  } while (0)
  if (r.T == 8) {
    if (r.chunks == 1) FP4_BWD(8, 1, 256);
    if (r.chunks == 2) FP4_BWD(8, 2, 256);
    if (r.chunks == 3) FP4_BWD(8, 3, 256);
    FP4_BWD(8, 4, 256);
  }
  if (r.T == 16) {
    if (r.chunks == 3) FP4_BWD(16, 3, 256);
    FP4_BWD(16, 4, 256);
  }
  if (r.threads > 256) {
    if (r.chunks == 3) FP4_BWD(32, 3, 512);
    FP4_BWD(32, 4, 512);
  }
  if (r.chunks == 3) FP4_BWD(32, 3, 256);
  FP4_BWD(32, 4, 256);
#undef FP4_BWD
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

fp4_status fqt_rmsnorm_fwd(const fqt_rmsnorm_fwd_args* args, void* ws, size_t ws_bytes, void* stream) {
  if (args == nullptr) return FP4_ERR_NULL;
  const auto& [x, ldx, residual, ldr, res_out, ldo, weight, y, ldy, q8, rstd, y_amax, rows, cols, eps,
               res_dtype, w_dtype, q8_of] = *args;
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

fp4_status fqt_rmsnorm_bwd(const fqt_rmsnorm_bwd_args* args, void* ws, size_t ws_bytes, void* stream) {
  if (args == nullptr) return FP4_ERR_NULL;
  const auto& [dy, lddy, sum, lds, xhat8, rstd, weight, dres, lddres, dx, lddx, dweight, rows, cols,
               s_dtype, w_dtype, grad_dtype] = *args;
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
  p.status = static_cast<uint32_t*>(ws);
  int grid = 0;
  const int src = xhat8 != nullptr ? 2 : s_dtype == FP4_OUT_F32 ? 1 : 0;
  cudaError_t e = src == 2   ? (p.grad_f32 ? launch_bwd<2, true>(p, grid, s) : launch_bwd<2, false>(p, grid, s))
                  : src == 1 ? (p.grad_f32 ? launch_bwd<1, true>(p, grid, s) : launch_bwd<1, false>(p, grid, s))
                             : (p.grad_f32 ? launch_bwd<0, true>(p, grid, s) : launch_bwd<0, false>(p, grid, s));
  if (e == cudaSuccess && dweight != nullptr) e = launch_colsum(p.partial, grid, cols, dweight, s);
  return e == cudaSuccess ? FP4_OK : FP4_ERR_CUDA;
}

}  // extern "C"
