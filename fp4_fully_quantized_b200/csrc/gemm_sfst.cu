// gemm_sfst.cu -- block-scaled FP4 GEMM with scale factors staged by
// tcgen05.st (one SM per 128 x 256 output tile), and its form with bias,
// activation, residual and 8-bit checkpoint in the epilogue (EPI).
//
// The product is the one of the "FP4" page (How it works: FP4 tensor-core
// products with higher-precision accumulation).  The design point is how the
// per-block scales reach tensor memory.  Copying them with tcgen05.cp from the
// MMA-issuing thread puts 12 copies per 256-element K step into the same
// in-order tensor pipe as the 4 MMAs, and measured on B200 the MMAs then run at
// about half their rate.  Here four "scale" warps, one per TMEM lane quadrant,
// read each stage's scale atoms from shared memory and write them into the
// stage's TMEM slot with tcgen05.st, which proceeds alongside the MMAs; the
// MMA thread only issues MMAs.
//
// 512 threads:
//   warps 0..3   scale stagers (TMEM lane quadrant = warp), one K step at a time
//   warps 4..11  epilogue: quadrant warp % 4, column half (warp - 4) / 4
//   warp 12      TMA producer (A, B and the scale atoms into a 4-stage ring)
//   warp 13      TMEM allocation and MMA issue
// Barriers per stage: atoms (the scale atoms landed) -> scales (4 stagers
// wrote TMEM); full (the A and B tiles landed); the MMAs wait for both, and
// empty (the MMAs that read the stage finished; tcgen05.commit) frees the stage
// and its TMEM slot.  All waits are bounded.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "act_device.cuh"
#include "fp4_device.cuh"
#include "internal.h"
#include "sm100_ptx.cuh"

namespace fp4impl {
namespace {
using namespace ptx;

constexpr int BM = 128, BK = 256, MMA_K = 64;
constexpr int NUM_THREADS = 512;
constexpr int SF_WARP0 = 0, EPI_WARP0 = 4, EPI_WARPS = 8, PRODUCER_WARP = 12, MMA_WARP = 13;
constexpr int TMEM_COLS = 512;

// What depends on the tile's width BN: 256, or 128 for products of few tiles
// (EPI kernels only, see narrow_tiles).
template <int BN_>
struct Tile {
  static constexpr int BN = BN_;
  static constexpr int STAGES = BN == 256 ? 4 : 6;
  static constexpr int ATOM_ROWS = BN / 128;             // scale atoms of B per K block
  static constexpr int A_BYTES = BM * BK / 2;            // 16 KB
  static constexpr int B_BYTES = BN * BK / 2;            // 32 KB (16 KB)
  static constexpr int SFA_BYTES = 4 * 512;
  static constexpr int SFB_BYTES = ATOM_ROWS * 4 * 512;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + SFA_BYTES + SFB_BYTES;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + 1024 + 256;
  static constexpr int EPI_SMEM_BYTES = SMEM_BYTES + EPI_WARPS * (BN / 2) * 4;   // and the bias values
  static constexpr int TMEM_SF_BASE = BN;
  static constexpr int TMEM_SF_STAGE = 16 + 16 * ATOM_ROWS;   // A's and B's columns per stage
  static_assert(TMEM_SF_BASE + STAGES * TMEM_SF_STAGE <= TMEM_COLS, "TMEM budget");
  static_assert(EPI_SMEM_BYTES <= 232448, "shared-memory budget");
  static_assert(8 * (4 * STAGES + 3) + 8 <= 256, "barrier area");
};

struct StParams {
  const uint8_t* a_sf; const uint8_t* b_sf;
  const float* a_sdec; const float* b_sdec;
  int M, N, K;
  int atoms_per_rowblk;
  float alpha;
  void* c; int64_t ldc; int out_mode;     // 0 BF16, 1 FP32, 2 NVFP4 1x16 RTN (q_*)
  float* c_amax;
  uint8_t* q_codes; uint8_t* q_scales; uint8_t* q_scales_mma;
  const float* q_amax_in; float* q_amax_out; float* q_s_dec;
  int q_sr;                   // out_mode 2: stochastic rounding (else to nearest)
  uint32_t q_stream;          // its Philox stream; keys below
  fp4dev::PhiloxKeys q_keys;
  // EPI kernels: bias, activation, residual, 8-bit checkpoint
  int act;
  const void* bias; bool bias_f32;
  const void* res; int64_t ldr; bool res_f32; bool res_wide;   // rows 32-byte aligned
  uint8_t* z_codes; uint8_t* z_scales; bool z_wide;   // codes 32-byte aligned
  uint32_t* status;
};

// Tile order: groups of kGroupM row blocks are walked column block by column
// block (row block fastest), so the tiles the persistent CTAs work on at one
// time share few A row blocks and few B column blocks, and both stay in L2
// while every CTA that needs them streams them (a row-major walk over all
// column blocks streams the whole of B once per wave of tiles).
constexpr int kGroupM = 16;

__device__ __forceinline__ void tile_coords(int tile, int tiles_m, int tiles_n, int& mb, int& nb) {
  const int per_group = kGroupM * tiles_n;
  const int g = tile / per_group, r = tile - g * per_group;
  const int m0 = g * kGroupM;
  const int gm = min(kGroupM, tiles_m - m0);
  nb = r / gm;
  mb = m0 + (r - nb * gm);
}

// Waits with one lane and broadcasts the result to the warp.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                          uint32_t* status, uint32_t where, int lane) {
  int ok = 1;
  if (lane == 0) ok = mbar_wait(bar, parity, abort_flag, status, where);
  return __shfl_sync(0xFFFFFFFFu, ok, 0) != 0;
}

// EPI epilogue, one thread: 32 columns from `col` of output row `row`, v = the
// scaled FP32 products, which become act(v + bias) + residual and are stored.
// Returns the scale byte of v + bias, a whole block of the checkpoint.
template <int ACT>
__device__ __forceinline__ void act32(float* v) {
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    const float2 f = fp4dev::unpair(fp4dev::act_value2<ACT>(fp4dev::pair(v[i], v[i + 1])));
    v[i] = f.x;
    v[i + 1] = f.y;
  }
}

// 64 bytes of a residual row from column `col`: 32 BF16 or 16 FP32 values.
__device__ __forceinline__ void load_residual(const StParams& p, int64_t row, int64_t col, uint32_t* r) {
  const char* src = static_cast<const char*>(p.res) + (row * p.ldr + col) * (p.res_f32 ? 4 : 2);
  if (p.res_wide) {
    ld_global_v8(src, r);
    ld_global_v8(src + 32, r + 8);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 x = reinterpret_cast<const uint4*>(src)[i];
      r[4 * i] = x.x; r[4 * i + 1] = x.y; r[4 * i + 2] = x.z; r[4 * i + 3] = x.w;
    }
  }
}

// `bias`: its 32 values in shared memory; `r`: the residual's first 64 bytes,
// replaced by those 32 columns on when `more`.
__device__ __forceinline__ uint32_t epilogue32(const StParams& p, int64_t row, int64_t col, float* v,
                                               const float* bias, uint32_t* r, bool more,
                                               bool wide_st, float& amax) {
  uint32_t byte = 0;
  if (p.bias != nullptr) {
#pragma unroll
    for (int i = 0; i < 32; i += 4) {        // __fadd_rn: no FMA, z is fp4_gemm's P + bias
      const float4 b = *reinterpret_cast<const float4*>(bias + i);
      v[i] = __fadd_rn(v[i], b.x);
      v[i + 1] = __fadd_rn(v[i + 1], b.y);
      v[i + 2] = __fadd_rn(v[i + 2], b.z);
      v[i + 3] = __fadd_rn(v[i + 3], b.w);
    }
  }
  if (p.z_codes != nullptr) {
    float m = fabsf(v[31]);
#pragma unroll
    for (int i = 0; i < 30; i += 2) m = fp4dev::max_abs3(m, v[i], v[i + 1]);
    m = fp4dev::max_abs3(m, v[30], v[30]);
    byte = fp4dev::ckpt_scale_byte(fp4dev::abs_bits(m));
    const float inv = fp4dev::ckpt_inv_scale(byte);
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w[i] = fp4dev::e4m3x4_rn(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv, v[4 * i + 3] * inv);
    uint8_t* d = p.z_codes + row * p.N + col;                             // a multiple of 32 from the start
    if (p.z_wide) {
      st_global_v8(d, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
    } else {
      reinterpret_cast<uint4*>(d)[0] = make_uint4(w[0], w[1], w[2], w[3]);
      reinterpret_cast<uint4*>(d)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
  switch (p.act) {
    case FQT_ACT_RELU: act32<FQT_ACT_RELU>(v); break;
    case FQT_ACT_GELU: act32<FQT_ACT_GELU>(v); break;
    case FQT_ACT_GELU_TANH: act32<FQT_ACT_GELU_TANH>(v); break;
    case FQT_ACT_SILU: act32<FQT_ACT_SILU>(v); break;
    default: break;
  }
  if (p.res != nullptr) {
    if (p.res_f32) {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] += __uint_as_float(r[i]);
      load_residual(p, row, col + 16, r);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[16 + i] += __uint_as_float(r[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        v[2 * i] += __uint_as_float(r[i] << 16);
        v[2 * i + 1] += __uint_as_float(r[i] & 0xFFFF0000u);
      }
    }
    if (more) load_residual(p, row, col + 32, r);
  }
  if (p.c_amax != nullptr) {
#pragma unroll
    for (int i = 0; i < 32; i += 2) amax = fp4dev::max_abs3(amax, v[i], v[i + 1]);   // NaN stays
  }
  if (p.out_mode == 1) {
    float* d = static_cast<float*>(p.c) + row * p.ldc + col;
#pragma unroll
    for (int i = 0; i < 32; i += 8) {
      if (wide_st)
        st_global_v8(d + i, __float_as_uint(v[i]), __float_as_uint(v[i + 1]), __float_as_uint(v[i + 2]),
                     __float_as_uint(v[i + 3]), __float_as_uint(v[i + 4]), __float_as_uint(v[i + 5]),
                     __float_as_uint(v[i + 6]), __float_as_uint(v[i + 7]));
      else
        fp4dev::store8(d, i, true, v + i);
    }
  } else {
    __nv_bfloat16* d = static_cast<__nv_bfloat16*>(p.c) + row * p.ldc + col;
#pragma unroll
    for (int i = 0; i < 32; i += 16) {
      const uint4 lo = fp4dev::pack_bf16x8(v + i), hi = fp4dev::pack_bf16x8(v + i + 8);
      if (wide_st) {
        st_global_v8(d + i, lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w);
      } else {
        reinterpret_cast<uint4*>(d + i)[0] = lo;
        reinterpret_cast<uint4*>(d + i)[1] = hi;
      }
    }
  }
  return byte;
}

// Registers of an EPI kernel's warpgroups (four warps each): the epilogue's two
// hold a row's 128 accumulator columns at once, so that the accumulator is free
// for the next tile's MMAs before any of the epilogue's arithmetic, which the K
// loop then hides (32768 x 11008 x 4096 with GELU and checkpoint: 1378 us with the
// accumulator held through it, 1113 without, 960-990 with the steps below).  What
// remains over fp4_gemm's time is 6 % more cycles, mostly the checkpoint's stores,
// and the power limit that long runs reach: 979 us at 1447 MHz against 860 at 1545;
// single launches take 87 against 79 us (8192 x 4096 x 4096).  The sum is
// what the 512 threads are launched with, 4 x 128.
constexpr int kEpiRegs = 192, kOtherRegs = 64;
static_assert(2 * kEpiRegs + 2 * kOtherRegs <= 4 * 128, "register split");
template <bool EPI>
__device__ __forceinline__ void fewer_registers() {
  if constexpr (EPI) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
}

template <bool NV, bool EPI, int BN>
__global__ void __launch_bounds__(NUM_THREADS, 1)
fp4_gemm_sfst_kernel(const __grid_constant__ CUtensorMap tmap_a,
                     const __grid_constant__ CUtensorMap tmap_b, const StParams p) {
  using TS = Tile<BN>;
  constexpr int STAGES = TS::STAGES, ATOM_ROWS = TS::ATOM_ROWS;
  constexpr int A_BYTES = TS::A_BYTES, B_BYTES = TS::B_BYTES, SFA_BYTES = TS::SFA_BYTES,
                SFB_BYTES = TS::SFB_BYTES, STAGE_BYTES = TS::STAGE_BYTES;
  constexpr int TMEM_SF_BASE = TS::TMEM_SF_BASE, TMEM_SF_STAGE = TS::TMEM_SF_STAGE;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  auto sA = [&](int s) { return base + s * A_BYTES; };
  auto sB = [&](int s) { return base + STAGES * A_BYTES + s * B_BYTES; };
  auto sSFA = [&](int s) { return base + STAGES * (A_BYTES + B_BYTES) + s * SFA_BYTES; };
  auto sSFB = [&](int s) {
    return base + STAGES * (A_BYTES + B_BYTES + SFA_BYTES) + s * SFB_BYTES;
  };
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + STAGES * STAGE_BYTES);
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
  auto sf_bar = [&](int s) { return bar0 + 8u * (2 * STAGES + s); };
  auto atoms_bar = [&](int s) { return bar0 + 8u * (3 * STAGES + s); };
  const uint32_t acc_full = bar0 + 8u * (4 * STAGES);
  const uint32_t acc_empty = bar0 + 8u * (4 * STAGES + 1);
  const uint32_t drain_bar = bar0 + 8u * (4 * STAGES + 2);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 4 * STAGES + 3);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles_m = p.M / BM, tiles_n = (p.N + BN - 1) / BN;
  const int num_tiles = tiles_m * tiles_n;
  const int k_blocks = (p.K + BK - 1) / BK;
  const int apr = p.atoms_per_rowblk;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
      mbar_init(sf_bar(s), 4);
      mbar_init(atoms_bar(s), 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, EPI_WARPS);
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == MMA_WARP) tmem_alloc(smem_u32(tmem_holder), TMEM_COLS);
  if constexpr (EPI) wait_previous_launch();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  // one branch per warpgroup: a register split is the whole warpgroup's
  if (warp < SF_WARP0 + 4) {
    fewer_registers<EPI>();
    // ------------------------------------------------------------ scale stagers
    // Tensor-memory scale layout the MMA reads (what a 32x128b.warpx4 copy of
    // a 512-byte atom produces): every lane quadrant holds the whole atom,
    // lane 32q + r holds the atom's 16-byte row r in 4 consecutive columns.
    const int q = warp - SF_WARP0;
    const uint32_t lane_base = (uint32_t)(q * 32) << 16;
    uint32_t it = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < num_tiles && ok; tile += gridDim.x) {
      for (int kb = 0; kb < k_blocks; ++kb, ++it) {
        const int s = it % STAGES;
        const uint32_t ph = (it / STAGES) & 1u;
        if (!warp_wait(atoms_bar(s), ph, abort_flag, p.status, 0x3300 + s, lane)) { ok = false; break; }
        uint32_t va[16], vb[16 * ATOM_ROWS];
        const uint8_t* fa = sSFA(s) + lane * 16;
        const uint8_t* fb = sSFB(s) + lane * 16;
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          const uint4 x = *reinterpret_cast<const uint4*>(fa + a * 512);
          va[4 * a] = x.x; va[4 * a + 1] = x.y; va[4 * a + 2] = x.z; va[4 * a + 3] = x.w;
          uint32_t* const w = vb + 4 * ATOM_ROWS * a;
          const uint4 y0 = *reinterpret_cast<const uint4*>(fb + a * 512);
          w[0] = y0.x; w[1] = y0.y; w[2] = y0.z; w[3] = y0.w;
          if constexpr (ATOM_ROWS == 2) {
            const uint4 y1 = *reinterpret_cast<const uint4*>(fb + 2048 + a * 512);
            w[4] = y1.x; w[5] = y1.y; w[6] = y1.z; w[7] = y1.w;
          }
        }
        const uint32_t t_sfa = tmem_base + TMEM_SF_BASE + s * TMEM_SF_STAGE;
        tmem_st_x16(lane_base + t_sfa, va);
        if constexpr (ATOM_ROWS == 2) tmem_st_x32(lane_base + t_sfa + 16, vb);
        else tmem_st_x16(lane_base + t_sfa + 16, vb);
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sf_bar(s));
      }
    }
  } else if (warp < EPI_WARP0 + EPI_WARPS) {
    if constexpr (EPI) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
    // ------------------------------------------------------------ epilogue
    const float scale = p.alpha * (*p.a_sdec) * (*p.b_sdec);
    const int esize = p.out_mode == 1 ? 4 : 2;
    const bool wide_st = (reinterpret_cast<uintptr_t>(p.c) % 32) == 0 && (p.ldc * esize) % 32 == 0;
    float q_senc = 1.0f;
    if (p.out_mode == 2) {
      // encode with the supplied tensor amax (the two-level NVFP4 scale of the
      // quantizers); record it and the decode scale with the codes
      const float A = *p.q_amax_in;
      float q_sdec;
      fp4dev::nvfp4_global_scales(A, q_senc, q_sdec);
      if (blockIdx.x == 0 && threadIdx.x == EPI_WARP0 * 32) {
        if (!(A <= FLT_MAX)) set_status(p.status, FP4_ERR_NONFINITE, 5);
        *p.q_s_dec = q_sdec;
        if (p.q_amax_out != p.q_amax_in) *p.q_amax_out = A;
      }
    }
    float amax = 0.0f;
    uint32_t tile_iter = 0;
    const int quad = warp & 3, half = (warp - EPI_WARP0) >> 2;
    const int c_begin = half * (BN / 2);
    // EPI: the bias values of this warp's columns, as FP32
    float* const bias_s = reinterpret_cast<float*>(base + STAGES * STAGE_BYTES + 256) + (warp - EPI_WARP0) * (BN / 2);
    for (int tile = blockIdx.x; tile < num_tiles; tile += gridDim.x, ++tile_iter) {
      int mb, nb;
      tile_coords(tile, tiles_m, tiles_n, mb, nb);
      const int64_t row = (int64_t)mb * BM + quad * 32 + lane;
      const int ncols = min(BN / 2, p.N - nb * BN - c_begin);
      const int64_t col = (int64_t)nb * BN + c_begin;
      uint32_t res[16];
      if constexpr (EPI) {
        // what the tile needs besides its accumulator, before the wait for that
        if (ncols > 0 && p.bias != nullptr) {
          __syncwarp();                     // the last tile's values have been read
          if (lane < BN / 8) {
            float4 b;
            const int64_t at = col + 4 * lane;
            if (p.bias_f32) {
              b = *reinterpret_cast<const float4*>(static_cast<const float*>(p.bias) + at);
            } else {
              const uint2 x = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.bias) + at);
              b = make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xFFFF0000u),
                              __uint_as_float(x.y << 16), __uint_as_float(x.y & 0xFFFF0000u));
            }
            reinterpret_cast<float4*>(bias_s)[lane] = b;
          }
          __syncwarp();
        }
        if (ncols > 0 && p.res != nullptr) {
          load_residual(p, row, col, res);
          // the rest of its row towards L2
          const char* src = static_cast<const char*>(p.res) + (row * p.ldr + col) * (p.res_f32 ? 4 : 2);
          const int bytes = BN / 2 * (p.res_f32 ? 4 : 2);
          for (int o = 128; o < bytes; o += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(src + o));
        }
      }
      if (!warp_wait(acc_full, tile_iter & 1u, abort_flag, p.status, 0x3700 + warp, lane)) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)c_begin;
      if constexpr (EPI) {
        // The whole row half leaves tensor memory first; then blocks of 32
        // columns, two to an iteration: of one, two and four that measured
        // fastest (fewer moves of the rest than one, less code than four).
        constexpr int COLS = BN / 2, BLOCKS = COLS / 32;
        uint32_t scales4 = 0;
        float v[COLS];
        {
          uint32_t r[COLS];
#pragma unroll
          for (int h = 0; h < BLOCKS; ++h) tmem_ld32_nowait(taddr + 32 * h, r + 32 * h);
          asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(acc_empty);
          if (tile + (int)gridDim.x >= num_tiles) allow_next_launch();   // only this epilogue is left
#pragma unroll
          for (int i = 0; i < COLS; ++i) v[i] = __uint_as_float(r[i]);
        }
        if (ncols > 0) {
#pragma unroll 1
          for (int h = 0; h < BLOCKS; h += 2) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
              for (int i = 0; i < 32; ++i) v[32 * k + i] = __fmul_rn(v[32 * k + i], scale);
              scales4 |= epilogue32(p, row, col + 32 * (h + k), v + 32 * k, bias_s + 32 * (h + k), res,
                                    h + k < BLOCKS - 1, wide_st, amax) << (8 * (h + k));
            }
#pragma unroll
            for (int i = 0; i < COLS - 64; ++i) v[i] = v[i + 64];
          }
        }
        if (p.z_codes != nullptr && ncols > 0) {
          uint8_t* const sc = p.z_scales + ((row * p.N + col) >> 5);
          if constexpr (BLOCKS == 4) *reinterpret_cast<uint32_t*>(sc) = scales4;
          else *reinterpret_cast<uint16_t*>(sc) = (uint16_t)scales4;
          // byte 255: Inf or NaN in one of the blocks
          if (__vcmpeq4(scales4, 0xFFFFFFFFu) != 0) set_status(p.status, FP4_ERR_NONFINITE, 8);
        }
      } else if (p.out_mode == 0) {
        // drain 128 columns in two 64-column loads, packing to BF16 as they
        // arrive (64 registers); the accumulator is released as soon as the
        // second load has landed, before that half is packed, so the next
        // tile's MMAs wait for two TMEM round trips and one packing only
        uint32_t pk[64];
        {
          uint32_t r2[64];
          tmem_ld32_nowait(taddr, r2);
          tmem_ld32_nowait(taddr + 32, r2 + 32);
          asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
          for (int h = 0; h < 32; ++h) {
            const float a0 = __uint_as_float(r2[2 * h]) * scale;
            const float a1 = __uint_as_float(r2[2 * h + 1]) * scale;
            amax = fmaxf(amax, fmaxf(fabsf(a0), fabsf(a1)));
            __nv_bfloat162 b2 = __floats2bfloat162_rn(a0, a1);
            memcpy(&pk[h], &b2, 4);
          }
        }
        {
          uint32_t r2[64];
          tmem_ld32_nowait(taddr + 64, r2);
          tmem_ld32_nowait(taddr + 96, r2 + 32);
          asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(acc_empty);
#pragma unroll
          for (int h = 0; h < 32; ++h) {
            const float a0 = __uint_as_float(r2[2 * h]) * scale;
            const float a1 = __uint_as_float(r2[2 * h + 1]) * scale;
            amax = fmaxf(amax, fmaxf(fabsf(a0), fabsf(a1)));
            __nv_bfloat162 b2 = __floats2bfloat162_rn(a0, a1);
            memcpy(&pk[32 + h], &b2, 4);
          }
        }
        if (ncols > 0) {
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.c) + row * p.ldc + col;
          if (wide_st) {          // full 32-byte sectors
#pragma unroll
            for (int q = 0; q < 8; ++q)
              st_global_v8(dst + 16 * q, pk[8 * q], pk[8 * q + 1], pk[8 * q + 2], pk[8 * q + 3],
                           pk[8 * q + 4], pk[8 * q + 5], pk[8 * q + 6], pk[8 * q + 7]);
          } else {
            uint4* d4 = reinterpret_cast<uint4*>(dst);
#pragma unroll
            for (int q = 0; q < 16; ++q) d4[q] = make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]);
          }
        }
      } else if (p.out_mode == 2) {
        // NVFP4 1x16, round to nearest: each 16-column block of the FP32
        // result gets its E4M3 scale from its own max, then 16 E2M1 codes;
        // two halves of 64 columns, the accumulator released after the second
        const int64_t S = p.N >> 4, S4 = (S + 3) & ~3LL;
#pragma unroll 1
        for (int h2 = 0; h2 < 2; ++h2) {
          uint32_t v[64];
          tmem_ld32_nowait(taddr + 64 * h2, v);
          tmem_ld32_nowait(taddr + 64 * h2 + 32, v + 32);
          asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
          if (h2 == 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acc_empty);
          }
          if (ncols > 0) {
            uint32_t cw[8];
            uint32_t sfw = 0;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              float o[16];
              float bmax = 0.0f;
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                o[e] = __uint_as_float(v[16 * b + e]) * scale;
                bmax = fmaxf(bmax, fabsf(o[e]));
              }
              amax = fmaxf(amax, bmax);
              const int64_t cb = col + 64 * h2 + 16 * b;   // first column of the block
              if (p.c != nullptr) {
                // the FP32 result also leaves as BF16 (for a consumer that
                // still needs it, e.g. the transposed quantization)
                uint32_t pk[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  __nv_bfloat162 b2 = __floats2bfloat162_rn(o[2 * e], o[2 * e + 1]);
                  memcpy(&pk[e], &b2, 4);
                }
                __nv_bfloat16* bd = static_cast<__nv_bfloat16*>(p.c) + row * p.ldc + cb;
                if (wide_st) {
                  st_global_v8(bd, pk[0], pk[1], pk[2], pk[3], pk[4], pk[5], pk[6], pk[7]);
                } else {
                  reinterpret_cast<uint4*>(bd)[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                  reinterpret_cast<uint4*>(bd)[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
                }
              }
              const uint32_t sf = fp4dev::e4m3_rn_sat(fp4dev::div6_for_scale(__fmul_rn(bmax, q_senc)));
              const float inv = (sf == 0u || sf == 127u)
                                    ? 0.0f : fminf(__fdiv_rn(q_senc, fp4dev::e4m3_value(sf)), FLT_MAX);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __fmul_rn(o[e], inv);
              if (p.q_sr) {
                // draws of elements row * N + cb .. + 15: two Philox blocks
                const uint64_t i0 = (uint64_t)row * (uint64_t)p.N + (uint64_t)cb;
                cw[2 * b] = fp4dev::e2m1x8_sr(o, fp4dev::philox_keyed(i0 >> 3, p.q_stream, p.q_keys));
                cw[2 * b + 1] = fp4dev::e2m1x8_sr(o + 8, fp4dev::philox_keyed((i0 >> 3) + 1, p.q_stream, p.q_keys));
              } else {
                cw[2 * b] = fp4dev::e2m1x8_rn(o);
                cw[2 * b + 1] = fp4dev::e2m1x8_rn(o + 8);
              }
              sfw |= sf << (8 * b);
            }
            const int64_t c0 = col + 64 * h2;              // first column of these 4 blocks
            uint4* cd = reinterpret_cast<uint4*>(p.q_codes + row * (p.N >> 1) + (c0 >> 1));
            cd[0] = make_uint4(cw[0], cw[1], cw[2], cw[3]);
            cd[1] = make_uint4(cw[4], cw[5], cw[6], cw[7]);
            const int64_t sb0 = c0 >> 4;                   // a multiple of 4
            if (p.q_scales != nullptr) *reinterpret_cast<uint32_t*>(p.q_scales + row * S + sb0) = sfw;
            if (p.q_scales_mma != nullptr)
              *reinterpret_cast<uint32_t*>(p.q_scales_mma + fp4dev::mma_sf_offset(row, sb0, S4)) = sfw;
          }
        }
      } else {
        // FP32: two halves of 64 columns; the accumulator is released after
        // the second half is in registers
        float* dst = static_cast<float*>(p.c) + row * p.ldc + col;
#pragma unroll 1
        for (int h2 = 0; h2 < 2; ++h2) {
          uint32_t v[64];
          tmem_ld32_nowait(taddr + 64 * h2, v);
          tmem_ld32_nowait(taddr + 64 * h2 + 32, v + 32);
          asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
          if (h2 == 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acc_empty);
          }
          if (ncols > 0) {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              float o[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                o[e] = __uint_as_float(v[8 * q + e]) * scale;
                amax = fmaxf(amax, fabsf(o[e]));
              }
              float* d = dst + 64 * h2 + 8 * q;
              if (wide_st) {
                st_global_v8(d, __float_as_uint(o[0]), __float_as_uint(o[1]), __float_as_uint(o[2]),
                             __float_as_uint(o[3]), __float_as_uint(o[4]), __float_as_uint(o[5]),
                             __float_as_uint(o[6]), __float_as_uint(o[7]));
              } else {
                reinterpret_cast<float4*>(d)[0] = make_float4(o[0], o[1], o[2], o[3]);
                reinterpret_cast<float4*>(d)[1] = make_float4(o[4], o[5], o[6], o[7]);
              }
            }
          }
        }
      }
    }
    if (p.c_amax != nullptr) {
      if constexpr (EPI) {
        // as bits without the sign: they order by magnitude, NaN on top
        const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, fp4dev::abs_bits(amax));
        if (lane == 0) atomicMax(reinterpret_cast<unsigned int*>(p.c_amax), top);
      } else {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
        if (lane == 0) atomicMax(reinterpret_cast<unsigned int*>(p.c_amax), __float_as_uint(amax));
      }
    }
  } else {
    fewer_registers<EPI>();
    if (warp == PRODUCER_WARP) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_a)) : "memory");
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_b)) : "memory");
      uint32_t it = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < num_tiles && ok; tile += gridDim.x) {
        int mb, nb;
        tile_coords(tile, tiles_m, tiles_n, mb, nb);
        const bool b_hi = ATOM_ROWS == 2 && (nb * 2 + 1) * 128 < p.N;
        for (int kb = 0; kb < k_blocks; ++kb, ++it) {
          const int s = it % STAGES;
          const uint32_t ph = (it / STAGES) & 1u;
          if (!mbar_wait(empty_bar(s), ph ^ 1u, abort_flag, p.status, 0x3100 + s)) { ok = false; break; }
          const int n_atoms = NV ? min(4, apr - kb * 4) : min(2, apr - kb * 2);
          const uint32_t atom_bytes = (uint32_t)n_atoms * 512u;
          // scale atoms first, on their own barrier: the stagers move them into
          // tensor memory while the operand tiles are still in flight
          mbar_arrive_expect_tx(atoms_bar(s), atom_bytes * (b_hi ? 3u : 2u));
          const int atom0 = kb * (NV ? 4 : 2);
          bulk_load(smem_u32(sSFA(s)), p.a_sf + ((size_t)mb * apr + atom0) * 512, atom_bytes,
                    atoms_bar(s));
          bulk_load(smem_u32(sSFB(s)), p.b_sf + ((size_t)(ATOM_ROWS * nb) * apr + atom0) * 512, atom_bytes,
                    atoms_bar(s));
          if (b_hi)
            bulk_load(smem_u32(sSFB(s) + 4 * 512), p.b_sf + ((size_t)(2 * nb + 1) * apr + atom0) * 512,
                      atom_bytes, atoms_bar(s));
          mbar_arrive_expect_tx(full_bar(s), A_BYTES + B_BYTES);
          tma_load_2d(smem_u32(sA(s)), &tmap_a, full_bar(s), kb * (BK / 2), mb * BM);
          tma_load_2d(smem_u32(sB(s)), &tmap_b, full_bar(s), kb * (BK / 2), nb * BN);
        }
      }
      if (it > 0) {
        const uint32_t first = it > (uint32_t)STAGES ? it - STAGES : 0;
        for (uint32_t j = first; j < it; ++j) {
          volatile int no_abort = 0;
          mbar_wait(atoms_bar(j % STAGES), (j / STAGES) & 1u, &no_abort, p.status, 0x3200 + j % STAGES);
          mbar_wait(full_bar(j % STAGES), (j / STAGES) & 1u, &no_abort, p.status, 0x3200 + j % STAGES);
        }
      }
    }
    } else if (warp == MMA_WARP) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      uint32_t it = 0, tile_iter = 0;
      bool ok = true, issued = false;
      for (int tile = blockIdx.x; tile < num_tiles && ok; tile += gridDim.x, ++tile_iter) {
        if (!mbar_wait(acc_empty, (tile_iter & 1u) ^ 1u, abort_flag, p.status, 0x3400)) { ok = false; break; }
        tc_fence_after();
        for (int kb = 0; kb < k_blocks; ++kb, ++it) {
          const int s = it % STAGES;
          const uint32_t ph = (it / STAGES) & 1u;
          if (!mbar_wait(sf_bar(s), ph, abort_flag, p.status, 0x3500 + s)) { ok = false; break; }
          if (!mbar_wait(full_bar(s), ph, abort_flag, p.status, 0x3580 + s)) { ok = false; break; }
          tc_fence_after();
          const int n_mma = min(BK / MMA_K, (p.K - kb * BK) / MMA_K);
          const uint32_t t_sfa = tmem_base + TMEM_SF_BASE + s * TMEM_SF_STAGE;
          const uint32_t t_sfb = t_sfa + 16;
          const uint32_t a_base = smem_u32(sA(s)), b_base = smem_u32(sB(s));
          auto step = [&](int kk) {
            uint32_t sfa_addr, sfb_addr, idesc;
            if (NV) {
              sfa_addr = t_sfa + 4 * kk;
              sfb_addr = t_sfb + 4 * ATOM_ROWS * kk;
              idesc = make_idesc(BN, BM, 0u, 0u, 0u);
            } else {
              const uint32_t byte = (uint32_t)(kk & 1) * 2u;
              sfa_addr = (t_sfa + 4 * (kk >> 1)) | (byte << 30);
              sfb_addr = (t_sfb + 4 * ATOM_ROWS * (kk >> 1)) | (byte << 30);
              idesc = make_idesc(BN, BM, 1u, byte, byte);
            }
            tc_mma<NV>(tmem_base, smem_desc(a_base + kk * (MMA_K / 2), 16, 1024, 2),
                       smem_desc(b_base + kk * (MMA_K / 2), 16, 1024, 2), idesc, sfa_addr,
                       sfb_addr, (kb > 0 || kk > 0) ? 1u : 0u);
          };
          if (n_mma == BK / MMA_K) {
#pragma unroll
            for (int kk = 0; kk < BK / MMA_K; ++kk) step(kk);
          } else {
            for (int kk = 0; kk < n_mma; ++kk) step(kk);
          }
          issued = true;
          tc_commit(empty_bar(s));
        }
        if (!ok) break;
        tc_commit(acc_full);
      }
      if (issued) {
        tc_commit(drain_bar);
        volatile int no_abort = 0;
        mbar_wait(drain_bar, 0, &no_abort, p.status, 0x3600);
      }
    }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* q = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &q, 12000, cudaEnableDefault,
                                         &r) == cudaSuccess &&
        r == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(q);
  });
  return fn;
}

bool codes_map(CUtensorMap* m, const uint8_t* codes, int64_t rows, int64_t K, uint32_t box_rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)(K / 2), (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)(K / 2)};
  cuuint32_t box[2] = {128u, box_rows};
  cuuint32_t es[2] = {1u, 1u};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(codes), dims, strides, box,
             es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// Tiles of 128 columns instead of 256 while those are at most half the SMs: twice
// the SMs then share the epilogue (128 x 4096 x 4096 with bias, GELU and an FP32
// output, 16 wide tiles: 13.8 us against 17.6; 512 x 4096 x 4096, 64: 13.8 against
// 16.3).  Beyond, the narrow tiles need a second wave (640 x 4096 x 4096, 80: 20.3
// against 16.4).  The K loop takes 0.42 us a step of 256 with either.
static bool narrow_tiles(int64_t tiles_wide) { return tiles_wide * 2 <= sm_count(); }

fp4_status gemm_launch(const GemmArgs& g, cudaStream_t s) {
  const bool nv = g.fmt == FP4_NVFP4;
  const bool narrow = g.epi && narrow_tiles((g.M / BM) * ((g.N + 255) / 256));
  const int BN = narrow ? 128 : 256;
  CUtensorMap ta, tb;
  if (!codes_map(&ta, g.a_codes, g.M, g.K, BM)) return FP4_ERR_CUDA;
  if (!codes_map(&tb, g.b_codes, g.N, g.K, BN)) return FP4_ERR_CUDA;
  StParams p;
  p.a_sf = g.a_sf; p.b_sf = g.b_sf; p.a_sdec = g.a_sdec; p.b_sdec = g.b_sdec;
  p.M = (int)g.M; p.N = (int)g.N; p.K = (int)g.K;
  p.atoms_per_rowblk = nv ? (int)(g.K / 64) : (int)((((g.K / 32) + 3) / 4 * 4) / 4);
  p.alpha = g.alpha; p.c = g.c; p.ldc = g.ldc; p.out_mode = g.out_mode;
  p.q_codes = g.q_codes; p.q_scales = g.q_scales; p.q_scales_mma = g.q_scales_mma;
  p.q_amax_in = g.q_amax_in; p.q_amax_out = g.q_amax_out; p.q_s_dec = g.q_s_dec;
  p.q_sr = g.q_sr; p.q_stream = g.q_stream; p.q_keys = fp4dev::philox_keys(g.q_seed);
  p.act = g.act; p.bias = g.bias; p.bias_f32 = g.bias_f32;
  p.res = g.res; p.ldr = g.ldr; p.res_f32 = g.res_f32;
  p.res_wide = ptr_aligned(g.res, 32) && (g.ldr * (g.res_f32 ? 4 : 2)) % 32 == 0;
  p.z_codes = g.z_codes; p.z_scales = g.z_scales; p.z_wide = ptr_aligned(g.z_codes, 32);
  p.c_amax = g.c_amax; p.status = g.status;
  const int tiles = (int)(g.M / BM) * (int)((g.N + BN - 1) / BN);
  const int grid = tiles < sm_count() ? tiles : sm_count();
  if (g.c_amax != nullptr && cudaMemsetAsync(g.c_amax, 0, sizeof(float), s) != cudaSuccess)
    return FP4_ERR_CUDA;
  const auto kernel = narrow ? (nv ? fp4_gemm_sfst_kernel<true, true, 128> : fp4_gemm_sfst_kernel<false, true, 128>)
                      : g.epi ? (nv ? fp4_gemm_sfst_kernel<true, true, 256> : fp4_gemm_sfst_kernel<false, true, 256>)
                              : (nv ? fp4_gemm_sfst_kernel<true, false, 256> : fp4_gemm_sfst_kernel<false, false, 256>);
  const int smem = narrow ? Tile<128>::EPI_SMEM_BYTES
                   : g.epi ? Tile<256>::EPI_SMEM_BYTES : Tile<256>::SMEM_BYTES;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return FP4_ERR_CUDA;
  if (g.epi)
    return launch_overlapped(kernel, dim3((unsigned)grid), NUM_THREADS, (size_t)smem, s, ta, tb, p) == cudaSuccess
               ? FP4_OK : FP4_ERR_CUDA;
  kernel<<<grid, NUM_THREADS, smem, s>>>(ta, tb, p);
  count_launches(1);
  return cudaGetLastError() == cudaSuccess ? FP4_OK : FP4_ERR_CUDA;
}

}  // namespace fp4impl
