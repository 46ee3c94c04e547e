// Projection in 8-bit floating point with a scale for each block of 128:
//
//   y[m, n] = sum_b xs[m, b] Ws[n / 128, b] (sum_{k in block b} xq[m, k] Wq[n, k]) + bias[n]
//
// xq [M, K], Wq [N, K] e4m3; xs [M, ceil(K/128)], Ws [ceil(N/128), ceil(K/128)]
// fp32.  The products of a block accumulate in fp32 on the tensor cores; the
// scaled sum over blocks is held in fp32 registers and rounded to bf16 once.
//
// A scale changes every 128 of K, so a tile's accumulator cannot stay in tensor
// memory over the whole sum: each 128-deep block gets a fresh TMEM buffer
// (four tcgen05.mma of K = 32), which the epilogue warps read, scale and add to
// the registers that hold the tile, while the MMAs of the next blocks run into
// the other buffers:
//   warp 0    TMA producer (one lane) and TMEM owner,
//   warp 1    MMA issuer (one lane),
//   warps 2-9 promotion and epilogue, two per 32-lane TMEM quarter, each half
//             of the tile's columns (one row per thread).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "lm.h"
#include "ptx.cuh"
#include "tc.cuh"

namespace srnn {
namespace {

constexpr int FBM = 128, FBK = 128;
constexpr int F_NEPI = 8;
constexpr int F_THREADS = 32 * (2 + F_NEPI);

template <int BN>
struct F8Cfg {
  static constexpr uint32_t TILE_A = FBM * FBK, TILE_B = BN * FBK;
  static constexpr uint32_t STAGE = TILE_A + TILE_B;
  static constexpr int NSTG = BN == 256 ? 4 : 6;
  static constexpr int NACC = 512 / BN;                 // TMEM buffers
  static constexpr int WCOLS = BN / 2;                  // columns of an epilogue warp
  static constexpr uint32_t OUT = F_NEPI * 32 * 128;    // 32 rows x 64 bf16 per warp
  static constexpr uint32_t SMEM = NSTG * STAGE + OUT + 1024 + (2 * NSTG + 2 * NACC) * 8 + 16;
};

struct F8Args {
  int M, N, tiles_m, tiles_n, nkb;
  const float* xs;
  const float* Ws;
  const float* bias;
  int* status;
  unsigned long long timeout_ns;
};

// Instruction descriptor, kind::f8f6f4: fp32 accumulator, e4m3 A and B, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ bool wait_f8(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                        int* status, unsigned long long limit_ns) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > limit_ns) {
      *abort_flag = 1;
      atomicOr(status, kStatusTimeout);
      return false;
    }
  }
}

template <int BN>
__global__ void __launch_bounds__(F_THREADS, 1)
    proj_fp8_kernel(const __grid_constant__ CUtensorMap mA, const __grid_constant__ CUtensorMap mB,
                    const __grid_constant__ CUtensorMap mC, const F8Args g) {
  using C = F8Cfg<BN>;
  constexpr int NSTG = C::NSTG, NACC = C::NACC, WC = C::WCOLS;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ int abort_flag_s, issued_s, consumed_s;
  volatile int* abort_flag = &abort_flag_s;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t ring = (raw + 1023u) & ~1023u;
  const uint32_t out_stage = ring + NSTG * C::STAGE;
  const uint32_t bar_full = out_stage + C::OUT, bar_empty = bar_full + 8 * NSTG;
  const uint32_t bar_tfull = bar_empty + 8 * NSTG, bar_tempty = bar_tfull + 8 * NACC;
  const uint32_t tslot = bar_tempty + 8 * NACC;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ntiles = g.tiles_m * g.tiles_n;
  const unsigned long long tlim = g.timeout_ns;

  if (threadIdx.x == 32) {
    for (int s = 0; s < NSTG; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      mbar_init(bar_empty + 8 * s, 1);
    }
    for (int a = 0; a < NACC; ++a) {
      mbar_init(bar_tfull + 8 * a, 1);
      mbar_init(bar_tempty + 8 * a, F_NEPI);
    }
    abort_flag_s = 0;
    issued_s = 0;
    consumed_s = 0;
    fence_mbar_init();
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 0) {
    tmem_alloc(tslot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  uint32_t tmem;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(tslot) : "memory");

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer --
    if (lane == 0) {
      tma_prefetch_map(&mA);
      tma_prefetch_map(&mB);
      int it = 0;
      bool stop = false;
      for (int u = blockIdx.x; u < ntiles && !stop; u += gridDim.x) {
        const int m0 = (u / g.tiles_n) * FBM, n0 = (u % g.tiles_n) * BN;
        for (int kb = 0; kb < g.nkb; ++kb, ++it) {
          const int s = it % NSTG, ph = it / NSTG;
          if (it >= NSTG &&
              !wait_f8(bar_empty + 8 * s, (ph - 1) & 1, abort_flag, g.status, tlim)) {
            stop = true;
            break;
          }
          const uint32_t sA = ring + s * C::STAGE, sB = sA + C::TILE_A, fb = bar_full + 8 * s;
          mbar_arrive_expect_tx(fb, C::STAGE);
          tma_load_2d(sA, &mA, kb * FBK, m0, fb);
          tma_load_2d(sB, &mB, kb * FBK, n0, fb);
        }
      }
      issued_s = it;
    }
  } else if (warp == 1) {
    // -------------------------------------------------------- MMA issuer --
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3_f32(FBM, BN);
      int it = 0;
      bool stop = false;
      for (int u = blockIdx.x; u < ntiles && !stop; u += gridDim.x) {
        for (int kb = 0; kb < g.nkb; ++kb, ++it) {
          const int s = it % NSTG, ph = it / NSTG, a = it % NACC, pa = it / NACC;
          if (!wait_f8(bar_full + 8 * s, ph & 1, abort_flag, g.status, tlim) ||
              (it >= NACC &&
               !wait_f8(bar_tempty + 8 * a, (pa - 1) & 1, abort_flag, g.status, tlim))) {
            stop = true;
            break;
          }
          tc_fence_after();
          const uint32_t sA = ring + s * C::STAGE, sB = sA + C::TILE_A;
          const uint32_t dacc = tmem + (uint32_t)(a * BN);
#pragma unroll
          for (int k4 = 0; k4 < FBK / 32; ++k4)  // 32 bytes along the K-major rows
            umma_f8(dacc, sdesc_sw128(sA + k4 * 32, 16, 1024), sdesc_sw128(sB + k4 * 32, 16, 1024),
                    idesc, k4 != 0 ? 1u : 0u);
          umma_commit(bar_empty + 8 * s);
          umma_commit(bar_tfull + 8 * a);
        }
      }
      consumed_s = it;
    }
  } else {
    // --------------------------------------------- promotion and epilogue --
    const int q = warp & 3;          // TMEM lane quarter this warp may access
    const int hc = (warp - 2) >> 2;  // column half of the tile
    const uint32_t stg = out_stage + (uint32_t)(warp - 2) * 4096;
    int it = 0;
    bool stop = false;
    for (int u = blockIdx.x; u < ntiles && !stop; u += gridDim.x) {
      const int m0 = (u / g.tiles_n) * FBM + q * 32, n0 = (u % g.tiles_n) * BN + hc * WC;
      const int row = m0 + lane < g.M ? m0 + lane : g.M - 1;
      const float* xs = g.xs + (long long)row * g.nkb;
      const int nb = (n0 < g.N ? n0 : g.N - 1) / 128;
      const float* ws = g.Ws + (long long)nb * g.nkb;
      float acc[WC];
#pragma unroll
      for (int j = 0; j < WC; ++j) acc[j] = 0.f;
      for (int kb = 0; kb < g.nkb; ++kb, ++it) {
        const int a = it % NACC, pa = it / NACC;
        const float sc = __ldg(xs + kb) * __ldg(ws + kb);
        if (!wait_f8(bar_tfull + 8 * a, pa & 1, abort_flag, g.status, tlim)) {
          stop = true;
          break;
        }
        tc_fence_after();
        const uint32_t t = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(a * BN + hc * WC);
#pragma unroll
        for (int c = 0; c < WC / 32; ++c) {
          uint32_t r[32];
          tmem_ld32(t + 32 * c, r);
          tmem_wait_ld();
          tmem_reg_fence(r);
#pragma unroll
          for (int j = 0; j < 32; ++j)
            acc[32 * c + j] = fmaf(sc, __uint_as_float(r[j]), acc[32 * c + j]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_tempty + 8 * a);
      }
      if (stop) break;
      // 64 columns at a time: bf16 (+ bias) into the warp's 128-byte swizzled box, TMA store
#pragma unroll
      for (int b = 0; b < WC / 64; ++b) {
        if (lane == 0) bulk_wait_read_all();
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          uint32_t pk[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int c = 64 * b + 8 * k + 2 * j, n = n0 + c;
            float b0 = 0.f, b1 = 0.f;
            if (g.bias) {
              b0 = n < g.N ? __ldg(g.bias + n) : 0.f;
              b1 = n + 1 < g.N ? __ldg(g.bias + n + 1) : 0.f;
            }
            pk[j] = pack_bf16x2(acc[c] + b0, acc[c + 1] + b1);
          }
          asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(
                           stg + (uint32_t)lane * 128 + (uint32_t)((k ^ (lane & 7)) * 16)),
                       "r"(pk[0]), "r"(pk[1]), "r"(pk[2]), "r"(pk[3])
                       : "memory");
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          if (n0 + 64 * b < g.N && m0 < g.M) tma_store_2d(&mC, n0 + 64 * b, m0, stg);
          bulk_commit();
        }
      }
    }
    if (lane == 0) bulk_wait_all();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    if (lane == 0 && *abort_flag) {
      // let TMA copies that were issued but never consumed land before exit
      for (int k = consumed_s; k < issued_s; ++k) {
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(bar_full + 8 * (k % NSTG), (k / NSTG) & 1))
          if (globaltimer_ns() - t0 > 10000000ull) break;
      }
    }
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn();  // tc_gemm.cu
int make_map(CUtensorMap* m, const void* ptr, uint64_t rows, uint64_t cols, uint64_t pitch,
             uint32_t bx, uint32_t by);

namespace {

// 8-bit row-major [rows, cols]; box of 128 columns x by rows, 128-byte swizzle
int make_map8(CUtensorMap* m, const void* ptr, uint64_t rows, uint64_t cols, uint32_t by) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return (int)cudaErrorNotSupported;
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {cols};
  const cuuint32_t box[2] = {FBK, by};
  const cuuint32_t es[2] = {1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides,
                        box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? 0 : (int)cudaErrorInvalidValue;
}

template <int BN>
int launch_bn(const ProjFp8Params& p, cudaStream_t s) {
  using C = F8Cfg<BN>;
  auto kern = proj_fp8_kernel<BN>;
  static int prepared[64][5];
  int e = prepare_launch(prepared, kern, C::SMEM, F_THREADS, 1);
  if (e != 0) return e;
  F8Args g{};
  g.M = p.M;
  g.N = p.N;
  g.tiles_m = (p.M + FBM - 1) / FBM;
  g.tiles_n = (p.N + BN - 1) / BN;
  g.nkb = (p.K + FBK - 1) / FBK;
  g.xs = p.xs;
  g.Ws = p.Ws;
  g.bias = p.bias;
  g.status = p.status;
  g.timeout_ns = p.timeout_ns;
  const long long tiles = (long long)g.tiles_m * g.tiles_n;
  // ring positions are counted in 32 bits
  if (tiles * g.nkb > 0x3fffffffLL) return (int)cudaErrorInvalidValue;
  CUtensorMap a, b, c;
  if ((e = make_map8(&a, p.xq, (uint64_t)p.M, (uint64_t)p.K, FBM))) return e;
  if ((e = make_map8(&b, p.Wq, (uint64_t)p.N, (uint64_t)p.K, BN))) return e;
  if ((e = make_map(&c, p.y, (uint64_t)p.M, (uint64_t)p.N, (uint64_t)p.N, 64, 32))) return e;
  const int cap = sm_count();
  const int grid = (int)(tiles < cap ? tiles : cap);
  kern<<<grid, F_THREADS, C::SMEM, s>>>(a, b, c, g);
  return (int)cudaGetLastError();
}

}  // namespace

int launch_proj_fp8(const ProjFp8Params& p, cudaStream_t s) { return launch_bn<128>(p, s); }

}  // namespace srnn
