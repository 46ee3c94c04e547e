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
// (four tcgen05.mma of K = 32), which the promotion warps read, scale and add to
// the registers that hold the tile, while the MMAs of the next blocks run into
// the other buffers:
//   warp 0       TMA producer (one lane) and TMEM owner,
//   warps 1, 2   MMA issuers (one lane each), every other block: what one of them spends on its
//                waits and commits (600 cycles a block) passes while the other's MMAs run,
//   warps 4-19   promotion and epilogue, a row and a quarter of the tile's columns per
//                thread; setmaxnreg moves registers to them from the first four.
// A 128 x 256 tile's MMAs read 96 bytes a clock of operands (a 128 x 128 one's the 128 that
// shared memory gives), and a block's 512 cycles of MMAs cover its promotion; the first
// blocks of a tile run during the epilogue of the one before.  The outputs leave by way of shared memory and
// TMA stores (stored straight from registers, an epilogue took 6,200 cycles).
//
// Measured at 16384 x 4096 x 1024: 84 us, 1.64 PFLOP/s (the bf16 matrix product's rate is 1.91), 23 us of bytes.
// What bounds it is the promotion: every fp32 sum of a block of 128 leaves TMEM, 32 columns a load, a wait and the multiply-adds
// one after the other (the tensor pipe is 34% busy), and a tile's epilogue between.
//
// A few rows (kFewRows at most) are bound by the weights' bytes instead: a kernel of its own reads each
// weight once, straight into the registers of mma.sync (16 x 2304 x 768: 2.3 us on the device, 4.7 with its call).
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

template <int BN>
struct F8Cfg {
  static constexpr uint32_t TILE_A = FBM * FBK, TILE_B = BN * FBK;
  static constexpr uint32_t STAGE = TILE_A + TILE_B;
  static constexpr int NSTG = BN == 256 ? 3 : 4;
  static constexpr int NACC = BN == 256 ? 2 : 4;  // TMEM buffers (at most NSTG, see `done`)
  static constexpr int WC = BN / 4;               // columns of a promotion warp
  static constexpr int NPW = 16;                  // promotion warps
  static constexpr int THREADS = 32 * (4 + NPW);
  static constexpr uint32_t STG = 32 * WC * 2;    // outputs on their way, per warp
  static constexpr uint32_t SMEM = NSTG * STAGE + NPW * STG + 1024 + (3 * NSTG + NACC) * 8 + 16;
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
__global__ void __launch_bounds__(F8Cfg<BN>::THREADS, 1)
    proj_fp8_kernel(const __grid_constant__ CUtensorMap mA, const __grid_constant__ CUtensorMap mB,
                    const __grid_constant__ CUtensorMap mC, const F8Args g) {
  using C = F8Cfg<BN>;
  constexpr int NSTG = C::NSTG, NACC = C::NACC, WC = C::WC;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ int abort_flag_s, issued_s;
  __shared__ __align__(8) uint64_t last_s;  // the last MMAs of both issuers done
  volatile int* abort_flag = &abort_flag_s;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t ring = (raw + 1023u) & ~1023u;
  const uint32_t out_stage = ring + NSTG * C::STAGE;
  // `full`: a block has landed; for each stage one barrier for the blocks of either issuer, so that each issuer
  // waits for every phase of its own (seeing every other one it would take the phase before for it).
  // `done`: a block's MMAs are complete, so its stage is free and its sums can be promoted
  const uint32_t bar_full = out_stage + C::NPW * C::STG, bar_done = bar_full + 16 * NSTG;
  const uint32_t bar_read = bar_done + 8 * NSTG, tslot = bar_read + 8 * NACC;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ntiles = g.tiles_m * g.tiles_n;
  const unsigned long long tlim = g.timeout_ns;

  if (threadIdx.x == 32) {
    for (int s = 0; s < 2 * NSTG; ++s) mbar_init(bar_full + 8 * s, 1);
    for (int s = 0; s < NSTG; ++s) mbar_init(bar_done + 8 * s, 1);
    for (int a = 0; a < NACC; ++a) mbar_init(bar_read + 8 * a, C::NPW);
    mbar_init(smem_u32(&last_s), 2);
    abort_flag_s = 0;
    issued_s = 0;
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
  depend_launch();
  depend_wait();
  // (a wait that runs out is told two seconds after its CTA began at the earliest; the grid fits on the GPU at once)
  if (blockIdx.x == 0 && threadIdx.x == 0) *g.status = 0;
  const int mine = (ntiles - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;  // this CTA's tiles
  const int blocks = mine * g.nkb;
  // an even number of stages gives a stage's blocks to one issuer anyway
  constexpr int NFULL = NSTG % 2 ? 2 * NSTG : NSTG;
  auto full_of = [](int it) { return it % NFULL; };

  // 640 threads x 96 registers at the launch = 128 x 32 + 512 x 112
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 32;");
    if (warp == 0) {
      // ---------------------------------------------------- TMA producer --
      if (lane == 0) {
        tma_prefetch_map(&mA);
        tma_prefetch_map(&mB);
        int it = 0;
        bool stop = false;
        for (int u = blockIdx.x; u < ntiles && !stop; u += gridDim.x) {
          const int m0 = (u / g.tiles_n) * FBM, n0 = (u % g.tiles_n) * BN;
          for (int kb = 0; kb < g.nkb; ++kb, ++it) {
            const int s = it % NSTG, ph = it / NSTG;
            if (it >= NSTG && !wait_f8(bar_done + 8 * s, (ph - 1) & 1, abort_flag, g.status, tlim)) {
              stop = true;
              break;
            }
            const uint32_t sA = ring + s * C::STAGE, sB = sA + C::TILE_A;
            const uint32_t fb = bar_full + 8 * full_of(it);
            mbar_arrive_expect_tx(fb, C::STAGE);
            tma_load_2d(sA, &mA, kb * FBK, m0, fb);
            tma_load_2d(sB, &mB, kb * FBK, n0, fb);
          }
        }
        issued_s = it;
      }
    } else if (warp < 3) {
      // ------------------------------------------------------ MMA issuers --
      if (lane == 0) {
        constexpr uint32_t idesc = idesc_e4m3_f32(FBM, BN);
        for (int it = warp - 1; it < blocks; it += 2) {
          const int s = it % NSTG, a = it % NACC;
          if (!wait_f8(bar_full + 8 * full_of(it), (it / NFULL) & 1, abort_flag, g.status, tlim)) break;
          if (it >= NACC && !wait_f8(bar_read + 8 * a, ((it - NACC) / NACC) & 1, abort_flag, g.status, tlim)) break;
          tc_fence_after();
          const uint32_t sA = ring + s * C::STAGE, sB = sA + C::TILE_A;
          const uint32_t dacc = tmem + (uint32_t)(a * BN);
#pragma unroll
          for (int k4 = 0; k4 < FBK / 32; ++k4)  // 32 bytes along the K-major rows
            umma_f8(dacc, sdesc_sw128(sA + k4 * 32, 16, 1024), sdesc_sw128(sB + k4 * 32, 16, 1024),
                    idesc, k4 != 0 ? 1u : 0u);
          umma_commit(bar_done + 8 * s);
        }
        umma_commit(smem_u32(&last_s));
      }
    }
    __syncwarp();
  } else {
    // --------------------------------------------- promotion and epilogue --
    asm volatile("setmaxnreg.inc.sync.aligned.u32 112;");
    const int q = warp & 3;          // TMEM lane quarter this warp may access
    const int hc = (warp - 4) >> 2;  // columns WC hc .. of the tile
    const uint32_t stg = out_stage + (uint32_t)(warp - 4) * C::STG;
    int it = 0;
    bool stop = false;
    for (int u = blockIdx.x; u < ntiles && !stop; u += gridDim.x) {
      const int m0 = (u / g.tiles_n) * FBM + q * 32, n0 = (u % g.tiles_n) * BN + hc * WC;
      const long long row = m0 + lane < g.M ? m0 + lane : g.M - 1;
      const float* xs = g.xs + row * g.nkb;
      const float* ws = g.Ws + (long long)((n0 < g.N ? n0 : g.N - 1) / 128) * g.nkb;
      float acc[WC];
#pragma unroll
      for (int j = 0; j < WC; ++j) acc[j] = 0.f;
      float sc = *xs * *ws;
      for (int kb = 0; kb < g.nkb; ++kb, ++it) {
        const int a = it % NACC;
        const int kn = kb + 1 < g.nkb ? kb + 1 : kb;
        const float x1 = xs[kn], w1 = ws[kn];  // the next block's scales on their way
        if (!wait_f8(bar_done + 8 * (it % NSTG), (it / NSTG) & 1, abort_flag, g.status, tlim)) {
          stop = true;
          break;
        }
        tc_fence_after();
        const uint32_t t = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(a * BN + hc * WC);
#pragma unroll
        for (int c = 0; c < WC; c += 32) {
          uint32_t r[32];
          tmem_ld32(t + c, r);
          tmem_wait_ld();
          tmem_reg_fence(r);
          if (c + 32 == WC) {  // the buffer has been read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_read + 8 * a);
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) acc[c + j] = fmaf(sc, __uint_as_float(r[j]), acc[c + j]);
        }
        sc = x1 * w1;
      }
      if (stop) break;
      // bf16 (+ bias) into the warp's swizzled box of 32 rows, TMA store
      if (lane == 0) bulk_wait_read_all();
      __syncwarp();
#pragma unroll
      for (int k = 0; k < WC / 8; ++k) {
        uint32_t pk[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = 8 * k + 2 * j, n = n0 + c;
          float b0 = 0.f, b1 = 0.f;
          if (g.bias && n < g.N) b0 = g.bias[n], b1 = g.bias[n + 1];  // (N is even)
          pk[j] = pack_bf16x2(acc[c] + b0, acc[c + 1] + b1);
        }
        const int ch = k ^ (WC == 64 ? lane & 7 : (lane >> 1) & 3);
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(stg + (uint32_t)(lane * WC * 2 + ch * 16)),
                     "r"(pk[0]), "r"(pk[1]), "r"(pk[2]), "r"(pk[3])
                     : "memory");
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        if (n0 < g.N && m0 < g.M) tma_store_2d(&mC, n0, m0, stg);
        bulk_commit();
      }
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    if (lane == 0 && *abort_flag) {
      // let the MMAs and TMA copies that were issued end before exit
      auto drain = [](uint32_t bar, uint32_t parity) {
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(bar, parity))
          if (globaltimer_ns() - t0 > 10000000ull) break;
      };
      drain(smem_u32(&last_s), 0);
      for (int k = issued_s - NSTG < 0 ? 0 : issued_s - NSTG; k < issued_s; ++k)
        drain(bar_full + 8 * full_of(k), (k / NFULL) & 1);
    }
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------- few rows --
constexpr int kFewRows = 64;
constexpr int kFewWarps = 8;

__device__ __forceinline__ void mma_e4m3_16832(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 16 weight rows (the MMA's M) x up to 8 NT tokens (its N) per CTA; the blocks of 128 go round
// the CTA's warps, whose sums meet in shared memory in a fixed order.  A thread's 16-byte loads
// take 32 consecutive k of a row: which k an MMA's operand slots stand for is free, as long as A's and
// B's agree, so the four MMAs of a block take them in the order in which they were loaded.
template <int NT>
__global__ void __launch_bounds__(32 * kFewWarps)
    proj_fp8_few_kernel(const uint8_t* xq, const float* xs, const uint8_t* Wq, const float* Ws, const float* bias,
                        __nv_bfloat16* y, int M, int N, int K, int* status) {
  __shared__ float part[kFewWarps][8 * NT][17];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * 16, nkb = (K + FBK - 1) / FBK;
  const uint8_t* w0 = Wq + (long long)(n0 + g) * K + t * 32;
  const uint8_t* w1 = w0 + 8LL * K;
  const bool has0 = n0 + g < N, has1 = n0 + g + 8 < N;
  const float* ws = Ws + (long long)(n0 / 128) * nkb;
  const uint4 z = make_uint4(0u, 0u, 0u, 0u);
  depend_launch();
  // (a kernel that begins while another one writes its inputs takes them by coherent loads alone)
  // the weights on their way to L2 (where alone they may still be written) while the kernel in front ends
  for (int kb = warp + kFewWarps * t; kb < nkb; kb += 4 * kFewWarps) {
    if (has0) asm volatile("prefetch.global.L2 [%0];" ::"l"(w0 - t * 32 + kb * FBK));
    if (has1) asm volatile("prefetch.global.L2 [%0];" ::"l"(w1 - t * 32 + kb * FBK));
  }
  depend_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *status = 0;  // no waits here: nothing to report
  float acc[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll 2
  for (int kb = warp; kb < nkb; kb += kFewWarps) {
    const int k = kb * FBK;
    uint4 a[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = k + t * 32 + 16 * h < K;
      a[0][h] = in && has0 ? *(reinterpret_cast<const uint4*>(w0 + k) + h) : z;
      a[1][h] = in && has1 ? *(reinterpret_cast<const uint4*>(w1 + k) + h) : z;
    }
    const float w = ws[kb];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int m = 8 * i + g;
      uint4 b[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        b[h] = m < M && k + t * 32 + 16 * h < K
                   ? *(reinterpret_cast<const uint4*>(xq + (long long)m * K + t * 32 + k) + h)
                   : z;
      float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t a0[4] = {a[0][h].x, a[1][h].x, a[0][h].y, a[1][h].y};
        const uint32_t a1[4] = {a[0][h].z, a[1][h].z, a[0][h].w, a[1][h].w};
        mma_e4m3_16832(d, a0, b[h].x, b[h].y);
        mma_e4m3_16832(d, a1, b[h].z, b[h].w);
      }
      const int c = 8 * i + 2 * t;  // this thread's two tokens
      const float s0 = c < M ? w * xs[(long long)c * nkb + kb] : 0.f;
      const float s1 = c + 1 < M ? w * xs[(long long)(c + 1) * nkb + kb] : 0.f;
      acc[i][0] = fmaf(s0, d[0], acc[i][0]);
      acc[i][1] = fmaf(s1, d[1], acc[i][1]);
      acc[i][2] = fmaf(s0, d[2], acc[i][2]);
      acc[i][3] = fmaf(s1, d[3], acc[i][3]);
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) part[warp][8 * i + 2 * t + (j & 1)][g + 8 * (j >> 1)] = acc[i][j];
  __syncthreads();
  for (int e = threadIdx.x; e < 8 * NT * 16; e += 32 * kFewWarps) {
    const int m = e / 16, n = e % 16;
    if (m >= M || n0 + n >= N) continue;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kFewWarps; ++k) s += part[k][m][n];
    y[(long long)m * N + n0 + n] = __float2bfloat16_rn(s + (bias ? bias[n0 + n] : 0.f));
  }
}

}  // namespace

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn();  // tc_gemm.cu

namespace {

// row-major [rows, cols] of `bytes`-byte values; box of bx columns x by rows
int make_map2(CUtensorMap* m, CUtensorMapDataType type, int bytes, const void* ptr, uint64_t rows, uint64_t cols,
              uint32_t bx, uint32_t by, CUtensorMapSwizzle swizzle) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return (int)cudaErrorNotSupported;
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {cols * bytes};
  const cuuint32_t box[2] = {bx, by};
  const cuuint32_t es[2] = {1, 1};
  const CUresult r = fn(m, type, 2, const_cast<void*>(ptr), dims, strides, box, es,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? 0 : (int)cudaErrorInvalidValue;
}

template <int BN>
int launch_bn(const ProjFp8Params& p, cudaStream_t s) {
  using C = F8Cfg<BN>;
  auto kern = proj_fp8_kernel<BN>;
  static int prepared[64][5];
  int e = prepare_launch(prepared, kern, C::SMEM, C::THREADS, 1);
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
  if ((e = make_map2(&a, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p.xq, (uint64_t)p.M, (uint64_t)p.K, FBK, FBM,
                     CU_TENSOR_MAP_SWIZZLE_128B)))
    return e;
  if ((e = make_map2(&b, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p.Wq, (uint64_t)p.N, (uint64_t)p.K, FBK, BN,
                     CU_TENSOR_MAP_SWIZZLE_128B)))
    return e;
  if ((e = make_map2(&c, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p.y, (uint64_t)p.M, (uint64_t)p.N, C::WC, 32,
                     C::WC == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B)))
    return e;
  const int cap = sm_count();
  const int grid = (int)(tiles < cap ? tiles : cap);
  return launch_dependent(kern, (unsigned)grid, C::THREADS, C::SMEM, s, a, b, c, g);
}

}  // namespace

template <int NT>
static int launch_few(const ProjFp8Params& p, cudaStream_t s) {
  return launch_dependent(proj_fp8_few_kernel<NT>, (unsigned)((p.N + 15) / 16), 32 * kFewWarps, 0, s,
                          static_cast<const uint8_t*>(p.xq), p.xs, static_cast<const uint8_t*>(p.Wq), p.Ws, p.bias,
                          static_cast<__nv_bfloat16*>(p.y), p.M, p.N, p.K, p.status);
}

int launch_proj_fp8(const ProjFp8Params& p, cudaStream_t s) {
  // Few rows: the kernel that reads each weight once, whose CTAs of 16 columns take longer with more rows, up to so many
  // rounds of them (us on the device, it / tiles; K = 768 and 4096: 16 rows, N = 8192 3.8 / 5.4, 9.6 / 13.5; 32 rows, N =
  // 4096 4.1 / 5.4, 12.4 / 13.2; 33 rows, N = 2304 3.6 / 5.3, 8.9 / 13.4, N = 4096 6.4 / 5.4, 16.5 / 13.2).
  const int rounds = (p.N + 16 * sm_count() - 1) / (16 * sm_count());
  if (p.M <= 16 && rounds <= 4) return p.M <= 8 ? launch_few<1>(p, s) : launch_few<2>(p, s);
  if (p.M <= 32 && rounds <= 2) return launch_few<4>(p, s);
  if (p.M <= kFewRows && rounds == 1) return launch_few<8>(p, s);
  // the larger tiles where they are enough for every SM
  const long long wide = (long long)((p.M + FBM - 1) / FBM) * ((p.N + 255) / 256);
  return wide >= sm_count() ? launch_bn<256>(p, s) : launch_bn<128>(p, s);
}

}  // namespace srnn
