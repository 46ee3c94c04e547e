// Root-mean-square norm with the residual's addition, its gradient, and the
// 8-bit weight quantiser.
//
//   h = round(x + residual);  r = 1 / sqrt(mean_n h^2 + eps);  y = h r w
//   8-bit output: per row and block of 128 columns s = max|y| / 448 (1 where
//   the block is all zero), q = e4m3(y / s)
//   gradient, xh = h r:  dx = r (w dy - xh mean_n(w dy xh)) + dh,
//                        dw = sum over rows of dy xh
//
// The norm is taken of h as it is stored (rounded to the input type), so that
// the gradient, which reads the stored h, differentiates the very function that
// was computed.  All sums are fp32.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "lm.h"
#include "ptx.cuh"

namespace srnn {
namespace {

constexpr float kE4m3Max = 448.f;
constexpr int kBlk = 128;  // columns that share a scale

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
template <class T>
__device__ __forceinline__ float rounded(float v);
template <>
__device__ __forceinline__ float rounded<float>(float v) { return v; }
template <>
__device__ __forceinline__ float rounded<__nv_bfloat16>(float v) { return bf16_round(v); }
__device__ __forceinline__ uint8_t to_e4m3(float v) {
  return (uint8_t)__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
}

// scale of a block whose largest magnitude is `top` (NaN values do not count towards it);
// 1 where the block is zero or so small that the quotient underflows
__device__ __forceinline__ float block_scale(float top) {
  const float s = top / kE4m3Max;
  return s > 0.f ? s : 1.f;
}

// sum over the block's threads (a multiple of 32), the same value in each
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[w] = v;
  __syncthreads();
  float t = 0.f;
  for (int i = 0; i < nw; ++i) t += red[i];
  return t;
}

// One CTA per row, any width and alignment.
template <class T>
__global__ void __launch_bounds__(256) norm_any_kernel(const NormParams p) {
  __shared__ float red[8];
  const int N = p.N;
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + row * N;
    const T* res = p.residual ? static_cast<const T*>(p.residual) + row * N : nullptr;
    T* h = p.h ? static_cast<T*>(p.h) + row * N : nullptr;
    float ss = 0.f;
    for (int n = threadIdx.x; n < N; n += 256) {
      const float v = rounded<T>(load1(x + n) + (res ? load1(res + n) : 0.f));
      ss += v * v;
    }
    const float r = rsqrtf(block_sum(ss, red) / (float)N + p.eps);
    if (p.rstd && threadIdx.x == 0) p.rstd[row] = r;
    const int nblk = (N + kBlk - 1) / kBlk, lane = threadIdx.x & 31;
    // a warp takes whole blocks of 128 columns; h is written last, since it may be x or residual
    for (int b = threadIdx.x >> 5; b < nblk; b += 8) {
      float hv[4], y[4], top = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = b * kBlk + 32 * j + lane;
        hv[j] = n < N ? rounded<T>(load1(x + n) + (res ? load1(res + n) : 0.f)) : 0.f;
        y[j] = n < N ? hv[j] * r * p.weight[n] : 0.f;
        top = fmaxf(top, fabsf(y[j]));
      }
      float inv = 1.f;
      if (p.scale) {
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float s = block_scale(top);
        if (lane == 0) p.scale[row * nblk + b] = s;
        inv = s;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = b * kBlk + 32 * j + lane;
        if (n >= N) continue;
        if (p.scale)
          static_cast<uint8_t*>(p.y)[row * N + n] = to_e4m3(y[j] / inv);
        else
          store1(static_cast<T*>(p.y) + row * N + n, y[j]);
        if (h) store1(h + n, hv[j]);
      }
    }
  }
}

// One CTA walks rows blockIdx.x, + gridDim.x, ..; thread t owns columns t, t + 256, ..
// of the tile of 1024 columns it is on, so dw needs no atomics.
constexpr int kBwdCols = 1024;
template <class T>
__global__ void __launch_bounds__(256) norm_bwd_any_kernel(const NormBwdParams p) {
  __shared__ float red[8];
  const int N = p.N;
  for (int c0 = 0; c0 < N; c0 += kBwdCols) {
    float dw[4] = {0.f, 0.f, 0.f, 0.f};
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
      const T* dy = static_cast<const T*>(p.dy) + row * N;
      const T* h = static_cast<const T*>(p.h) + row * N;
      const float r = p.rstd[row];
      float dot = 0.f;
      for (int n = threadIdx.x; n < N; n += 256) dot += load1(dy + n) * p.weight[n] * (load1(h + n) * r);
      dot = block_sum(dot, red) / (float)N;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = c0 + 256 * j + threadIdx.x;
        if (n >= N) continue;
        const float g = load1(dy + n), xh = load1(h + n) * r;
        dw[j] += g * xh;
        float dx = r * (p.weight[n] * g - xh * dot);
        if (p.dh) dx += load1(static_cast<const T*>(p.dh) + row * N + n);
        store1(static_cast<T*>(p.dx) + row * N + n, dx);
      }
    }
    if (p.dw)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = c0 + 256 * j + threadIdx.x;
        if (n < N) p.part[(long long)blockIdx.x * N + n] = dw[j];
      }
  }
}

// dw[n] = sum over the partial rows, in their order
__global__ void __launch_bounds__(256) norm_dw_kernel(const float* part, float* dw, int parts, int N) {
  const int n = blockIdx.x * 256 + threadIdx.x;
  if (n >= N) return;
  float s = 0.f;
  for (int i = 0; i < parts; ++i) s += part[(long long)i * N + n];
  dw[n] = s;
}

// One CTA per 128 x 128 block of W [N, K]; thread t holds column t of the block.
template <class T>
__global__ void __launch_bounds__(128)
    quantize_weight_kernel(const T* W, int N, int K, uint8_t* Wq, float* Ws) {
  __shared__ float red[4];
  const int k = blockIdx.x * kBlk + threadIdx.x, n0 = blockIdx.y * kBlk;
  const int n1 = n0 + kBlk < N ? n0 + kBlk : N;
  float top = 0.f;
  if (k < K)
    for (int n = n0; n < n1; ++n) top = fmaxf(top, fabsf(load1(W + (long long)n * K + k)));
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = top;
  __syncthreads();
  top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  const float s = block_scale(top);
  if (threadIdx.x == 0) Ws[(long long)blockIdx.y * gridDim.x + blockIdx.x] = s;
  if (k < K)
    for (int n = n0; n < n1; ++n)
      Wq[(long long)n * K + k] = to_e4m3(load1(W + (long long)n * K + k) / s);
}

}  // namespace

int launch_rms_norm(const NormParams& p, bool bf16, cudaStream_t s) {
  const int grid = (int)(p.rows < 65536 ? p.rows : 65536);
  if (bf16)
    norm_any_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(p);
  else
    norm_any_kernel<float><<<grid, 256, 0, s>>>(p);
  return (int)cudaGetLastError();
}

int norm_bwd_parts(long long rows, int) { return (int)(rows < 608 ? rows : 608); }

int launch_rms_norm_bwd(const NormBwdParams& p, bool bf16, cudaStream_t s) {
  const int parts = norm_bwd_parts(p.rows, p.N);
  if (bf16)
    norm_bwd_any_kernel<__nv_bfloat16><<<parts, 256, 0, s>>>(p);
  else
    norm_bwd_any_kernel<float><<<parts, 256, 0, s>>>(p);
  if (p.dw) norm_dw_kernel<<<(p.N + 255) / 256, 256, 0, s>>>(p.part, p.dw, parts, p.N);
  return (int)cudaGetLastError();
}

int launch_quantize_weight(const void* W, bool bf16, int N, int K, void* Wq, float* Ws,
                           cudaStream_t s) {
  const dim3 grid((unsigned)((K + kBlk - 1) / kBlk), (unsigned)((N + kBlk - 1) / kBlk));
  if (bf16)
    quantize_weight_kernel<<<grid, 128, 0, s>>>(static_cast<const __nv_bfloat16*>(W), N, K,
                                                static_cast<uint8_t*>(Wq), Ws);
  else
    quantize_weight_kernel<<<grid, 128, 0, s>>>(static_cast<const float*>(W), N, K,
                                                static_cast<uint8_t*>(Wq), Ws);
  return (int)cudaGetLastError();
}

}  // namespace srnn
