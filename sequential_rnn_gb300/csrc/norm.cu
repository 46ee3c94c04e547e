// Root-mean-square norm with the residual's addition, its gradient, and the
// 8-bit weight quantiser.
//
//   h = round(x + residual);  r = 1 / sqrt(mean_n h^2 + eps);  y = h r w
//   8-bit output: per row and block of 128 columns s = max|y| / 448 (1 where
//   the block is all zero), q = e4m3(y / s), the code nearest to the exact quotient:
//   r cancels, y / s = 448 h w / max|h w|
//   gradient, xh = h r:  dx = r (w dy - xh mean_n(w dy xh)) + dh,
//                        dw = sum over rows of dy xh
//
// The norm is taken of h as it is stored (rounded to the input type), so that
// the gradient, which reads the stored h, differentiates the very function that
// was computed.  All sums are fp32.
//
// Both are bound by their bytes.  Rows of up to 128 vectors take a warp each, persistent, with the weights (gradient:
// the columns' share of dw) in registers and the next row's loads in flight: 16384 x 768 to 8 bits 16.5 us,
// 5.4 TB/s of the copy's 6.8 (a row to each warp of a launch, without the next row's loads: 2 us more);
// gradient, 16384 x 1000, 29.3 us, 4.5 TB/s.  Wider rows take a CTA, which registers hold as well.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
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

__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3) |
         (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3) << 16;
}

// scale of a block whose largest magnitude is `top` (NaN values do not count towards it);
// 1 where the block is zero or so small that the quotient underflows
__device__ __forceinline__ float block_scale(float top) {
  const float s = top / kE4m3Max;
  return s > 0.f ? s : 1.f;
}

// a block's largest product and r: between them the scale, their product / 448, is no subnormal number
__device__ __forceinline__ bool in_range(float v) { return v >= 0x1p-58f && v <= 0x1p60f; }
__device__ __forceinline__ float e4m3_value(uint32_t code) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)code, __NV_E4M3)));
}

// The codes of E of a block's 128 columns and the block's scale, together with the LANES neighbouring threads of its
// other columns and all of the warp.  t = h w in fp32, its products with the ends of an interval of 448 / max|t| that
// is wider than the five roundings between them and the exact quotient (5 2^-24): where both give the same code
// the quotient does, too.  Where they give neighbours (values near a tie between them; with weights of one, whose
// products are short numbers, many are ties) 448 h w and the tie times max|h w| are compared as sums of two fp32 numbers,
// exact to 2^-46; what rounds to the tie in fp32 goes to the even code.  (A division in fp32 for each value instead took
// half of the kernel's time, and, with y and s rounded before it, put every millionth value on the other side of
// a tie; in 64 bits rows with many ties took four times as long.)
// False where the numbers leave the range of this (zeros stay in it): then quantize_wide() has to do it.
template <int E, int LANES>
__device__ __forceinline__ bool quantize_block(const float (&h)[E], const float (&w)[E], float r, uint32_t (&q)[E / 4],
                                               float& s) {
  float t[E], top = 0.f;
#pragma unroll
  for (int j = 0; j < E; ++j) {
    t[j] = h[j] * w[j];
    top = fmaxf(top, fabsf(t[j]));
  }
#pragma unroll
  for (int o = LANES / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float inv = kE4m3Max / top, a = inv * (1.f - 0x1p-21f), b = inv * (1.f + 0x1p-21f);
  uint32_t hi[E / 4], differ = 0;
#pragma unroll
  for (int j = 0; j < E; j += 4) {
    q[j / 4] = pack_e4m3(t[j] * a, t[j + 1] * a, t[j + 2] * a, t[j + 3] * a);
    hi[j / 4] = pack_e4m3(t[j] * b, t[j + 1] * b, t[j + 2] * b, t[j + 3] * b);
    differ |= q[j / 4] ^ hi[j / 4];
  }
  s = top * r * (1.f / kE4m3Max);
  if (__any_sync(0xffffffffu, differ)) {
    float rest = -INFINITY;  // what rounding took from the largest product
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const float e = fmaf(h[j], w[j], -t[j]);
      if (fabsf(t[j]) == top) rest = fmaxf(rest, t[j] < 0.f ? -e : e);
    }
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) rest = fmaxf(rest, __shfl_xor_sync(0xffffffffu, rest, o));
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const int at = 8 * (j % 4);
      const uint32_t lo = q[j / 4] >> at & 0xffu, up = hi[j / 4] >> at & 0xffu;
      if (lo == up) continue;
      const float tie = 0.5f * fabsf(e4m3_value(lo) + e4m3_value(up)), e = fmaf(h[j], w[j], -t[j]);
      const float x = kE4m3Max * fabsf(t[j]), y = tie * top;
      const float d = (x - y) + ((fmaf(kE4m3Max, fabsf(t[j]), -x) + kE4m3Max * (t[j] < 0.f ? -e : e)) -
                                 (fmaf(tie, top, -y) + tie * rest));
      // half of the tie's last place, times max|t|
      const float near = top * __uint_as_float((__float_as_uint(tie) & 0x7f800000u) - (24u << 23));
      const bool take = fabsf(d) <= near ? (lo & 1u) != 0 : d > 0.f;
      if (take) q[j / 4] ^= (lo ^ up) << at;
    }
  }
  if (top == 0.f && r <= 0x1p60f) {  // (r is not a number where h has one)
    bool zero = true;  // (fmaxf passes over products that are not numbers)
#pragma unroll
    for (int j = 0; j < E; ++j) zero = zero && t[j] == 0.f;
    if (!zero) return false;
    s = 1.f;
#pragma unroll
    for (int j = 0; j < E / 4; ++j) q[j] = 0u;
    return true;
  }
  return in_range(top) && in_range(r);
}
// The same in 64 bits, by the whole warp: products or scales near the ends of fp32's range, values that are not finite.
template <int E, int LANES>
__device__ __forceinline__ void quantize_wide(const float (&h)[E], const float (&w)[E], float r, uint32_t (&q)[E / 4],
                                              float& s) {
  double top = 0.0;
#pragma unroll
  for (int j = 0; j < E; ++j) top = fmax(top, fabs((double)h[j] * w[j]));
#pragma unroll
  for (int o = LANES / 2; o; o >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, o));
  s = (float)(top * r / kE4m3Max);
  double f = kE4m3Max / top;
  if (!(s >= 0x1p-126f)) f = s > 0.f ? (double)r / s : r;  // (a subnormal scale is coarse: the quotient by what is stored)
  if (!(s > 0.f)) s = 1.f;  // zeros, values that underflow, a row whose r is zero or not a number
#pragma unroll
  for (int j = 0; j < E; j += 4) {
    float c[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) c[k] = (float)((double)h[j + k] * w[j + k] * f);
    q[j / 4] = pack_e4m3(c[0], c[1], c[2], c[3]);
  }
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

// Any width and alignment up to 4096 columns: a CTA per row of as many warps as the row has blocks of 128 columns, up to
// eight; a thread's values, four of each block of its warp, stay in registers between the sum and the output.
// Values are loaded one by one, since a row may begin at any of them; 16384 x 1001 bf16 with a residual in
// 62.5 us, 67 to 8 bits.
template <class T, int NB>
__global__ void __launch_bounds__(256) norm_rows_kernel(const NormParams p) {
  __shared__ float red[8];
  depend_launch();
  depend_wait();
  const int N = p.N, nblk = (N + kBlk - 1) / kBlk, W = blockDim.x >> 5, wp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + row * N;
    const T* res = p.residual ? static_cast<const T*>(p.residual) + row * N : nullptr;
    T* h = p.h ? static_cast<T*>(p.h) + row * N : nullptr;
    float hv[NB][4], ss = 0.f;
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = (wp + W * i) * kBlk + 32 * j + lane;
        hv[i][j] = n < N ? load1(x + n) : 0.f;
      }
    if (res)
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int n = (wp + W * i) * kBlk + 32 * j + lane;
          if (n < N) hv[i][j] = rounded<T>(hv[i][j] + load1(res + n));
        }
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) ss += hv[i][j] * hv[i][j];
    const float r = rsqrtf(block_sum(ss, red) / (float)N + p.eps);
    if (p.rstd && threadIdx.x == 0) p.rstd[row] = r;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int b = wp + W * i;
      if (b >= nblk) break;
      float w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = b * kBlk + 32 * j + lane;
        w[j] = n < N ? p.weight[n] : 0.f;
      }
      uint32_t q[1];
      if (p.scale) {
        float s;
        if (__any_sync(0xffffffffu, !quantize_block<4, 32>(hv[i], w, r, q, s))) quantize_wide<4, 32>(hv[i], w, r, q, s);
        if (lane == 0) p.scale[row * nblk + b] = s;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = b * kBlk + 32 * j + lane;
        if (n >= N) continue;
        if (p.scale)
          static_cast<uint8_t*>(p.y)[row * N + n] = (uint8_t)(q[0] >> (8 * j));
        else
          store1(static_cast<T*>(p.y) + row * N + n, hv[i][j] * r * w[j]);
        if (h) store1(h + n, hv[i][j]);
      }
    }
  }
}
// Its gradient, in the same places: a persistent grid, a thread keeps its columns' weights and share of dw.
template <class T, int NB>
__global__ void __launch_bounds__(256) norm_bwd_rows_kernel(const NormBwdParams p) {
  __shared__ float red[8];
  depend_wait();
  const int N = p.N, W = blockDim.x >> 5, n0 = (threadIdx.x >> 5) * kBlk + (threadIdx.x & 31);
  float w[NB][4], dw[NB][4];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + W * i * kBlk + 32 * j;
      w[i][j] = n < N ? p.weight[n] : 0.f;
      dw[i][j] = 0.f;
    }
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* dy = static_cast<const T*>(p.dy) + row * N;
    const T* h = static_cast<const T*>(p.h) + row * N;
    const float r = p.rstd[row];
    float g[NB][4], xh[NB][4], e[NB][4], dot = 0.f;
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + W * i * kBlk + 32 * j;
        g[i][j] = n < N ? load1(dy + n) : 0.f;
        xh[i][j] = n < N ? load1(h + n) : 0.f;
        e[i][j] = n < N && p.dh ? load1(static_cast<const T*>(p.dh) + row * N + n) : 0.f;
      }
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        xh[i][j] *= r;
        dw[i][j] = fmaf(g[i][j], xh[i][j], dw[i][j]);
        g[i][j] *= w[i][j];
        dot = fmaf(g[i][j], xh[i][j], dot);
      }
    dot = block_sum(dot, red) / (float)N;
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + W * i * kBlk + 32 * j;
        if (n < N)
          store1(static_cast<T*>(p.dx) + row * N + n, e[i][j] + r * (g[i][j] - xh[i][j] * dot));
      }
  }
  depend_launch();
  if (p.dw)
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + W * i * kBlk + 32 * j;
        if (n < N) p.part[(long long)blockIdx.x * N + n] = dw[i][j];
      }
}

// One CTA per row, any width and alignment.
template <class T>
__global__ void __launch_bounds__(256) norm_any_kernel(const NormParams p) {
  __shared__ float red[8];
  const int N = p.N;
  depend_launch();
  depend_wait();
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
      float hv[4], w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = b * kBlk + 32 * j + lane;
        hv[j] = n < N ? rounded<T>(load1(x + n) + (res ? load1(res + n) : 0.f)) : 0.f;
        w[j] = n < N ? p.weight[n] : 0.f;
      }
      uint32_t q[1];
      if (p.scale) {
        float s;
        if (__any_sync(0xffffffffu, !quantize_block<4, 32>(hv, w, r, q, s))) quantize_wide<4, 32>(hv, w, r, q, s);
        if (lane == 0) p.scale[row * nblk + b] = s;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = b * kBlk + 32 * j + lane;
        if (n >= N) continue;
        if (p.scale)
          static_cast<uint8_t*>(p.y)[row * N + n] = (uint8_t)(q[0] >> (8 * j));
        else
          store1(static_cast<T*>(p.y) + row * N + n, hv[j] * r * w[j]);
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
  depend_wait();
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

// ------------------------------------------------------- vector kernels --
// Rows whose width and pointers allow 16-byte accesses (8 bf16 or 4 fp32 values)
// and fit a CTA's registers.  W = 1: a warp per row (up to 128 vectors), else a
// CTA per row.  A row's vectors v = t + i TPR stay in registers between the sum and the
// output, so every byte moves once; 128 columns are 16 (bf16) or 32 (fp32)
// neighbouring threads' vectors, which find the block's largest value by shuffles.
template <class T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int E = 8;
  static __device__ __forceinline__ void unpack(const uint4& u, float (&f)[8]) {
    f[0] = bf16_lo(u.x), f[1] = bf16_hi(u.x), f[2] = bf16_lo(u.y), f[3] = bf16_hi(u.y);
    f[4] = bf16_lo(u.z), f[5] = bf16_hi(u.z), f[6] = bf16_lo(u.w), f[7] = bf16_hi(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
};
template <>
struct Vec<float> {
  static constexpr int E = 4;
  static __device__ __forceinline__ void unpack(const uint4& u, float (&f)[4]) {
    f[0] = __uint_as_float(u.x), f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z), f[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
};
template <int E>
__device__ __forceinline__ void load_weight(const float* w, int col, float (&f)[E]) {
#pragma unroll
  for (int j = 0; j < E; j += 4) {
    const float4 v = *reinterpret_cast<const float4*>(w + col + j);
    f[j] = v.x, f[j + 1] = v.y, f[j + 2] = v.z, f[j + 3] = v.w;
  }
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// quantize_wide() for a vector of h and its weights: out of line, it is rare
struct Codes {
  uint32_t q[2];
  float s;
};
template <class T>
__device__ __noinline__ Codes wide_codes(uint4 h, const float* weight, float r) {
  constexpr int E = Vec<T>::E;
  float y[E], w[E];
  uint32_t q[E / 4];
  Codes c;
  load_weight<E>(weight, 0, w);
  Vec<T>::unpack(h, y);
  quantize_wide<E, kBlk / E>(y, w, r, q, c.s);
  c.q[0] = q[0], c.q[1] = q[E / 4 - 1];
  return c;
}
constexpr int kRowsPerCta = 8;  // warp-per-row kernels: 256 threads
constexpr int kNormCtas = 2;    // their CTAs per SM

template <class T, int NV, bool WARP, bool QUANT>
__global__ void __launch_bounds__(WARP ? 256 : 1024, WARP ? kNormCtas : 1) norm_vec_kernel(const NormParams p) {
  constexpr int E = Vec<T>::E;
  __shared__ float red[32];
  const int TPR = WARP ? 32 : blockDim.x;
  const int t = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int nv = p.N / E;
  depend_launch();
  depend_wait();
  // a warp keeps its columns' weights for all of its rows
  float w[WARP ? NV : 1][E];
  if (WARP)
#pragma unroll
    for (int i = 0; i < NV; ++i) load_weight<E>(p.weight, (t + i * TPR < nv ? t + i * TPR : 0) * E, w[i]);
  const long long stride = WARP ? (long long)gridDim.x * kRowsPerCta : gridDim.x;
  long long row = WARP ? (long long)blockIdx.x * kRowsPerCta + (threadIdx.x >> 5) : blockIdx.x;
  uint4 hv[NV], rv[NV];
  auto load_row = [&](long long at) {
    const uint4* x = reinterpret_cast<const uint4*>(p.x) + at * nv;
    const uint4* res = reinterpret_cast<const uint4*>(p.residual) + at * nv;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t + i * TPR;
      const bool in = at < p.rows && v < nv;
      hv[i] = in ? x[v] : make_uint4(0u, 0u, 0u, 0u);
      rv[i] = in && p.residual ? res[v] : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  load_row(row);
  for (; row < p.rows; row += stride) {
    uint4* h = reinterpret_cast<uint4*>(p.h) + row * nv;
    uint4 cur[NV];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float a[E];
      cur[i] = hv[i];
      Vec<T>::unpack(cur[i], a);
      if (p.residual) {
        float b[E];
        Vec<T>::unpack(rv[i], b);
#pragma unroll
        for (int j = 0; j < E; ++j) a[j] += b[j];
        cur[i] = Vec<T>::pack(a);  // the rounding of h
        Vec<T>::unpack(cur[i], a);
      }
#pragma unroll
      for (int j = 0; j < E; ++j) ss += a[j] * a[j];
    }
    if (WARP) load_row(row + stride);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (p.h && t + i * TPR < nv) h[t + i * TPR] = cur[i];
    const float sum = WARP ? warp_sum(ss) : block_sum(ss, red);
    const float r = rsqrtf(sum / (float)p.N + p.eps);
    if (p.rstd && t == 0) p.rstd[row] = r;
    uint32_t bad = 0;  // vectors to be done again
    auto store_block = [&](int v, const uint32_t* q, float s) {
      if (v >= nv) return;
      if (v % (kBlk / E) == 0) p.scale[row * ((p.N + kBlk - 1) / kBlk) + v / (kBlk / E)] = s;
      uint8_t* dst = static_cast<uint8_t*>(p.y) + row * p.N + v * E;
      if constexpr (E == 8)
        *reinterpret_cast<uint2*>(dst) = make_uint2(q[0], q[1]);
      else
        *reinterpret_cast<uint32_t*>(dst) = q[0];
    };
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t + i * TPR;
      if (!QUANT && v >= nv) break;
      float y[E];
      if (!WARP) load_weight<E>(p.weight, (v < nv ? v : 0) * E, w[0]);
      Vec<T>::unpack(cur[i], y);
      if constexpr (QUANT) {  // (past the row h is zero)
        uint32_t q[E / 4];
        float s;
        bad |= (quantize_block<E, kBlk / E>(y, w[WARP ? i : 0], r, q, s) ? 0u : 1u) << i;
        store_block(v, q, s);
      } else {
#pragma unroll
        for (int j = 0; j < E; ++j) y[j] = y[j] * r * w[WARP ? i : 0][j];
        reinterpret_cast<uint4*>(p.y)[row * nv + v] = Vec<T>::pack(y);
      }
    }
    if constexpr (QUANT) {
      if (__any_sync(0xffffffffu, bad)) {
        bad = __reduce_or_sync(0xffffffffu, bad);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (!(bad >> i & 1)) continue;
          const int v = t + i * TPR;
          const Codes c = wide_codes<T>(cur[i], p.weight + (v < nv ? v : 0) * E, r);
          store_block(v, c.q, c.s);
        }
      }
    }
    if (!WARP) break;  // (a CTA has one row)
  }
}

// Gradient: a persistent grid; every thread keeps its columns' share of dw in
// registers over all of its rows.
template <class T, int NV, bool WARP>
__global__ void __launch_bounds__(256) norm_bwd_vec_kernel(const NormBwdParams p) {
  constexpr int E = Vec<T>::E;
  depend_wait();
  __shared__ float red[32];
  const int TPR = WARP ? 32 : blockDim.x;
  const int t = WARP ? (threadIdx.x & 31) : threadIdx.x, wp = threadIdx.x >> 5;
  const int nv = p.N / E;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  float dw[NV][E];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < E; ++j) dw[i][j] = 0.f;
  constexpr int RPC = WARP ? kRowsPerCta : 1;  // rows of a CTA, side by side
  const long long first = (long long)blockIdx.x * RPC + (WARP ? wp : 0);
  const long long step = (long long)gridDim.x * RPC;
  uint4 gv[NV], hv[NV], ev[NV];
  float r = 0.f;
  auto load = [&](long long row) {
    const uint4* dy = reinterpret_cast<const uint4*>(p.dy) + row * nv;
    const uint4* h = reinterpret_cast<const uint4*>(p.h) + row * nv;
    const uint4* dh = reinterpret_cast<const uint4*>(p.dh) + row * nv;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t + i * TPR;
      gv[i] = v < nv ? dy[v] : zero;
      hv[i] = v < nv ? h[v] : zero;
      ev[i] = p.dh && v < nv ? dh[v] : zero;
    }
    r = p.rstd[row];
  };
  constexpr bool AHEAD = NV <= 4;  // registers for the next row
  if (AHEAD && first < p.rows) load(first);
  for (long long row = first; row < p.rows; row += step) {
    if (!AHEAD) load(row);
    uint4 g0[NV], h0[NV], e0[NV];
    const float rs = r;
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t + i * TPR;
      float g[E], a[E], w[E];
      Vec<T>::unpack(gv[i], g);
      Vec<T>::unpack(hv[i], a);
      load_weight<E>(p.weight, (v < nv ? v : 0) * E, w);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const float xh = a[j] * rs;
        dw[i][j] = fmaf(g[j], xh, dw[i][j]);
        dot = fmaf(g[j] * w[j], xh, dot);
      }
      g0[i] = gv[i];
      h0[i] = hv[i];
      e0[i] = ev[i];
    }
    // the next row is on its way while this one's sum is taken and its dx written
    if (AHEAD && row + step < p.rows) load(row + step);
    dot = (WARP ? warp_sum(dot) : block_sum(dot, red)) / (float)p.N;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t + i * TPR;
      if (v >= nv) break;
      float g[E], a[E], e[E], w[E];
      Vec<T>::unpack(g0[i], g);
      Vec<T>::unpack(h0[i], a);
      Vec<T>::unpack(e0[i], e);
      load_weight<E>(p.weight, v * E, w);
#pragma unroll
      for (int j = 0; j < E; ++j) e[j] += rs * (w[j] * g[j] - a[j] * rs * dot);
      reinterpret_cast<uint4*>(p.dx)[row * nv + v] = Vec<T>::pack(e);
    }
  }
  depend_launch();
  if (p.dw == nullptr) return;
  float* part = p.part + (long long)blockIdx.x * p.N;
  if (WARP) {  // the CTA's warps one after the other, in shared memory
    __shared__ float acc[NV * 32 * E];
    for (int k = 0; k < RPC; ++k) {
      if (wp == k)
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < E; ++j) {
            float* a = acc + (i * E + j) * 32 + t;
            *a = k == 0 ? dw[i][j] : *a + dw[i][j];
          }
      __syncthreads();
    }
    for (int n = threadIdx.x; n < p.N; n += 32 * RPC) {
      const int v = n / E;
      part[n] = acc[((v / 32) * E + n % E) * 32 + v % 32];
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t + i * TPR;
      if (v >= nv) break;
#pragma unroll
      for (int j = 0; j < E; ++j) part[v * E + j] = dw[i][j];
    }
  }
}

// dw[n] = sum over the partial rows: 32 columns per CTA, the 32 threads of a column take every
// 32nd row (all their loads in flight at once), then meet in a fixed order
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float* part, float* dw, int parts, int N) {
  __shared__ float red[32][33];
  const int c = threadIdx.x & 31, k = threadIdx.x >> 5, n = blockIdx.x * 32 + c;
  float s = 0.f;
  depend_launch();
  depend_wait();
  if (n < N)
#pragma unroll 20
    for (int i = k; i < parts; i += 32) s += part[(long long)i * N + n];
  red[c][k] = s;
  __syncthreads();
  s = warp_sum(red[k][c]);
  if (c == 0 && blockIdx.x * 32 + k < N) dw[blockIdx.x * 32 + k] = s;
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

namespace {

bool vec_ok(const void* q) { return reinterpret_cast<uintptr_t>(q) % 16 == 0; }
// threads of a CTA for a row of nv vectors, at most four each; 0: too wide
int vec_threads(int nv) {
  for (int t = 64; t <= 1024; t *= 2)
    if (nv <= 4 * t) return t;
  return 0;
}

template <class T, bool QUANT>
int norm_typed(const NormParams& p, cudaStream_t s) {
  constexpr int E = Vec<T>::E;
  const bool vec = p.N % (QUANT ? 8 : E) == 0 && vec_ok(p.x) && vec_ok(p.residual) && vec_ok(p.h) &&
                   vec_ok(p.weight) && vec_ok(p.y);
  const int nv = p.N / E, th = vec_threads(nv);
  if (!vec && p.N <= 4096) {
    const int nblk = (p.N + kBlk - 1) / kBlk, threads = 32 * (nblk < 8 ? nblk : 8);
    const unsigned grid = (unsigned)(p.rows < 1000000 ? p.rows : 1000000);
    return nblk <= 8    ? launch_dependent(norm_rows_kernel<T, 1>, grid, threads, 0, s, p)
           : nblk <= 16 ? launch_dependent(norm_rows_kernel<T, 2>, grid, threads, 0, s, p)
                        : launch_dependent(norm_rows_kernel<T, 4>, grid, threads, 0, s, p);
  }
  if (!vec || th == 0) {
    return launch_dependent(norm_any_kernel<T>, (unsigned)(p.rows < 65536 ? p.rows : 65536), 256, 0, s, p);
  } else if (nv <= 128) {
    const long long ctas = (p.rows + kRowsPerCta - 1) / kRowsPerCta, most = (long long)kNormCtas * sm_count();
    const unsigned grid = (unsigned)(ctas < most ? ctas : most);
    if (nv <= 64)
      return launch_dependent(norm_vec_kernel<T, 2, true, QUANT>, grid, 256, 0, s, p);
    if (nv <= 96) return launch_dependent(norm_vec_kernel<T, 3, true, QUANT>, grid, 256, 0, s, p);
    return launch_dependent(norm_vec_kernel<T, 4, true, QUANT>, grid, 256, 0, s, p);
  }
  return launch_dependent(norm_vec_kernel<T, 4, false, QUANT>, (unsigned)p.rows, th, 0, s, p);
}

template <class T>
int norm_bwd_typed(const NormBwdParams& p, cudaStream_t s) {
  constexpr int E = Vec<T>::E;
  const bool vec = p.N % E == 0 && vec_ok(p.dy) && vec_ok(p.h) && vec_ok(p.weight) &&
                   vec_ok(p.dh) && vec_ok(p.dx);
  const int nv = p.N / E;
  int parts = norm_bwd_parts(p.rows, p.N);
  int e;
  if (!vec && p.N <= 4096) {
    const int nblk = (p.N + kBlk - 1) / kBlk, threads = 32 * (nblk < 8 ? nblk : 8);
    e = nblk <= 8    ? launch_dependent(norm_bwd_rows_kernel<T, 1>, parts, threads, 0, s, p)
        : nblk <= 16 ? launch_dependent(norm_bwd_rows_kernel<T, 2>, parts, threads, 0, s, p)
                     : launch_dependent(norm_bwd_rows_kernel<T, 4>, parts, threads, 0, s, p);
  } else if (!vec || nv > 8 * 256) {
    e = launch_dependent(norm_bwd_any_kernel<T>, parts, 256, 0, s, p);
  } else if (nv <= 128) {
    // (eight warps an SM with four vectors a thread: twelve, of 168 registers, took 31 us for 16384 x 1000, eight 25)
    const long long ctas = (p.rows + kRowsPerCta - 1) / kRowsPerCta, cap = (nv <= 64 ? 2LL : 1LL) * sm_count();
    if (ctas < parts) parts = (int)ctas;
    if (cap < parts) parts = (int)cap;
    e = nv <= 64 ? launch_dependent(norm_bwd_vec_kernel<T, 2, true>, parts, 256, 0, s, p)
                 : launch_dependent(norm_bwd_vec_kernel<T, 4, true>, parts, 256, 0, s, p);
  } else {
    const int th = vec_threads(nv);
    e = th != 0 && th <= 256 ? launch_dependent(norm_bwd_vec_kernel<T, 4, false>, parts, th, 0, s, p)
                             : launch_dependent(norm_bwd_vec_kernel<T, 8, false>, parts, 256, 0, s, p);
  }
  if (e == 0 && p.dw)
    e = launch_dependent(norm_dw_kernel, (unsigned)((p.N + 31) / 32), 1024, 0, s, (const float*)p.part, p.dw,
                         parts, p.N);
  return e;
}

}  // namespace

int launch_rms_norm(const NormParams& p, bool bf16, cudaStream_t s) {
  if (p.scale) return bf16 ? norm_typed<__nv_bfloat16, true>(p, s) : norm_typed<float, true>(p, s);
  return bf16 ? norm_typed<__nv_bfloat16, false>(p, s) : norm_typed<float, false>(p, s);
}

int norm_bwd_parts(long long rows, int) { return (int)(rows < 608 ? rows : 608); }  // 4 x 152 SMs

int launch_rms_norm_bwd(const NormBwdParams& p, bool bf16, cudaStream_t s) {
  return bf16 ? norm_bwd_typed<__nv_bfloat16>(p, s) : norm_bwd_typed<float>(p, s);
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
