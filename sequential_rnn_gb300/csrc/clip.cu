// The common norm of many tensors and their scaling to a limit:
//   norm = sqrt(sum of all x^2),   x <- x (limit / norm) where norm > limit
//
// Two kernels over units of 16 KB (the tensors' addresses and sizes come as kernel parameters, so a captured call
// needs no copy): the sums, one partial a CTA, each CTA a contiguous range of units; then every CTA adds the partials in
// one order and goes through its range again, from its end, where the L2 still holds it.  Bound by bytes: 3 for every
// byte of gradient past what the L2 keeps.
//
// Squares are summed in fp32 for the 64 bytes that a thread takes at a time, and those sums in fp64.  Where
// such a sum leaves the range in which fp32 keeps its bits (squares that overflow or vanish), its values are
// squared in fp64.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "kernels.h"
#include "lm.h"
#include "ptx.cuh"

namespace srnn {
namespace {

constexpr int kThreads = 256;
constexpr int kCtasPerSm = 4;

struct Table {  // of one launch
  void* at[kClipTensors];
  long long size[kClipTensors];   // elements; negative: bf16
  int first[kClipTensors + 1];    // its first unit; the last: units in all
  int n;
};

__device__ __forceinline__ int tensor_of(const Table& t, int unit) {  // the last with first <= unit
  int lo = 0, hi = t.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (t.first[mid] <= unit)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}
// a CTA's units
__device__ __forceinline__ void range_of(const Table& t, int& u0, int& u1) {
  const long long units = t.first[t.n];
  u0 = (int)(units * blockIdx.x / gridDim.x);
  u1 = (int)(units * (blockIdx.x + 1) / gridDim.x);
}

// sum over the CTA in a fixed order; every thread gets it
__device__ double cta_sum(double v, double* sh) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (threadIdx.x % 32 == 0) sh[threadIdx.x / 32] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) s += sh[i];
  return s;
}

// the values of a 16-byte vector
template <bool BF>
__device__ __forceinline__ void values(const uint4& r, float (&x)[BF ? 8 : 4]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (BF)
      x[2 * i] = bf16_lo(w[i]), x[2 * i + 1] = bf16_hi(w[i]);
    else
      x[i] = __uint_as_float(w[i]);
  }
}

constexpr int kVecs = kClipUnit / 16 / kThreads;  // vectors of a unit that a thread takes

template <bool BF>
__device__ __forceinline__ double squares(const uint4 (&r)[kVecs]) {
  constexpr int E = BF ? 8 : 4;
  float s[kVecs] = {};
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    float x[E];
    values<BF>(r[i], x);
#pragma unroll
    for (int j = 0; j < E; ++j) s[i] = fmaf(x[j], x[j], s[i]);
  }
  float all = 0.f;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) all += s[i];
  if (all >= 0x1p-100f && all <= 0x1p127f) return all;
  // (what is below 2^-100 in all may have lost squares below 2^-126; NaN comes here, too)
  double d = 0.0;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    if (((r[i].x | r[i].y | r[i].z | r[i].w) & (BF ? 0x7fff7fffu : 0x7fffffffu)) == 0u) continue;
    float x[E];
    values<BF>(r[i], x);
#pragma unroll
    for (int j = 0; j < E; ++j) d = fma((double)x[j], (double)x[j], d);
  }
  return d;
}

template <bool BF>
__device__ double unit_sum(const void* at, long long size, long long e0) {
  constexpr int E = BF ? 8 : 4, UNIT = kClipUnit / (16 / E);
  const char* p = static_cast<const char*>(at) + e0 * (16 / E);
  const long long left = size - e0;
  const int n = (int)(left < UNIT ? left : UNIT);
  const bool aligned = reinterpret_cast<uintptr_t>(p) % 16 == 0;
  const int whole = aligned ? n / E : 0;
  uint4 r[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int v = threadIdx.x + i * kThreads;
    r[i] = make_uint4(0u, 0u, 0u, 0u);
    if (v < whole) r[i] = reinterpret_cast<const uint4*>(p)[v];
  }
  double d = squares<BF>(r);
  for (int i = whole * E + threadIdx.x; i < n; i += kThreads) {
    const double x = BF ? (double)__bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i])
                        : (double)reinterpret_cast<const float*>(p)[i];
    d = fma(x, x, d);
  }
  return d;
}

__global__ void __launch_bounds__(kThreads) clip_sum_kernel(const __grid_constant__ Table t, double* part) {
  __shared__ double sh[kThreads / 32];
  depend_launch();
  int u0, u1;
  range_of(t, u0, u1);
  int i = tensor_of(t, u0);
  depend_wait();
  double d = 0.0;
  for (int u = u0; u < u1; ++u) {
    while (u >= t.first[i + 1]) ++i;
    const long long size = t.size[i], k = u - t.first[i];
    d += size < 0 ? unit_sum<true>(t.at[i], -size, k * (kClipUnit / 2)) : unit_sum<false>(t.at[i], size, k * (kClipUnit / 4));
  }
  d = cta_sum(d, sh);
  if (threadIdx.x == 0) part[blockIdx.x] = d;
}

template <bool BF>
__device__ void unit_scale(void* at, long long size, long long e0, float by, float again) {
  constexpr int E = BF ? 8 : 4, UNIT = kClipUnit / (16 / E);
  char* p = static_cast<char*>(at) + e0 * (16 / E);
  const long long left = size - e0;
  const int n = (int)(left < UNIT ? left : UNIT);
  const bool aligned = reinterpret_cast<uintptr_t>(p) % 16 == 0;
  const int whole = aligned ? n / E : 0;
  uint4 r[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int v = threadIdx.x + i * kThreads;
    if (v < whole) r[i] = reinterpret_cast<uint4*>(p)[v];
  }
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int v = threadIdx.x + i * kThreads;
    if (v >= whole) continue;
    float x[E];
    values<BF>(r[i], x);
#pragma unroll
    for (int j = 0; j < E; ++j) x[j] = x[j] * by * again;
    if (BF)
      r[i] = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[E - 4], x[E - 3]),
                        pack_bf16x2(x[E - 2], x[E - 1]));
    else
      r[i] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    reinterpret_cast<uint4*>(p)[v] = r[i];
  }
  for (int i = whole * E + threadIdx.x; i < n; i += kThreads) {
    if (BF) {
      __nv_bfloat16* x = reinterpret_cast<__nv_bfloat16*>(p) + i;
      *x = __float2bfloat16_rn(__bfloat162float(*x) * by * again);
    } else {
      float* x = reinterpret_cast<float*>(p) + i;
      *x = *x * by * again;
    }
  }
}

// parts: of all launches of clip_sum_kernel, which only the last of these kernels' launches may overwrite
__global__ void __launch_bounds__(kThreads)
    clip_scale_kernel(const __grid_constant__ Table t, const double* part, int parts, double limit, float* norm) {
  __shared__ double sh[kThreads / 32];
  depend_launch();
  int u0, u1;
  range_of(t, u0, u1);
  int i = u1 > u0 ? tensor_of(t, u1 - 1) : 0;
  depend_wait();
  double d = 0.0;
  for (int j = threadIdx.x; j < parts; j += kThreads) d += part[j];
  const double all = sqrt(cta_sum(d, sh));
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)all;
  if (!(all > limit) || isinf(all)) return;
  // a factor that is no normal fp32 number is applied in two steps
  const double f = limit / all;
  const bool tiny = f < 0x1p-100;
  const float by = tiny ? 0x1p-64f : (float)f, again = tiny ? (float)(f * 0x1p64) : 1.f;
  for (int u = u1 - 1; u >= u0; --u) {
    while (u < t.first[i]) --i;
    const long long size = t.size[i], k = u - t.first[i];
    if (size < 0)
      unit_scale<true>(t.at[i], -size, k * (kClipUnit / 2), by, again);
    else
      unit_scale<false>(t.at[i], size, k * (kClipUnit / 4), by, again);
  }
}

}  // namespace

int clip_parts(int n) { return (n / kClipTensors + 1) * kCtasPerSm * sm_count(); }

int launch_clip(const ClipParams& p, cudaStream_t s) {
  Table t;
  int parts = 0;
  // the tensors from i on that fit a launch; returns the next one
  auto fill = [&](int i) {
    t.n = 0;
    long long units = 0;
    for (; i < p.n && t.n < kClipTensors; ++i) {
      const long long size = p.sizes[i];
      if (size == 0) continue;
      const long long per = kClipUnit / (p.dtypes[i] == 1 ? 2 : 4), more = (size + per - 1) / per;
      if (units + more > 0x7fffffff) break;  // (of one tensor: refused before)
      t.at[t.n] = p.at[i];
      t.size[t.n] = p.dtypes[i] == 1 ? -size : size;
      t.first[t.n++] = (int)units;
      units += more;
    }
    t.first[t.n] = (int)units;
    return i;
  };
  const long long most = (long long)kCtasPerSm * sm_count();
  auto grid = [&] { return (unsigned)(t.first[t.n] < most ? t.first[t.n] : most); };
  for (int i = 0; i < p.n;) {
    i = fill(i);
    if (t.n == 0) continue;
    const int e = launch_dependent(clip_sum_kernel, grid(), kThreads, 0, s, t, p.part + parts);
    if (e != 0) return e;
    parts += (int)grid();
  }
  bool told = false;
  for (int i = 0; !told || (p.limit < INFINITY && i < p.n);) {
    i = fill(i);
    if (t.n == 0 && told) continue;
    // (without a limit, or without tensors, one CTA for the norm)
    const bool scale = p.limit < INFINITY && t.n > 0;
    if (!scale) t.n = 0, t.first[0] = 0;
    const int e = launch_dependent(clip_scale_kernel, scale ? grid() : 1u, kThreads, 0, s, t, (const double*)p.part, parts,
                                   (double)p.limit, told ? (float*)nullptr : p.norm);
    if (e != 0) return e;
    told = true;
  }
  return 0;
}

}  // namespace srnn
