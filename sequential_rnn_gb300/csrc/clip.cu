// The common norm of many tensors and their scaling to a limit:
//   norm = sqrt(sum of all x^2),   x <- x (limit / norm) where norm > limit
//
// Two kernels over units of 16 KB (the tensors' addresses and sizes come as kernel parameters, so a captured call
// needs no copy): the sums, one partial a CTA, each CTA a contiguous range of units; then every CTA adds the partials in
// one order and goes through its range again, from its end, where the L2 still holds it.  Bound by bytes: 3 for every
// byte of gradient past what the L2 keeps (217 MB take 110 us, 5.9 TB/s of those, 94 the same tensors again), and small calls by two kernels'
// latencies one after the other (4.7 MB in 6 tensors: 9 us).  Four CTAs on an SM: six take 126 us for the 217 MB; rings of
// asynchronous copies instead of 64 bytes a thread in registers 118.
//
// Squares are summed in fp32 for the 64 bytes that a thread takes at a time, and those sums with their rounding errors
// beside them; fp64, which is slow here (two multiply-adds a clock on an SM), adds the CTAs' and takes the root.
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

struct Entry {
  void* at;
  long long size;  // elements; negative: bf16
  int first;       // its first unit
  int pad;
};
template <int N>
struct Table {  // of one launch
  int units, n;
  Entry t[N];
};

template <int N>
__device__ __forceinline__ int tensor_of(const Table<N>& t, int unit) {  // the last that begins at or before it
  int lo = 0, hi = t.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (t.t[mid].first <= unit)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}
// a CTA's units
template <int N>
__device__ __forceinline__ void range_of(const Table<N>& t, int& u0, int& u1) {
  u0 = (int)((long long)t.units * blockIdx.x / gridDim.x);
  u1 = (int)((long long)t.units * (blockIdx.x + 1) / gridDim.x);
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

// a sum of fp32 numbers with its rounding errors beside it
struct Sum {
  float s, c;
  __device__ __forceinline__ void add(float x, float more) {
    const float t = s + x, z = t - s;
    c += (s - (t - z)) + (x - z) + more;
    s = t;
  }
  __device__ __forceinline__ void over_warp() {
#pragma unroll
    for (int o = 16; o; o >>= 1) add(__shfl_xor_sync(0xffffffffu, s, o), __shfl_xor_sync(0xffffffffu, c, o));
  }
  // (the error of a sum that is not finite is not a number)
  __device__ double value() const { return isfinite(s) ? (double)s + (double)c : (double)s; }
};
// Squares of the values as they are, and of those whose squares would vanish or overflow times 2^100 and 2^-80: a group's
// sum below 2^-100 may have lost squares below 2^-126 (its values are below 2^-50, the smallest 2^-149); one above
// 2^90 loses with the factor what is 2^-50 of it.  What is not finite counts among the large ones.
struct Sums {
  Sum mid, low, high;
};
template <int N>
__device__ __forceinline__ float squares(const float (&x)[N], float by) {
  float s[4] = {};
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float y = x[j] * by;
    s[j % 4] = fmaf(y, y, s[j % 4]);
  }
  return (s[0] + s[1]) + (s[2] + s[3]);
}
template <int N>
__device__ __forceinline__ void add_squares(Sums& sums, const float (&x)[N]) {
  const float all = squares(x, 1.f);
  if (all >= 0x1p-100f && all <= 0x1p90f)
    sums.mid.add(all, 0.f);
  else if (all < 0x1p-100f)
    sums.low.add(squares(x, 0x1p100f), 0.f);
  else
    sums.high.add(squares(x, 0x1p-80f), 0.f);
}
template <bool BF>
__device__ __forceinline__ void add_vectors(Sums& sums, const uint4 (&r)[kVecs]) {
  constexpr int E = BF ? 8 : 4;
  float x[kVecs * E];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    float v[E];
    values<BF>(r[i], v);
#pragma unroll
    for (int j = 0; j < E; ++j) x[i * E + j] = v[j];
  }
  add_squares(sums, x);
}

// a unit of a tensor: its address and how many values it has
struct Unit {
  char* p;
  int n;
  bool bf16, aligned;
  __device__ Unit(const Entry& e, int u) {
    bf16 = e.size < 0;
    const int es = bf16 ? 2 : 4;
    const long long size = bf16 ? -e.size : e.size, e0 = (long long)(u - e.first) * (kClipUnit / es);
    p = static_cast<char*>(e.at) + e0 * es;
    n = (int)(size - e0 < kClipUnit / es ? size - e0 : kClipUnit / es);
    aligned = reinterpret_cast<uintptr_t>(e.at) % 16 == 0;
  }
  __device__ int whole() const { return aligned ? n / (bf16 ? 8 : 4) : 0; }  // vectors; the rest is taken value by value
  __device__ int rest() const { return whole() * (bf16 ? 8 : 4); }
  __device__ __forceinline__ void load(uint4 (&r)[kVecs]) const {
    const uint4* v = reinterpret_cast<const uint4*>(p) + threadIdx.x;
    const int left = whole() - (int)threadIdx.x;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      r[i] = make_uint4(0u, 0u, 0u, 0u);
      if (i * kThreads < left) r[i] = v[i * kThreads];
    }
  }
};

template <int N>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) clip_sum_kernel(const __grid_constant__ Table<N> t, double* part) {
  __shared__ Sum sh[3][kThreads / 32];
  depend_launch();
  int u0, u1;
  range_of(t, u0, u1);
  int i = tensor_of(t, u0);
  depend_wait();
  Sums sums{};
  for (int u = u0; u < u1; ++u) {
    while (i + 1 < t.n && u >= t.t[i + 1].first) ++i;
    const Unit x(t.t[i], u);
    uint4 r[kVecs];
    x.load(r);
    if (x.bf16)
      add_vectors<true>(sums, r);
    else
      add_vectors<false>(sums, r);
    for (int j = x.rest() + threadIdx.x; j < x.n; j += kThreads) {
      const float v[1] = {x.bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(x.p)[j])
                                 : reinterpret_cast<const float*>(x.p)[j]};
      add_squares(sums, v);
    }
  }
  const bool more = __syncthreads_or(!(sums.low.s == 0.f && sums.high.s == 0.f));  // (NaN is not 0)
  sums.mid.over_warp();
  if (more) sums.low.over_warp(), sums.high.over_warp();
  if (threadIdx.x % 32 == 0) {
    const int w = threadIdx.x / 32;
    sh[0][w] = sums.mid, sh[1][w] = sums.low, sh[2][w] = sums.high;
  }
  __syncthreads();
  if (threadIdx.x < 32) {  // (fp64 is slow: one warp's work)
    double d = 0.0;
    if (threadIdx.x < kThreads / 32) {
      d = sh[0][threadIdx.x].value();
      if (more) d += sh[1][threadIdx.x].value() * 0x1p-200 + sh[2][threadIdx.x].value() * 0x1p160;
    }
#pragma unroll
    for (int o = kThreads / 64; o; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if (threadIdx.x == 0) part[blockIdx.x] = d;
  }
}

template <bool BF>
__device__ __forceinline__ void scale(uint4& r, float by, float again) {
  constexpr int E = BF ? 8 : 4;
  float x[E];
  values<BF>(r, x);
#pragma unroll
  for (int j = 0; j < E; ++j) x[j] = x[j] * by * again;
  if (BF)
    r = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[E - 4], x[E - 3]),
                   pack_bf16x2(x[E - 2], x[E - 1]));
  else
    r = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}

// part: of all launches of clip_sum_kernel; read by every launch of this one
template <int N>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    clip_scale_kernel(const __grid_constant__ Table<N> t, const double* part, int parts, double limit, float* norm) {
  __shared__ float factor[2];
  depend_launch();
  int u0, u1;
  range_of(t, u0, u1);
  int i = u1 > u0 ? tensor_of(t, u1 - 1) : 0;
  depend_wait();
  uint4 r[kVecs];
  if (u1 > u0) Unit(t.t[i], u1 - 1).load(r);  // on its way while the norm is formed
  if (threadIdx.x < 32) {
    double d = 0.0;
#pragma unroll 4
    for (int j = threadIdx.x; j < parts; j += 32) d += part[j];
#pragma unroll
    for (int o = 16; o; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if (threadIdx.x == 0) {
      const double all = sqrt(d);
      if (norm && blockIdx.x == 0) *norm = (float)all;
      const bool clip = all > limit && !isinf(all);
      // a factor that is no normal fp32 number is applied in two steps; 2: not at all
      const double f = clip ? limit / all : 2.0;
      const bool tiny = f < 0x1p-100;
      factor[0] = tiny ? 0x1p-64f : (float)f;
      factor[1] = tiny ? (float)(f * 0x1p64) : 1.f;
    }
  }
  __syncthreads();
  const float by = factor[0], again = factor[1];
  if (by > 1.f) return;
  for (int u = u1 - 1; u >= u0; --u) {
    while (u < t.t[i].first) --i;
    const Unit x(t.t[i], u);
    if (u < u1 - 1) x.load(r);
    uint4* const v = reinterpret_cast<uint4*>(x.p) + threadIdx.x;
    const int left = x.whole() - (int)threadIdx.x;
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      if (x.bf16)
        scale<true>(r[k], by, again);
      else
        scale<false>(r[k], by, again);
      if (k * kThreads < left) __stcs(v + k * kThreads, r[k]);
    }
    for (int j = x.rest() + threadIdx.x; j < x.n; j += kThreads) {
      if (x.bf16) {
        __nv_bfloat16* y = reinterpret_cast<__nv_bfloat16*>(x.p) + j;
        *y = __float2bfloat16_rn(__bfloat162float(*y) * by * again);
      } else {
        float* y = reinterpret_cast<float*>(x.p) + j;
        *y = *y * by * again;
      }
    }
  }
}

// N: tensors of a launch at most
template <int N>
int launch_n(const ClipParams& p, cudaStream_t s) {
  Table<N> t;
  int parts = 0;
  // the tensors from i on that fit a launch; returns the next one
  auto fill = [&](int i) {
    t.n = 0;
    t.units = 0;  // (no more than 32 bits hold: refused before)
    for (; i < p.n && t.n < N; ++i) {
      const long long size = p.sizes[i];
      if (size == 0) continue;
      t.t[t.n++] = Entry{p.at[i], p.dtypes[i] == 1 ? -size : size, t.units, 0};
      t.units += (int)clip_units(size, p.dtypes[i]);
    }
    return i;
  };
  const long long most = (long long)kCtasPerSm * sm_count();
  auto grid = [&] { return (unsigned)(t.units < most ? t.units : most); };
  for (int i = 0; i < p.n;) {
    i = fill(i);
    if (t.n == 0) continue;
    const int e = launch_dependent(clip_sum_kernel<N>, grid(), kThreads, 0, s, t, p.part + parts);
    if (e != 0) return e;
    parts += (int)grid();
  }
  bool told = false;
  for (int i = 0; !told || (p.limit < INFINITY && i < p.n);) {
    i = fill(i);
    if (t.n == 0 && told) continue;
    // (without a limit, or without tensors, one CTA for the norm)
    const bool scale = p.limit < INFINITY && t.n > 0;
    if (!scale) t.n = 0, t.units = 0;
    const int e = launch_dependent(clip_scale_kernel<N>, scale ? grid() : 1u, kThreads, 0, s, t, (const double*)p.part,
                                   parts, (double)p.limit, told ? (float*)nullptr : p.norm);
    if (e != 0) return e;
    told = true;
  }
  return 0;
}

}  // namespace

int clip_parts(int n) { return (n / kClipTensors + 1) * kCtasPerSm * sm_count(); }

int launch_clip(const ClipParams& p, cudaStream_t s) {
  // (a table of 256 is 6 KB that every launch copies)
  return p.n <= 16 ? launch_n<16>(p, s) : launch_n<kClipTensors>(p, s);
}

}  // namespace srnn
