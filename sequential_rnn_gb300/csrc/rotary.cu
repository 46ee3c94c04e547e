// Norm of each query's and key's head with the rotation by its token's position, and the gradient.
//
//   y = x / sqrt(mean_d x^2 + eps) w;  pairs (y1, y2) of the first 2 n columns turn by the angle pos freqs[j]:
//   (y1 cos - y2 sin, y2 cos + y1 sin), the other columns stay.
//   gradient: g = the turned-back dy;  r = 1 / sqrt(..), xh = x r:
//   dx = r (w g - xh mean_d(w g xh)),  dw = sum over tokens and heads of g xh
//
// The angle is a whole number of 2^-64 turns: a frequency in turns, rounded to that, times the position, modulo
// 2^64, which is the fraction of a turn.  So the angle of any position is off by 2^-65 turns times the position, whatever
// the number of whole turns (in fp32 position 10^6 would be off by 2^-4 radians).  A frequency is a double
// (the caller's), its quotient by 2 pi is formed in two doubles.
//
// Bound by bytes.  A warp takes a token: the lanes of a head hold 8 columns each, in pairs, and the token's sines and
// cosines, taken once, serve all heads of q and k.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "lm.h"
#include "ptx.cuh"

namespace srnn {
namespace {

// 2^64 turns of a frequency in radians: f / (2 pi) in two doubles, the whole turns dropped
__device__ __forceinline__ unsigned long long turns(double f) {
  constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;  // 1 / (2 pi) and the rest of it
  const double hi = f * kHi, lo = fma(f, kHi, -hi) + f * kLo;
  const double frac = hi - rint(hi);  // exact, in [-1/2, 1/2]
  // (1/2 is 2^63, which wraps round to the same angle as -2^63)
  const long long a = frac == 0.5 ? (long long)(1ull << 63) : __double2ll_rn(frac * 0x1p64);
  return (unsigned long long)a + (unsigned long long)__double2ll_rn(lo * 0x1p64);
}
// cos and sin of pos times that
__device__ __forceinline__ void turn(unsigned long long f, long long pos, float& c, float& s) {
  const long long t = (long long)(f * (unsigned long long)pos);
  sincospif((float)t * 0x1p-63f, &s, &c);
}

__device__ __forceinline__ float get1(const float* p) { return *p; }
__device__ __forceinline__ float get1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void put1(float* p, float v) { *p = v; }
__device__ __forceinline__ void put1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// four neighbouring columns
struct Bf4 {
  uint2 v;
  __device__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint2*>(p); }
  __device__ void get(float* x) const { x[0] = bf16_lo(v.x), x[1] = bf16_hi(v.x), x[2] = bf16_lo(v.y), x[3] = bf16_hi(v.y); }
  static __device__ void store(__nv_bfloat16* p, const float* x) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
  }
};
struct F4 {
  float4 v;
  __device__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
  __device__ void get(float* x) const { x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w; }
  static __device__ void store(float* p, const float* x) { *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]); }
};
template <class T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> { typedef Bf4 type; };
template <>
struct Vec<float> { typedef F4 type; };

__device__ __forceinline__ long long position(const RotaryParams& p, unsigned t, unsigned b) {
  if (p.positions == nullptr) return t;
  return p.per_token ? p.positions[(long long)t * p.B + b] : (long long)p.positions[b] + t;
}

// A head's columns among LPH lanes: lane l of them holds two pieces of four columns at a0, a1 (l: valid where a0 >= 0)
// whose values are pairs: (x[i], x[4 + i]) or, INTER, (x[2 i], x[2 i + 1]).
template <int LPH, bool INTER>
struct Lanes {
  int l, sub, a0, a1, j0;  // lane within the head, the warp's head of it, columns, first pair's frequency (-1: not turned)
  __device__ explicit Lanes(const RotaryParams& p) {
    const int lane = threadIdx.x % 32;
    l = lane % LPH, sub = lane / LPH;
    const int c = 4 * l, half = p.rot / 2;
    if (INTER) {
      a0 = 2 * c, a1 = a0 + 4;
      j0 = 2 * c < p.rot ? c : -1;  // (the last one may be turned in part)
    } else if (c < half) {
      a0 = c, a1 = c + half, j0 = c;
    } else {
      a0 = p.rot + c - half, a1 = a0 + (p.D - p.rot) / 2, j0 = -1;
    }
    if (2 * c >= p.D) a0 = -1, j0 = -1;
  }
};
// frequencies that this lane computes: its pairs are shared out among the lanes of the other heads
template <int LPH>
struct Freqs {
  static constexpr int kHeads = 32 / LPH, kN = kHeads >= 4 ? 1 : 4 / kHeads;
  unsigned long long f[kN];
  template <class L>
  __device__ void load(const RotaryParams& p, const L& w) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int j = w.j0 + (w.sub * kN + i) % 4;
      f[i] = w.j0 >= 0 && j < p.rot / 2 ? turns(p.freqs[j]) : 0ull;
    }
  }
  template <class L>
  __device__ void at(const L& w, long long pos, float (&c)[4], float (&s)[4]) const {
    float cc[kN], ss[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) turn(f[i], pos, cc[i], ss[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = __shfl_sync(0xffffffffu, cc[i % kN], w.l + LPH * (i / kN));
      s[i] = __shfl_sync(0xffffffffu, ss[i % kN], w.l + LPH * (i / kN));
    }
  }
};

template <bool INTER>
__device__ __forceinline__ void rotate(float (&x)[8], const float (&c)[4], const float (&s)[4], float sign) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float &a = x[INTER ? 2 * i : i], &b = x[INTER ? 2 * i + 1 : 4 + i];
    const float sn = sign * s[i], y = fmaf(a, c[i], -b * sn), z = fmaf(b, c[i], a * sn);
    a = y, b = z;
  }
}
template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = LPH / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

constexpr int kBatch = 3;  // heads that a lane loads before it uses the first

template <class T, int LPH, bool INTER>
__global__ void __launch_bounds__(256) rotary_kernel(const RotaryParams p) {
  typedef typename Vec<T>::type V4;
  constexpr int HPW = 32 / LPH;
  depend_launch();
  const Lanes<LPH, INTER> w(p);
  depend_wait();
  Freqs<LPH> fr;
  fr.load(p, w);
  float wq[8], wk[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int at = (i < 4 ? w.a0 : w.a1 - 4) + i;
    wq[i] = p.qw && w.a0 >= 0 ? p.qw[at] : 1.f;
    wk[i] = p.kw && w.a0 >= 0 ? p.kw[at] : 1.f;
  }
  const int H = p.NQ + p.NK, groups = (H + HPW * kBatch - 1) / (HPW * kBatch);
  const int parts = p.split ? groups : 1;  // work items of a token
  const long long items = (long long)p.T * p.B * parts, stride = (long long)gridDim.x * (blockDim.x / 32);
  for (long long it = (long long)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32; it < items; it += stride) {
    const unsigned tb = (unsigned)(it / parts), part = (unsigned)(it % parts), t = tb / p.B, b = tb % p.B;
    const T* q = static_cast<const T*>(p.q) + t * p.qs[0] + b * p.qs[1];
    const T* k = static_cast<const T*>(p.k) + t * p.ks[0] + b * p.ks[1];
    T* qo = static_cast<T*>(p.qo) + (long long)tb * p.NQ * p.D;
    T* ko = static_cast<T*>(p.ko) + (long long)tb * p.NK * p.D;
    float c[4], s[4];
    bool have = false;
    for (int h0 = (p.split ? part * kBatch : 0) * HPW, end = p.split ? h0 + kBatch * HPW : H; h0 < min(end, H);
         h0 += kBatch * HPW) {
      V4 raw[kBatch][2];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int h = h0 + i * HPW + w.sub;
        if (h < H && w.a0 >= 0) {
          const T* x = h < p.NQ ? q + h * p.qs[2] : k + (h - p.NQ) * p.ks[2];
          raw[i][0].load(x + w.a0);
          raw[i][1].load(x + w.a1);
        }
      }
      if (!have) fr.at(w, position(p, t, b), c, s), have = true;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int h = h0 + i * HPW + w.sub;
        const bool on = h < H && w.a0 >= 0, isq = h < p.NQ;
        float x[8] = {};
        if (on) raw[i][0].get(x), raw[i][1].get(x + 4);
        if (p.qw) {
          float sum = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) sum = fmaf(x[j], x[j], sum);
          const float r = rsqrtf(head_sum<LPH>(sum) / p.D + p.eps);
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] *= r * (isq ? wq[j] : wk[j]);
        }
        rotate<INTER>(x, c, s, 1.f);
        if (on) {
          T* o = isq ? qo + h * p.D : ko + (h - p.NQ) * p.D;
          V4::store(o + w.a0, x);
          V4::store(o + w.a1, x + 4);
        }
      }
    }
  }
}

// dw's partial sums: a row of 2 D for each CTA (q's, then k's)
template <class T, int LPH, bool INTER>
__global__ void __launch_bounds__(256) rotary_bwd_kernel(const RotaryParams p) {
  typedef typename Vec<T>::type V4;
  constexpr int HPW = 32 / LPH, W = 8;
  __shared__ float part[W][2][LPH * 8];
  depend_launch();
  const Lanes<LPH, INTER> w(p);
  depend_wait();
  Freqs<LPH> fr;
  fr.load(p, w);
  float wq[8], wk[8], gq[8] = {}, gk[8] = {};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int at = (i < 4 ? w.a0 : w.a1 - 4) + i;
    wq[i] = p.qw && w.a0 >= 0 ? p.qw[at] : 1.f;
    wk[i] = p.kw && w.a0 >= 0 ? p.kw[at] : 1.f;
  }
  const int H = p.NQ + p.NK, warp = threadIdx.x / 32;
  const long long items = (long long)p.T * p.B, stride = (long long)gridDim.x * W;
  for (long long tb = (long long)blockIdx.x * W + warp; tb < items; tb += stride) {
    const unsigned t = (unsigned)tb / p.B, b = (unsigned)tb % p.B;
    const T* q = static_cast<const T*>(p.q) + t * p.qs[0] + b * p.qs[1];
    const T* k = static_cast<const T*>(p.k) + t * p.ks[0] + b * p.ks[1];
    const T* dq = static_cast<const T*>(p.dq) + t * p.dqs[0] + b * p.dqs[1];
    const T* dk = static_cast<const T*>(p.dk) + t * p.dks[0] + b * p.dks[1];
    T* qo = static_cast<T*>(p.qo) + tb * p.NQ * p.D;
    T* ko = static_cast<T*>(p.ko) + tb * p.NK * p.D;
    float c[4], s[4];
    fr.at(w, position(p, t, b), c, s);
    for (int h0 = 0; h0 < H; h0 += HPW) {
      const int h = h0 + w.sub;
      const bool on = h < H && w.a0 >= 0, isq = h < p.NQ;
      float x[8] = {}, g[8] = {};
      if (on) {
        V4 raw[4];
        const T* xp = isq ? q + h * p.qs[2] : k + (h - p.NQ) * p.ks[2];
        const T* gp = isq ? dq + h * p.dqs[2] : dk + (h - p.NQ) * p.dks[2];
        raw[0].load(xp + w.a0), raw[1].load(xp + w.a1), raw[2].load(gp + w.a0), raw[3].load(gp + w.a1);
        raw[0].get(x), raw[1].get(x + 4), raw[2].get(g), raw[3].get(g + 4);
      }
      rotate<INTER>(g, c, s, -1.f);
      if (p.qw) {
        float sum = 0.f, along = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          sum = fmaf(x[j], x[j], sum);
          along = fmaf(g[j] * (isq ? wq[j] : wk[j]), x[j], along);
        }
        const float r = rsqrtf(head_sum<LPH>(sum) / p.D + p.eps);
        const float m = head_sum<LPH>(along) * r * r / p.D;  // mean(w g xh) r
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float gw = g[j] * (isq ? wq[j] : wk[j]);
          if (isq)
            gq[j] = fmaf(g[j], x[j] * r, gq[j]);
          else
            gk[j] = fmaf(g[j], x[j] * r, gk[j]);
          g[j] = r * fmaf(-m, x[j], gw);
        }
      }
      if (on) {
        T* o = isq ? qo + h * p.D : ko + (h - p.NQ) * p.D;
        V4::store(o + w.a0, g);
        V4::store(o + w.a1, g + 4);
      }
    }
  }
  if (!p.qw) return;
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int o = LPH; o < 32; o <<= 1) {
      gq[j] += __shfl_xor_sync(0xffffffffu, gq[j], o);
      gk[j] += __shfl_xor_sync(0xffffffffu, gk[j], o);
    }
  if (w.sub == 0 && w.a0 >= 0)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int at = (j < 4 ? w.a0 : w.a1 - 4) + j;
      part[warp][0][at] = gq[j];
      part[warp][1][at] = gk[j];
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * p.D; i += blockDim.x) {
    float v = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) v += part[j][i / p.D][i % p.D];
    p.part[(long long)blockIdx.x * 2 * p.D + i] = v;
  }
}

// The same for any even head size, value by value: a CTA of one warp takes a head of a token at a time.
// (Gradient: the CTA's dw stays in shared memory; its threads own the columns of their pairs.)
template <class T, bool BWD>
__global__ void __launch_bounds__(32) rotary_any_kernel(const RotaryParams p) {
  extern __shared__ float acc[];  // [2][D]
  depend_launch();
  depend_wait();
  const int H = p.NQ + p.NK, half = p.rot / 2, lane = threadIdx.x, rest = (p.D - p.rot) / 2;
  if (BWD && p.qw)
    for (int i = lane; i < 2 * p.D; i += 32) acc[i] = 0.f;
  __syncwarp();
  auto columns = [&](int i, int& a, int& b) {  // of pair i; pairs past rot / 2 do not turn
    if (p.interleaved)
      a = 2 * i, b = a + 1;
    else if (i < half)
      a = i, b = i + half;
    else
      a = p.rot + i - half, b = a + rest;
  };
  const long long items = (long long)p.T * p.B * H;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const unsigned tb = (unsigned)(it / H), t = tb / p.B, b = tb % p.B;
    const int hh = (int)(it % H), h = hh < p.NQ ? hh : hh - p.NQ;
    const bool isq = hh < p.NQ;
    const long long* xs = isq ? p.qs : p.ks;
    const T* x = static_cast<const T*>(isq ? p.q : p.k) + t * xs[0] + b * xs[1] + h * xs[2];
    const long long* gs = isq ? p.dqs : p.dks;
    const T* g = BWD ? static_cast<const T*>(isq ? p.dq : p.dk) + t * gs[0] + b * gs[1] + h * gs[2] : nullptr;
    T* o = static_cast<T*>(isq ? p.qo : p.ko) + ((long long)tb * (isq ? p.NQ : p.NK) + h) * p.D;
    const float* w = isq ? p.qw : p.kw;
    const long long pos = position(p, t, b);
    float sum = 0.f, along = 0.f;
    for (int i = lane; i < p.D / 2; i += 32) {
      int ia, ib;
      columns(i, ia, ib);
      const float xa = get1(x + ia), xb = get1(x + ib);
      sum = fmaf(xa, xa, fmaf(xb, xb, sum));
      if (BWD && w) {
        float c = 1.f, s = 0.f, ga = get1(g + ia), gb = get1(g + ib);
        if (i < half) turn(turns(p.freqs[i]), pos, c, s);
        along = fmaf(fmaf(ga, c, gb * s) * w[ia], xa, fmaf(fmaf(gb, c, -ga * s) * w[ib], xb, along));
      }
    }
    const float r = w ? rsqrtf(head_sum<32>(sum) / p.D + p.eps) : 1.f;
    const float m = BWD && w ? head_sum<32>(along) * r * r / p.D : 0.f;
    for (int i = lane; i < p.D / 2; i += 32) {
      int ia, ib;
      columns(i, ia, ib);
      const float wa = w ? w[ia] : 1.f, wb = w ? w[ib] : 1.f, xa = get1(x + ia), xb = get1(x + ib);
      float c = 1.f, s = 0.f;
      if (i < half) turn(turns(p.freqs[i]), pos, c, s);
      if (BWD) {
        const float ya = get1(g + ia), yb = get1(g + ib), ga = fmaf(ya, c, yb * s), gb = fmaf(yb, c, -ya * s);
        if (w) {
          float* to = acc + (isq ? 0 : p.D);
          to[ia] = fmaf(ga, xa * r, to[ia]);
          to[ib] = fmaf(gb, xb * r, to[ib]);
        }
        put1(o + ia, r * fmaf(-m, xa, ga * wa));
        put1(o + ib, r * fmaf(-m, xb, gb * wb));
      } else {
        const float ya = xa * (r * wa), yb = xb * (r * wb);
        put1(o + ia, fmaf(ya, c, -yb * s));
        put1(o + ib, fmaf(yb, c, ya * s));
      }
    }
  }
  if (BWD && p.qw) {
    __syncwarp();
    for (int i = lane; i < 2 * p.D; i += 32) p.part[(long long)blockIdx.x * 2 * p.D + i] = acc[i];
  }
}

// dw[i] = sum of the CTAs' parts, in their order: a warp for each column
__global__ void __launch_bounds__(256) rotary_dw_kernel(const float* part, float* dqw, float* dkw, int parts, int D) {
  depend_launch();
  depend_wait();
  const int i = blockIdx.x * 8 + threadIdx.x / 32, lane = threadIdx.x % 32;
  if (i >= 2 * D) return;
  float v = 0.f;
  for (int j = lane; j < parts; j += 32) v += part[(long long)j * 2 * D + i];
  v = head_sum<32>(v);
  if (lane == 0) (i < D ? dqw : dkw)[i % D] = v;
}

bool at16(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool strides4(const long long (&s)[3]) { return s[0] % 4 == 0 && s[1] % 4 == 0 && s[2] % 4 == 0; }

// two pieces of four columns a lane need sizes and addresses that are multiples of four values (half layout: of a turned
// part that is, too)
template <class T>
bool vector_form(const RotaryParams& p, bool bwd) {
  constexpr size_t A = 4 * sizeof(T);
  bool ok = p.D % 8 == 0 && p.D <= 256 && (p.interleaved || p.rot % 8 == 0) && strides4(p.qs) && strides4(p.ks) &&
            at16(p.q, A) && at16(p.k, A) && at16(p.qo, A) && at16(p.ko, A);
  if (bwd) ok = ok && strides4(p.dqs) && strides4(p.dks) && at16(p.dq, A) && at16(p.dk, A);
  return ok;
}

int bwd_ctas(long long items, int per) {
  const long long want = (items + per - 1) / per;
  return (int)(want < kRotaryParts ? want : kRotaryParts);
}

template <class T, int LPH, bool INTER>
int launch_vec(RotaryParams& p, bool bwd, cudaStream_t s) {
  const long long tokens = (long long)p.T * p.B;
  if (bwd) {
    const int grid = bwd_ctas(tokens, 8);
    const int e = launch_dependent(rotary_bwd_kernel<T, LPH, INTER>, (unsigned)grid, 256, 0, s, (const RotaryParams)p);
    if (e != 0 || !p.qw) return e;
    return launch_dependent(rotary_dw_kernel, (unsigned)((2 * p.D + 7) / 8), 256, 0, s, (const float*)p.part, p.dqw,
                            p.dkw, grid, p.D);
  }
  const int groups = (p.NQ + p.NK + 32 / LPH * kBatch - 1) / (32 / LPH * kBatch);
  p.split = tokens < 8LL * sm_count();
  const long long want = (tokens * (p.split ? groups : 1) + 7) / 8, most = 6LL * sm_count();
  return launch_dependent(rotary_kernel<T, LPH, INTER>, (unsigned)(want < most ? want : most), 256, 0, s,
                          (const RotaryParams)p);
}
template <class T, int LPH>
int launch_l(RotaryParams& p, bool bwd, cudaStream_t s) {
  return p.interleaved ? launch_vec<T, LPH, true>(p, bwd, s) : launch_vec<T, LPH, false>(p, bwd, s);
}
template <class T>
int launch_t(RotaryParams& p, bool bwd, cudaStream_t s) {
  if (vector_form<T>(p, bwd)) {
    if (p.D <= 32) return launch_l<T, 4>(p, bwd, s);
    if (p.D <= 64) return launch_l<T, 8>(p, bwd, s);
    if (p.D <= 128) return launch_l<T, 16>(p, bwd, s);
    return launch_l<T, 32>(p, bwd, s);
  }
  const long long items = (long long)p.T * p.B * (p.NQ + p.NK);
  if (!bwd) {
    const long long most = 32LL * sm_count();
    return launch_dependent(rotary_any_kernel<T, false>, (unsigned)(items < most ? items : most), 32, 0, s,
                            (const RotaryParams)p);
  }
  const int grid = bwd_ctas(items, 1);
  const int e = launch_dependent(rotary_any_kernel<T, true>, (unsigned)grid, 32, p.qw ? 8 * (size_t)p.D : 0, s,
                                 (const RotaryParams)p);
  if (e != 0 || !p.qw) return e;
  return launch_dependent(rotary_dw_kernel, (unsigned)((2 * p.D + 7) / 8), 256, 0, s, (const float*)p.part, p.dqw, p.dkw,
                          grid, p.D);
}

}  // namespace

int launch_rotary(RotaryParams p, bool bf16, bool bwd, cudaStream_t s) {
  return bf16 ? launch_t<__nv_bfloat16>(p, bwd, s) : launch_t<float>(p, bwd, s);
}

}  // namespace srnn
