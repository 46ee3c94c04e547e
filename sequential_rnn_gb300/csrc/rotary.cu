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
// Bound by bytes, and issue slots beside them: 16384 tokens of 12 + 12 x 64 heads in bf16 take 19.7 us, 5.1 TB/s.  A warp takes a
// token: the lanes of a head hold 8 columns each, in pairs, and the token's sines and cosines, taken once, serve all its
// heads.  Few tokens are bound by the launch and one pass of latencies: 16 of them 3.5 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "lm.h"
#include "num.cuh"
#include "ptx.cuh"

namespace srnn {
namespace {

// 2^64 turns of a frequency in radians: f / (2 pi) in two doubles, the whole turns dropped
__device__ __forceinline__ unsigned long long turns(double f) {
  constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;  // 1 / (2 pi) and the rest of it
  const double hi = f * kHi, lo = ::fma(f, kHi, -hi) + f * kLo;
  const double frac = hi - rint(hi);  // exact, in [-1/2, 1/2]
  // (1/2 is 2^63, which wraps round to the same angle as -2^63)
  const long long a = frac == 0.5 ? (long long)(1ull << 63) : __double2ll_rn(frac * 0x1p64);
  return (unsigned long long)a + (unsigned long long)__double2ll_rn(lo * 0x1p64);
}
// cos and sin of pos times that: the quarter turn nearest to the angle, and the Taylor series of the rest (at most 1/8 of a
// turn, formed from 32 bits: off by less than 2^-31) up to x^9 and x^10, which leave out less than 2 10^-9
__device__ __forceinline__ void turn(unsigned long long f, long long pos, float& c, float& s) {
  const uint32_t u = (uint32_t)((f * (unsigned long long)pos) >> 32), q = (u + 0x20000000u) >> 30;
  const float x = (float)(int)(u - (q << 30)) * 0x1.921fb6p-30f;  // 2 pi 2^-32
  const float z = x * x;
  const float sx = fmaf(x * z, fmaf(z, fmaf(z, fmaf(z, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f), x);
  const float cx = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f), -0.5f), 1.f);
  const float cc = q & 1 ? sx : cx, ss = q & 1 ? cx : sx;
  c = (q + 1) & 2 ? -cc : cc;
  s = q & 2 ? -ss : ss;
}

__device__ __forceinline__ float get1(const float* p) { return *p; }
__device__ __forceinline__ float get1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void put1(float* p, float v) { *p = v; }
__device__ __forceinline__ void put1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ long long position(const RotaryParams& p, unsigned t, unsigned b) {
  if (p.positions == nullptr) return t;
  return p.per_token ? p.positions[(long long)t * p.B + b] : (long long)p.positions[b] + t;
}

// A head among LPH lanes, four pairs of columns each: how a lane reaches them.
//   kHalf   pairs (j, j + rot / 2): two pieces of four neighbouring columns (past rot, two of what is not turned)
//   kNext   pairs (2 j, 2 j + 1): eight neighbouring columns, all turned or none
//   kSome   the same where one lane of a head has both (rot no multiple of 8)
//   kAny    either, pairs LPH apart, value by value: sizes and addresses that are no multiples of four values
enum : int { kHalf = 0, kNext = 1, kAny = 2, kSome = 3 };

template <class T, int MODE>
struct Head;  // a lane's raw values
template <>
struct Head<__nv_bfloat16, kHalf> {
  uint2 a, b;
};
template <>
struct Head<__nv_bfloat16, kNext> {
  uint2 a, b;
};
template <>
struct Head<float, kHalf> {
  float4 a, b;
};
template <>
struct Head<float, kNext> {
  float4 a, b;
};
template <class T>
struct Head<T, kSome> : Head<T, kNext> {};
template <class T>
struct Head<T, kAny> {
  T a[4], b[4];
};

// two pairs' first values, and their second ones; twice
struct Pairs {
  Num<2> a[2], b[2];
};

template <int LPH, int MODE>
struct Lanes {
  static constexpr bool NEXT = MODE == kNext || MODE == kSome;
  int l, sub;    // lane of the head, the warp's head of it
  int a0, gap;   // vector forms: first column, from the first piece to the second
  int half, D;
  bool inter, on;
  bool swap;     // kHalf: the pair's second value first
  int live;      // so many of the lane's pairs turn, the first ones
  bool mixed;    // some lanes have pairs of both kinds (the same for all)
  __device__ explicit Lanes(const RotaryParams& p) {
    const int lane = threadIdx.x % 32;
    l = lane % LPH, sub = lane / LPH;
    half = p.rot / 2, D = p.D, inter = p.interleaved;
    a0 = 0, gap = 4;
    on = 8 * l < D;
    if (NEXT) {
      a0 = 8 * l;
    } else if (MODE == kHalf) {
      if (4 * l < half)
        a0 = 4 * l, gap = half;
      else
        a0 = 4 * l + half, gap = (D - 2 * half) / 2;
    } else {
      on = l < D / 2;
    }
    if (!on && MODE != kAny) a0 = 0;
    swap = false;
    live = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) live += pair(i) < half ? 1 : 0;
    mixed = MODE == kAny ? p.rot < D : MODE == kSome;
    if (!mixed && MODE == kAny) live = 4;
  }
  // The lanes of some heads read their pieces in the other order, so that those that shared memory serves at once
  // (128 bytes) lie in different banks.  row: bytes of a head
  __device__ void spread(int row) {
    if (MODE != kHalf || ((sub * row) >> 7 & 1) == 0) return;
    a0 += gap, gap = -gap;
    swap = true;
  }
  __device__ int step() const { return NEXT ? 4 : gap; }
  // index of the lane's pair i; pairs below `half` turn
  __device__ int pair(int i) const { return MODE == kAny ? l + LPH * i : 4 * l + i; }
  __device__ void columns(int i, int& a, int& b) const {  // kAny
    const int j = pair(i);
    if (inter)
      a = 2 * j, b = a + 1;
    else if (j < half)
      a = j, b = j + half;
    else
      a = j + half, b = a + D / 2 - half;
  }
  template <class T>
  __device__ void load(Head<T, MODE>& h, const T* x) const {
    if constexpr (MODE == kAny) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        int a, b;
        columns(i, a, b);
        const bool in = pair(i) < D / 2;
        h.a[i] = in ? x[a] : T(0.f);
        h.b[i] = in ? x[b] : T(0.f);
      }
    } else {
      h.a = *reinterpret_cast<const decltype(h.a)*>(x + a0);
      h.b = *reinterpret_cast<const decltype(h.b)*>(x + a0 + step());
    }
  }
  template <class T>
  __device__ Pairs get(const Head<T, MODE>& h) const {
    Pairs r;
    float v[8];
    if constexpr (MODE == kAny) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = get1(&h.a[i]), v[4 + i] = get1(&h.b[i]);
    } else {
      float y[8];
      if constexpr (sizeof(T) == 2) {
        const uint32_t w[4] = {h.a.x, h.a.y, h.b.x, h.b.y};
#pragma unroll
        for (int i = 0; i < 4; ++i) y[2 * i] = bf16_lo(w[i]), y[2 * i + 1] = bf16_hi(w[i]);
      } else {
        y[0] = h.a.x, y[1] = h.a.y, y[2] = h.a.z, y[3] = h.a.w, y[4] = h.b.x, y[5] = h.b.y, y[6] = h.b.z, y[7] = h.b.w;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = y[NEXT ? 2 * i : i], v[4 + i] = y[NEXT ? 2 * i + 1 : 4 + i];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) r.a[i].x = make_float2(v[2 * i], v[2 * i + 1]), r.b[i].x = make_float2(v[4 + 2 * i], v[5 + 2 * i]);
    return r;
  }
  template <class T>
  __device__ void store(T* x, const Pairs& r) const {
    const float a[4] = {r.a[0].x.x, r.a[0].x.y, r.a[1].x.x, r.a[1].x.y};
    const float b[4] = {r.b[0].x.x, r.b[0].x.y, r.b[1].x.x, r.b[1].x.y};
    if constexpr (MODE == kAny) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        int ia, ib;
        columns(i, ia, ib);
        if (pair(i) < D / 2) put1(x + ia, a[i]), put1(x + ib, b[i]);
      }
    } else {
      float y[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) y[NEXT ? 2 * i : i] = a[i], y[NEXT ? 2 * i + 1 : 4 + i] = b[i];
      if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint2*>(x + a0) = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
        *reinterpret_cast<uint2*>(x + a0 + step()) = make_uint2(pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
      } else {
        *reinterpret_cast<float4*>(x + a0) = make_float4(y[0], y[1], y[2], y[3]);
        *reinterpret_cast<float4*>(x + a0 + step()) = make_float4(y[4], y[5], y[6], y[7]);
      }
    }
  }
  // the lane's weights, from shared memory (what lanes without columns get does not matter)
  __device__ Pairs weights(const float* w) const {
    Pairs r;
    float a[4], b[4];
    if constexpr (MODE == kAny) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        int ia, ib;
        columns(i, ia, ib);
        const bool in = pair(i) < D / 2;
        a[i] = in ? w[ia] : 0.f, b[i] = in ? w[ib] : 0.f;
      }
    } else {
      const float4 x = *reinterpret_cast<const float4*>(w + a0), y = *reinterpret_cast<const float4*>(w + a0 + step());
      const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = v[NEXT ? 2 * i : i], b[i] = v[NEXT ? 2 * i + 1 : 4 + i];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) r.a[i].x = make_float2(a[2 * i], a[2 * i + 1]), r.b[i].x = make_float2(b[2 * i], b[2 * i + 1]);
    return r;
  }
  __device__ void add_to(float* sum, const Pairs& r) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int a, b;
      if (MODE == kAny)
        columns(i, a, b);
      else
        a = NEXT ? a0 + 2 * i : a0 + i, b = NEXT ? a + 1 : a + gap;
      if (on && pair(i) < D / 2) sum[a] = r.a[i / 2].get(i % 2), sum[b] = r.b[i / 2].get(i % 2);
    }
  }
};

struct Turn {
  Num<2> c[2], s[2], n[2];  // cos, sin, -sin of the lane's four pairs
};
// a token's: the lanes that hold the same pairs of different heads share them out
template <class L, int LPH>
__device__ __forceinline__ Turn turn_of(const L& w, const unsigned long long* freqs, long long pos) {
  constexpr int HEADS = 32 / LPH, N = HEADS >= 4 ? 1 : 4 / HEADS;
  float cc[N], ss[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int j = w.pair((w.sub * N + i) % 4);
    cc[i] = 1.f, ss[i] = 0.f;
    if (j < w.half) turn(freqs[j], pos, cc[i], ss[i]);
  }
  Turn t;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float c = __shfl_sync(0xffffffffu, cc[i % N], w.l + LPH * (i / N));
    const float s = __shfl_sync(0xffffffffu, ss[i % N], w.l + LPH * (i / N));
    t.c[i / 2].set(i % 2, c), t.s[i / 2].set(i % 2, w.swap ? -s : s), t.n[i / 2].set(i % 2, w.swap ? s : -s);
  }
  return t;
}
// Pairs that do not turn keep their values: zero times the other one would be NaN where that is not finite.  (The lane's
// predicate costs nothing measurable, 1024 x 16 tokens of 12 x 64 19.6 us; a test of each pair where kNext needs none 20.5.)
template <int LPH, int MODE>
__device__ __forceinline__ void rotate(const Lanes<LPH, MODE>& w, Pairs& x, const Num<2> (&c)[2], const Num<2> (&s)[2],
                                       const Num<2> (&n)[2]) {
  auto two = [&](int i) {
    const Num<2> a = x.a[i], b = x.b[i];
    x.a[i] = fma(b, n[i], a * c[i]);
    x.b[i] = fma(a, s[i], b * c[i]);
  };
  if (MODE == kHalf || MODE == kNext || !w.mixed) {
    if (w.live > 0) {
      two(0);
      two(1);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (w.live > 2 * i) {
        const float a = x.a[i].get(1), b = x.b[i].get(1);
        two(i);
        if (w.live == 2 * i + 1) x.a[i].set(1, a), x.b[i].set(1, b);
      }
  }
}
__device__ __forceinline__ float dot(const Pairs& x, const Pairs& y) {
  const Num<2> s = fma(x.b[1], y.b[1], x.b[0] * y.b[0]) + fma(x.a[1], y.a[1], x.a[0] * y.a[0]);
  return s.x.x + s.x.y;
}
template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = LPH / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// over the lanes that hold the same pairs of different heads
template <int LPH>
__device__ __forceinline__ void sum_lanes(Pairs& x) {
#pragma unroll
  for (int o = LPH; o < 32; o <<= 1)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        x.a[j].set(v, x.a[j].get(v) + __shfl_xor_sync(0xffffffffu, x.a[j].get(v), o));
        x.b[j].set(v, x.b[j].get(v) + __shfl_xor_sync(0xffffffffu, x.b[j].get(v), o));
      }
}

constexpr int kMaxPairs = 128;  // of a head that lanes hold: D up to 256

// What a CTA keeps: the frequencies in turns (the double arithmetic once, not for each warp), the weights
struct Consts {
  unsigned long long freqs[kMaxPairs];
  alignas(16) float w[2][2 * kMaxPairs];
  __device__ void load(const RotaryParams& p) {
    for (int i = threadIdx.x; i < p.rot / 2; i += blockDim.x) freqs[i] = turns(p.freqs[i]);
    for (int i = threadIdx.x; i < p.D; i += blockDim.x) w[0][i] = p.qw ? p.qw[i] : 1.f, w[1][i] = p.kw ? p.kw[i] : 1.f;
    __syncthreads();
  }
};
// Items: whole tokens, or (p.split) the batches of heads of a token one by one
struct Items {
  long long n, at, step;
  int groups, nbq;
  template <int HEADS>
  __device__ static Items of(const RotaryParams& p) {
    Items r;
    r.nbq = (p.NQ + HEADS - 1) / HEADS;
    r.groups = r.nbq + (p.NK + HEADS - 1) / HEADS;
    r.n = (long long)p.T * p.B * (p.split ? r.groups : 1);
    r.at = (long long)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
    r.step = (long long)gridDim.x * (blockDim.x / 32);
    return r;
  }
};

constexpr int kRingTokens = 16, kRingTokensBwd = 8;  // for each SM
constexpr size_t kRingMost = 200 * 1024;             // bytes of a CTA's rings
constexpr int kBatch = 3, kBatchBwd = 2;  // heads that a lane loads before it uses the first

template <class T, int LPH, int MODE>
__global__ void __launch_bounds__(256, 3) rotary_kernel(const RotaryParams p) {
  constexpr int HPW = 32 / LPH;
  __shared__ Consts sh;
  depend_launch();
  const Lanes<LPH, MODE> w(p);
  depend_wait();
  sh.load(p);
  const Pairs wq = w.weights(sh.w[0]), wk = w.weights(sh.w[1]);
  const float inv = 1.f / p.D;
  Items it = Items::of<HPW * kBatch>(p);
  for (; it.at < it.n; it.at += it.step) {
    const unsigned tb = p.split ? (unsigned)(it.at / it.groups) : (unsigned)it.at, t = tb / p.B, b = tb % p.B;
    const int g0 = p.split ? (int)(it.at % it.groups) : 0, g1 = p.split ? g0 + 1 : it.groups;
    Turn tn;
    bool have = false;
    auto heads = [&](const T* x, long long hs, T* o, int h0, int n, const Pairs& wt) {
      Head<T, MODE> raw[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int h = h0 + i * HPW + w.sub;
        raw[i] = Head<T, MODE>{};
        if (w.on && h < n) w.load(raw[i], x + h * hs);
      }
      if (!have) tn = turn_of<Lanes<LPH, MODE>, LPH>(w, sh.freqs, position(p, t, b)), have = true;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (h0 + i * HPW >= n) break;
        const int h = h0 + i * HPW + w.sub;
        Pairs y = w.get(raw[i]);
        if (p.qw) {
          const Num<2> r(rsqrtf(fmaf(head_sum<LPH>(dot(y, y)), inv, p.eps)));
#pragma unroll
          for (int j = 0; j < 2; ++j) y.a[j] = y.a[j] * (r * wt.a[j]), y.b[j] = y.b[j] * (r * wt.b[j]);
        }
        rotate(w, y, tn.c, tn.s, tn.n);
        if (w.on && h < n) w.store(o + (long long)h * p.D, y);
      }
    };
    for (int g = g0; g < g1; ++g) {
      if (g < it.nbq)
        heads(static_cast<const T*>(p.q) + t * p.qs[0] + b * p.qs[1], p.qs[2], static_cast<T*>(p.qo) + (long long)tb * p.NQ * p.D,
              g * HPW * kBatch, p.NQ, wq);
      else
        heads(static_cast<const T*>(p.k) + t * p.ks[0] + b * p.ks[1], p.ks[2], static_cast<T*>(p.ko) + (long long)tb * p.NK * p.D,
              (g - it.nbq) * HPW * kBatch, p.NK, wk);
    }
  }
}

// dw's partial sums: a row of 2 D for each CTA (q's, then k's)
template <class T, int LPH, int MODE>
__global__ void __launch_bounds__(256, 2) rotary_bwd_kernel(const RotaryParams p) {
  constexpr int HPW = 32 / LPH, W = 8;
  __shared__ Consts sh;
  __shared__ float part[W][2][LPH * 8];
  depend_launch();
  const Lanes<LPH, MODE> w(p);
  depend_wait();
  sh.load(p);
  const Pairs wq = w.weights(sh.w[0]), wk = w.weights(sh.w[1]);
  const float inv = 1.f / p.D;
  Pairs sq, sk;
#pragma unroll
  for (int j = 0; j < 2; ++j) sq.a[j] = sq.b[j] = sk.a[j] = sk.b[j] = Num<2>(0.f);
  Items it = Items::of<HPW * kBatchBwd>(p);
  for (; it.at < it.n; it.at += it.step) {
    const unsigned tb = p.split ? (unsigned)(it.at / it.groups) : (unsigned)it.at, t = tb / p.B, b = tb % p.B;
    const int g0 = p.split ? (int)(it.at % it.groups) : 0, g1 = p.split ? g0 + 1 : it.groups;
    Turn tn;
    bool have = false;
    auto heads = [&](const T* x, long long hs, const T* d, long long ds, T* o, int h0, int n, const Pairs& wt, Pairs& sum) {
      Head<T, MODE> rx[kBatchBwd], rd[kBatchBwd];
#pragma unroll
      for (int i = 0; i < kBatchBwd; ++i) {
        const int h = h0 + i * HPW + w.sub;
        rx[i] = Head<T, MODE>{}, rd[i] = Head<T, MODE>{};
        if (w.on && h < n) w.load(rx[i], x + h * hs), w.load(rd[i], d + h * ds);
      }
      if (!have) tn = turn_of<Lanes<LPH, MODE>, LPH>(w, sh.freqs, position(p, t, b)), have = true;
#pragma unroll
      for (int i = 0; i < kBatchBwd; ++i) {
        if (h0 + i * HPW >= n) break;
        const int h = h0 + i * HPW + w.sub;
        Pairs g = w.get(rd[i]);
        rotate(w, g, tn.c, tn.n, tn.s);  // back
        if (p.qw) {
          const Pairs v = w.get(rx[i]);
          Pairs gw;
#pragma unroll
          for (int j = 0; j < 2; ++j) gw.a[j] = g.a[j] * wt.a[j], gw.b[j] = g.b[j] * wt.b[j];
          const float r = rsqrtf(fmaf(head_sum<LPH>(dot(v, v)), inv, p.eps));
          const Num<2> m(-(head_sum<LPH>(dot(gw, v)) * inv) * r * r), rr(r);  // - mean(w g xh) r
          if (h < n)  // (others have zeros for x: with eps = 0 an infinite r, whose product is not a number)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              sum.a[j] = fma(g.a[j], v.a[j] * rr, sum.a[j]);
              sum.b[j] = fma(g.b[j], v.b[j] * rr, sum.b[j]);
            }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            g.a[j] = rr * fma(m, v.a[j], gw.a[j]);
            g.b[j] = rr * fma(m, v.b[j], gw.b[j]);
          }
        }
        if (w.on && h < n) w.store(o + (long long)h * p.D, g);
      }
    };
    for (int g = g0; g < g1; ++g) {
      if (g < it.nbq)
        heads(static_cast<const T*>(p.q) + t * p.qs[0] + b * p.qs[1], p.qs[2],
              static_cast<const T*>(p.dq) + t * p.dqs[0] + b * p.dqs[1], p.dqs[2],
              static_cast<T*>(p.qo) + (long long)tb * p.NQ * p.D, g * HPW * kBatchBwd, p.NQ, wq, sq);
      else
        heads(static_cast<const T*>(p.k) + t * p.ks[0] + b * p.ks[1], p.ks[2],
              static_cast<const T*>(p.dk) + t * p.dks[0] + b * p.dks[1], p.dks[2],
              static_cast<T*>(p.ko) + (long long)tb * p.NK * p.D, (g - it.nbq) * HPW * kBatchBwd, p.NK, wk, sk);
    }
  }
  if (!p.qw) return;
  sum_lanes<LPH>(sq);
  sum_lanes<LPH>(sk);
  const int warp = threadIdx.x / 32;
  if (w.sub == 0) w.add_to(part[warp][0], sq), w.add_to(part[warp][1], sk);
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * p.D; i += blockDim.x) {
    float v = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) v += part[j][i / p.D][i % p.D];
    p.part[(long long)blockIdx.x * 2 * p.D + i] = v;
  }
}

// Many tokens, heads of 32, 64, 128 or 256 at 16-byte addresses: asynchronous copies bring what a warp takes next into a ring
// of its own in shared memory, so that it is on its way while the warp works and no register holds it (two on
// their way, with fewer CTAs on an SM, are no faster: 1024 x 16 tokens of 12 + 12 x 64 heads 20.8 us against 19.6, 1024 x 8 of
// 16 + 8 x 128 30.9 against 22.5).  A sweep is what the warp takes at once: 32 / LPH heads.
template <class T, int LPH>
struct Ring {
  static constexpr int HPW = 32 / LPH, D = 8 * LPH, SWEEP = 32 * 8 * sizeof(T), STAGES = 2;
  static constexpr int E = 16 / sizeof(T), COPIES = SWEEP / 512;  // values of a copy, copies of a sweep for each lane
  __host__ __device__ static int sweeps(int heads) { return (heads + HPW - 1) / HPW; }
  static size_t smem(const RotaryParams& p) { return (size_t)STAGES * 8 * (sweeps(p.NQ) + sweeps(p.NK)) * SWEEP; }
  // H heads, `stride` apart, brought to `to` (16 bytes a lane)
  static __device__ __forceinline__ void bring(uint32_t to, const T* x, long long stride, int H, int lane) {
#pragma unroll
    for (int c = 0; c < COPIES; ++c) {
      const int v = (c * 32 + lane) * E, h = v / D;
      const T* from = x + h * stride + v % D;
      uint32_t d = to + c * 512 + 16 * lane;
#pragma unroll 3
      for (int i = 0; i < H; i += HPW) {
        if (i + h < H) cp_async16(d, from);
        from += HPW * stride, d += SWEEP;
      }
    }
  }
};

// A warp takes whole tokens.
template <class T, int LPH, int MODE>
__global__ void __launch_bounds__(256, sizeof(T) == 4 ? 2 : 3) rotary_ring_kernel(const RotaryParams p) {
  using C = Ring<T, LPH>;
  constexpr int HPW = C::HPW, D = C::D, STAGES = C::STAGES;
  extern __shared__ __align__(128) char dyn[];
  __shared__ Consts sh;
  depend_launch();
  Lanes<LPH, MODE> w(p);
  w.spread(D * sizeof(T));
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int nq = C::sweeps(p.NQ), nk = C::sweeps(p.NK), size = (nq + nk) * C::SWEEP;
  char* const ring = dyn + warp * STAGES * size;
  const unsigned line = blockIdx.x * 8 + warp, lines = gridDim.x * 8, dt = lines / p.B, db = lines % p.B;
  depend_wait();
  // token (t, b): the one to be copied, then the one to be worked on
  unsigned at = line / p.B, ab = line % p.B, t = at, b = ab;
  auto next = [&](unsigned& t, unsigned& b) {
    t += dt, b += db;
    if (b >= (unsigned)p.B) b -= p.B, ++t;
  };
  auto bring = [&](int stage) {
    if (at < (unsigned)p.T) {
      const uint32_t to = smem_u32(ring + stage * size);
      C::bring(to, static_cast<const T*>(p.q) + at * p.qs[0] + ab * p.qs[1], p.qs[2], p.NQ, lane);
      C::bring(to + nq * C::SWEEP, static_cast<const T*>(p.k) + at * p.ks[0] + ab * p.ks[1], p.ks[2], p.NK, lane);
    }
    cp_async_commit();
    next(at, ab);
  };
#pragma unroll
  for (int k = 0; k < STAGES - 1; ++k) bring(k);
  sh.load(p);
  constexpr float inv = 1.f / D;
  const Pairs wq = w.weights(sh.w[0]), wk = w.weights(sh.w[1]);
  Turn tn;
  const bool norm = p.qw != nullptr;  // (without: weights of one, r = 1)
  auto sweep = [&](const T* x, T* o, const Pairs& wt, bool on) {
    Head<T, MODE> raw;
    w.load(raw, x);
    Pairs y = w.get(raw);
    const Num<2> r(norm ? rsqrtf(fmaf(head_sum<LPH>(dot(y, y)), inv, p.eps)) : 1.f);
#pragma unroll
    for (int j = 0; j < 2; ++j) y.a[j] = y.a[j] * (r * wt.a[j]), y.b[j] = y.b[j] * (r * wt.b[j]);
    rotate(w, y, tn.c, tn.s, tn.n);
    if (on) w.store(o, y);
  };
  auto heads = [&](const T* x, T* o, int n, const Pairs& wt) {
#pragma unroll 3
    for (int i = n / HPW; i > 0; --i) {
      sweep(x, o, wt, true);
      x += HPW * D, o += HPW * D;
    }
    if (n % HPW) sweep(x, o, wt, w.sub < n % HPW);  // (what the others compute stays in their own head)
  };
  long long pos = t < (unsigned)p.T ? position(p, t, b) : 0;
  const int mine = w.sub * D;
  T* qo = static_cast<T*>(p.qo) + (long long)line * p.NQ * D + mine;
  T* ko = static_cast<T*>(p.ko) + (long long)line * p.NK * D + mine;
  for (int stage = 0; t < (unsigned)p.T; stage = stage + 1 == STAGES ? 0 : stage + 1) {
    bring(stage == 0 ? STAGES - 1 : stage - 1);
    tn = turn_of<Lanes<LPH, MODE>, LPH>(w, sh.freqs, pos);
    next(t, b);
    if (t < (unsigned)p.T) pos = position(p, t, b);  // a token ahead
    cp_async_wait<STAGES - 1>();
    __syncwarp();
    const T* x = reinterpret_cast<const T*>(ring + stage * size) + mine;
    heads(x, qo, p.NQ, wq);
    heads(x + nq * HPW * D, ko, p.NK, wk);
    __syncwarp();  // (the stage is filled again by the next copies)
    qo += (long long)lines * p.NQ * D, ko += (long long)lines * p.NK * D;
  }
}

// Gradient: a CTA takes q's heads or k's, so that a warp keeps one set of weights and of their gradients' sums, and a warp
// a group of a token's heads at a time, so that rings hold any number of heads.  8004 tokens of 6 + 6 x 128 heads take
// 20.6 us with dw's sum (3.7 TB/s; bound by latency, with 16 warps an SM, and issue slots), whole tokens by a warp 22.8; 1024 x 8
// of 16 + 8 x 128 37 and 48, 1024 x 4 of 8 + 4 x 256 24 and 33, but of 12 + 1 x 64 12.0 and 11.2, where k's sweeps are
// mostly empty.  (Forward, whole tokens keep fewer registers and take their sines once: 19.7 us against 20.6 for 16384 tokens of
// 12 + 12 x 64.)  Sixteen warps a CTA, one on an SM: twice eight leave twice the sums (21.4 us), twenty spill (21.2).
template <class T, int LPH>
struct Groups {
  using C = Ring<T, LPH>;
  // warps; sweeps of a group (192 KB for a CTA; of 2 rather than 3 sweeps 30.7 us for the 8004 tokens above)
  static constexpr int W = 16, MOST = 6 * 512 / C::SWEEP;
  int n, sweeps;  // groups of a token, sweeps of each but the last
  __host__ __device__ explicit Groups(int heads) {
    const int all = C::sweeps(heads);
    n = (all + MOST - 1) / MOST;
    sweeps = n > 0 ? (all + n - 1) / n : 0;
  }
  __host__ __device__ int bytes() const { return C::STAGES * 2 * sweeps * C::SWEEP; }  // of a warp
  // of a token, in half sweeps: a group's sines are that of one
  int work(int heads) const { return 2 * C::sweeps(heads) + n; }
};

// ONE: of q and of k, one group at most (20.6 us for the tokens above against 21.5 that keep count of groups)
template <class T, int LPH, int MODE, bool ONE>
__global__ void __launch_bounds__(32 * Groups<T, LPH>::W, 1) rotary_ring_bwd_kernel(const RotaryParams p) {
  using C = Ring<T, LPH>;
  constexpr int HPW = C::HPW, D = C::D, STAGES = C::STAGES, W = Groups<T, LPH>::W;
  extern __shared__ __align__(128) char dyn[];
  __shared__ Consts sh;
  __shared__ float part[W][D];
  depend_launch();
  Lanes<LPH, MODE> w(p);
  w.spread(D * sizeof(T));
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const bool isk = blockIdx.x >= (unsigned)p.ctas_q;
  const int H = isk ? p.NK : p.NQ;
  const long long* const xs = isk ? p.ks : p.qs;
  const long long* const ds = isk ? p.dks : p.dqs;
  const T* const x0 = static_cast<const T*>(isk ? p.k : p.q);
  const T* const d0 = static_cast<const T*>(isk ? p.dk : p.dq);
  const Groups<T, LPH> gr(H);
  const int most = gr.sweeps * HPW, size = gr.sweeps * C::SWEEP;
  char* const ring = dyn + warp * gr.bytes();
  const unsigned cta = isk ? blockIdx.x - p.ctas_q : blockIdx.x, ctas = isk ? gridDim.x - p.ctas_q : p.ctas_q;
  const unsigned line = cta * W + warp, lines = ctas * W;
  depend_wait();
  struct At {  // a group of a token
    unsigned t, b, g;
  };
  auto place = [&](unsigned i) {
    const unsigned row = ONE ? i : i / gr.n, t = row / p.B;
    return At{t, row - t * p.B, ONE ? 0 : i - row * gr.n};
  };
  const At step = place(lines);
  At to = place(line), at = to;  // the one to be copied, the one to be worked on
  auto next = [&](At& x) {
    x.t += step.t, x.b += step.b;
    if (!ONE) {
      x.g += step.g;
      if (x.g >= (unsigned)gr.n) x.g -= gr.n, ++x.b;
    }
    if (x.b >= (unsigned)p.B) x.b -= p.B, ++x.t;
  };
  auto bring = [&](int stage) {
    if (to.t < (unsigned)p.T) {
      const uint32_t a = smem_u32(ring + stage * 2 * size);
      const int h = ONE ? 0 : to.g * most, n = ONE || H - h < most ? H - h : most;
      C::bring(a, x0 + to.t * xs[0] + to.b * xs[1] + h * xs[2], xs[2], n, lane);
      C::bring(a + size, d0 + to.t * ds[0] + to.b * ds[1] + h * ds[2], ds[2], n, lane);
    }
    cp_async_commit();
    next(to);
  };
#pragma unroll
  for (int k = 0; k < STAGES - 1; ++k) bring(k);
  sh.load(p);
  constexpr float inv = 1.f / D;
  const Pairs wt = w.weights(sh.w[isk]);
  Pairs sum;
#pragma unroll
  for (int j = 0; j < 2; ++j) sum.a[j] = sum.b[j] = Num<2>(0.f);
  Turn tn;
  const bool norm = p.qw != nullptr;  // (without: weights of one, r = 1)
  auto sweep = [&](const T* x, const T* d, T* o, bool on) {
    Head<T, MODE> raw, rd;
    w.load(raw, x);
    Pairs y = w.get(raw);
    if (!norm)  // (x does not matter then, whatever it is)
#pragma unroll
      for (int j = 0; j < 2; ++j) y.a[j] = y.b[j] = Num<2>(0.f);
    const float r1 = norm ? rsqrtf(fmaf(head_sum<LPH>(dot(y, y)), inv, p.eps)) : 1.f;
    const Num<2> r(r1);
    w.load(rd, d);
    Pairs g = w.get(rd), gw;
    rotate(w, g, tn.c, tn.n, tn.s);  // back
#pragma unroll
    for (int j = 0; j < 2; ++j) gw.a[j] = g.a[j] * wt.a[j], gw.b[j] = g.b[j] * wt.b[j];
    const float along = head_sum<LPH>(dot(gw, y));
    const Num<2> m(norm ? -(along * inv) * r1 * r1 : 0.f);  // - mean(w g xh) r
    if (on)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        sum.a[j] = fma(g.a[j], y.a[j] * r, sum.a[j]);
        sum.b[j] = fma(g.b[j], y.b[j] * r, sum.b[j]);
      }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      g.a[j] = r * fma(m, y.a[j], gw.a[j]);
      g.b[j] = r * fma(m, y.b[j], gw.b[j]);
    }
    if (on) w.store(o, g);
  };
  long long pos = at.t < (unsigned)p.T ? position(p, at.t, at.b) : 0;
  const int mine = w.sub * D;
  T* const out = static_cast<T*>(isk ? p.ko : p.qo) + mine;
  for (int stage = 0; at.t < (unsigned)p.T; stage = stage + 1 == STAGES ? 0 : stage + 1) {
    bring(stage == 0 ? STAGES - 1 : stage - 1);
    tn = turn_of<Lanes<LPH, MODE>, LPH>(w, sh.freqs, pos);
    const int h = ONE ? 0 : at.g * most, n = ONE || H - h < most ? H - h : most;
    T* o = out + ((long long)(at.t * p.B + at.b) * H + h) * D;
    next(at);
    if (at.t < (unsigned)p.T) pos = position(p, at.t, at.b);  // a group ahead
    cp_async_wait<STAGES - 1>();
    __syncwarp();
    const T* x = reinterpret_cast<const T*>(ring + stage * 2 * size) + mine;
    const T* d = x + size / (int)sizeof(T);
#pragma unroll 3
    for (int i = n / HPW; i > 0; --i) {
      sweep(x, d, o, true);
      x += HPW * D, d += HPW * D, o += HPW * D;
    }
    if (n % HPW) sweep(x, d, o, w.sub < n % HPW);  // (what the others compute stays in their own head)
    __syncwarp();  // (the stage is filled again by the next copies)
  }
  if (!p.qw) return;
  if (w.swap) {
    const Pairs x = sum;
#pragma unroll
    for (int j = 0; j < 2; ++j) sum.a[j] = x.b[j], sum.b[j] = x.a[j];
  }
  sum_lanes<LPH>(sum);
  if (w.sub == 0) w.add_to(part[warp], sum);
  __syncthreads();
  for (int i = threadIdx.x; i < D; i += blockDim.x) {
    float v = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) v += part[j][i];
    p.part[(long long)blockIdx.x * 2 * D + isk * D + i] = v;
  }
}

// The same for larger heads, value by value: a CTA of one warp takes a head of a token at a time.
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
  auto turned = [&](int i, long long pos, float way, float& a, float& b) {  // pair i; way: -1 turns back
    if (i >= half) return;
    float c, s;
    turn(turns(p.freqs[i]), pos, c, s);
    s *= way;
    const float a0 = a;
    a = fmaf(a0, c, -b * s);
    b = fmaf(b, c, a0 * s);
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
    for (int i = lane; w && i < p.D / 2; i += 32) {
      int ia, ib;
      columns(i, ia, ib);
      const float xa = get1(x + ia), xb = get1(x + ib);
      sum = fmaf(xa, xa, fmaf(xb, xb, sum));
      if (BWD) {
        float ga = get1(g + ia), gb = get1(g + ib);
        turned(i, pos, -1.f, ga, gb);
        along = fmaf(ga * w[ia], xa, fmaf(gb * w[ib], xb, along));
      }
    }
    const float r = w ? rsqrtf(head_sum<32>(sum) / p.D + p.eps) : 1.f;
    const float m = BWD && w ? head_sum<32>(along) * r * r / p.D : 0.f;
    for (int i = lane; i < p.D / 2; i += 32) {
      int ia, ib;
      columns(i, ia, ib);
      const float wa = w ? w[ia] : 1.f, wb = w ? w[ib] : 1.f;
      if (BWD) {
        float ga = get1(g + ia), gb = get1(g + ib);
        turned(i, pos, -1.f, ga, gb);
        if (w) {
          const float xa = get1(x + ia), xb = get1(x + ib);
          float* to = acc + (isq ? 0 : p.D);
          to[ia] = fmaf(ga, xa * r, to[ia]);
          to[ib] = fmaf(gb, xb * r, to[ib]);
          put1(o + ia, r * fmaf(-m, xa, ga * wa));
          put1(o + ib, r * fmaf(-m, xb, gb * wb));
        } else {  // (x does not matter then, whatever it is)
          put1(o + ia, ga);
          put1(o + ib, gb);
        }
      } else {
        float ya = get1(x + ia) * (r * wa), yb = get1(x + ib) * (r * wb);
        turned(i, pos, 1.f, ya, yb);
        put1(o + ia, ya);
        put1(o + ib, yb);
      }
    }
  }
  if (BWD && p.qw) {
    __syncwarp();
    for (int i = lane; i < 2 * p.D; i += 32) p.part[(long long)blockIdx.x * 2 * p.D + i] = acc[i];
  }
}

// dw[i] = sum of the CTAs' parts in a fixed order: 8 columns a CTA, 32 threads for each.  q's are of the parts up to end_q,
// k's of those from first_k on.  (CTAs of 256 threads find room beside those of the kernel before and wait there: 0.4 us less
// than with 1024)
__global__ void __launch_bounds__(256) rotary_dw_kernel(const float* part, float* dqw, float* dkw, int parts, int end_q,
                                                         int first_k, int D) {
  __shared__ float sh[32][9];
  depend_launch();
  depend_wait();
  const int x = threadIdx.x % 8, y = threadIdx.x / 8, i = blockIdx.x * 8 + x;
  float v = 0.f;
  if (i < 2 * D) {
    const int n = i < D ? end_q : parts - first_k;
    const float* at = part + i + (i < D ? 0LL : (long long)first_k * 2 * D);
#pragma unroll 8
    for (int j = y; j < n; j += 32) v += at[(long long)j * 2 * D];
  }
  sh[y][x] = v;
  __syncthreads();
  v = head_sum<32>(sh[threadIdx.x % 32][threadIdx.x / 32]);
  const int c = blockIdx.x * 8 + threadIdx.x / 32;
  if (threadIdx.x % 32 == 0 && c < 2 * D) (c < D ? dqw : dkw)[c % D] = v;
}

bool at16(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool strides4(const long long (&s)[3]) { return s[0] % 4 == 0 && s[1] % 4 == 0 && s[2] % 4 == 0; }

// pieces of four columns need sizes and addresses that are multiples of four values (kHalf: a turned part that is, too)
template <class T>
bool vector_form(const RotaryParams& p, bool bwd) {
  constexpr size_t A = 4 * sizeof(T);
  bool ok = p.D % 8 == 0 && (p.interleaved || p.rot % 8 == 0) && strides4(p.qs) && strides4(p.ks) &&
            at16(p.q, A) && at16(p.k, A) && at16(p.qo, A) && at16(p.ko, A);
  if (bwd) ok = ok && strides4(p.dqs) && strides4(p.dks) && at16(p.dq, A) && at16(p.dk, A);
  return ok;
}

int reduce_dw(const RotaryParams& p, int parts, int end_q, int first_k, cudaStream_t s) {
  return launch_dependent(rotary_dw_kernel, (unsigned)((2 * p.D + 7) / 8), 256, 0, s, (const float*)p.part, p.dqw, p.dkw,
                          parts, end_q, first_k, p.D);
}

template <class T, int LPH, int MODE>
int launch_lanes(RotaryParams& p, bool bwd, cudaStream_t s) {
  const long long tokens = (long long)p.T * p.B;
  const int heads = 32 / LPH * (bwd ? kBatchBwd : kBatch), per_sm = bwd ? 2 : 3;
  const int groups = (p.NQ + heads - 1) / heads + (p.NK + heads - 1) / heads;
  // few tokens: a warp for each batch of heads, so that the latency of one batch is that of all (608 tokens of 12 + 12 x 64
  // heads 3.6 us against 4.3, 1216 4.5 against 4.4; gradient 1216 8.0 against 9.4, 2432 11.2 against 9.2, where rings cannot
  // take them)
  p.split = tokens < (bwd ? 16LL : 8LL) * sm_count();
  const long long want = (tokens * (p.split ? groups : 1) + 7) / 8, most = (long long)per_sm * sm_count();
  unsigned grid = (unsigned)(want < most ? want : most);
  if (!bwd) return launch_dependent(rotary_kernel<T, LPH, MODE>, grid, 256, 0, s, (const RotaryParams)p);
  if (grid > kRotaryParts) grid = kRotaryParts;
  const int e = launch_dependent(rotary_bwd_kernel<T, LPH, MODE>, grid, 256, 0, s, (const RotaryParams)p);
  return e != 0 || !p.qw ? e : reduce_dw(p, (int)grid, (int)grid, 0, s);
}
// 16-byte copies, and tokens enough: 4864 of 12 + 12 x 64 heads take 7.9 us against 8.3 by batches (gradient 13.5 against
// 16.0), 2432 5.6 against 5.9 (9.0 against 9.4; 1216 7.1 against 8.2), 608 4.2 against 4.3, and 3.6 with the batches split
template <class T, int LPH>
bool ring_form(const RotaryParams& p, bool bwd) {
  auto even = [](const void* x, const long long (&s)[3]) {
    return reinterpret_cast<uintptr_t>(x) % 16 == 0 && (s[0] | s[1] | s[2]) * (long long)sizeof(T) % 16 == 0;
  };
  bool ok = p.D == 8 * LPH && vector_form<T>(p, bwd) && even(p.q, p.qs) && even(p.k, p.ks);
  if (bwd) ok = ok && even(p.dq, p.dqs) && even(p.dk, p.dks);
  ok = ok && (bwd || Ring<T, LPH>::smem(p) <= kRingMost);
  return ok && (long long)p.T * p.B >= (bwd ? kRingTokensBwd : kRingTokens) * sm_count();
}
template <class T, int LPH, int MODE>
int launch_ring(const RotaryParams& p, cudaStream_t s) {
  static int prep[64][5];
  const size_t smem = Ring<T, LPH>::smem(p);
  const int e = prepare_launch(prep, rotary_ring_kernel<T, LPH, MODE>, (uint32_t)smem, 256, 1);
  if (e != 0) return e;
  const long long want = ((long long)p.T * p.B + 7) / 8, most = (sizeof(T) == 4 ? 2LL : 3LL) * sm_count();
  return launch_dependent(rotary_ring_kernel<T, LPH, MODE>, (unsigned)(want < most ? want : most), 256, smem, s, p);
}
template <class T, int LPH, int MODE, bool ONE>
int launch_ring_bwd(RotaryParams& p, cudaStream_t s) {
  using G = Groups<T, LPH>;
  static int prep[64][5];
  const G q(p.NQ), k(p.NK);
  const size_t smem = (size_t)G::W * (q.bytes() > k.bytes() ? q.bytes() : k.bytes());
  const int e = prepare_launch(prep, rotary_ring_bwd_kernel<T, LPH, MODE, ONE>, (uint32_t)smem, 32 * G::W, 1);
  if (e != 0) return e;
  // q's and k's CTAs by their work; at least one for each that has heads
  const int most = sm_count() < kRotaryParts ? sm_count() : kRotaryParts;
  const long long wq = q.work(p.NQ), wk = k.work(p.NK);
  int nq = (int)((most * wq + (wq + wk) / 2) / (wq + wk));
  if (wq > 0 && wk > 0) nq = nq < 1 ? 1 : nq > most - 1 ? most - 1 : nq;
  p.ctas_q = nq;
  const int err = launch_dependent(rotary_ring_bwd_kernel<T, LPH, MODE, ONE>, (unsigned)most, 32 * G::W, smem, s,
                                   (const RotaryParams)p);
  return err != 0 || !p.qw ? err : reduce_dw(p, most, nq, nq, s);
}
template <class T, int LPH, int MODE>
int launch_ring(RotaryParams& p, bool bwd, cudaStream_t s) {
  if (!bwd) return launch_ring<T, LPH, MODE>(p, s);
  return Groups<T, LPH>(p.NQ).n <= 1 && Groups<T, LPH>(p.NK).n <= 1 ? launch_ring_bwd<T, LPH, MODE, true>(p, s)
                                                                    : launch_ring_bwd<T, LPH, MODE, false>(p, s);
}
template <class T, int LPH>
int launch_mode(RotaryParams& p, bool bwd, cudaStream_t s) {
  if (ring_form<T, LPH>(p, bwd))
    return !p.interleaved ? launch_ring<T, LPH, kHalf>(p, bwd, s)
           : p.rot % 8 == 0 ? launch_ring<T, LPH, kNext>(p, bwd, s)
                            : launch_ring<T, LPH, kSome>(p, bwd, s);
  if (!vector_form<T>(p, bwd)) return launch_lanes<T, LPH, kAny>(p, bwd, s);
  return !p.interleaved ? launch_lanes<T, LPH, kHalf>(p, bwd, s)
         : p.rot % 8 == 0 ? launch_lanes<T, LPH, kNext>(p, bwd, s)
                          : launch_lanes<T, LPH, kSome>(p, bwd, s);
}
template <class T>
int launch_t(RotaryParams& p, bool bwd, cudaStream_t s) {
  if (p.D <= 32) return launch_mode<T, 4>(p, bwd, s);
  if (p.D <= 64) return launch_mode<T, 8>(p, bwd, s);
  if (p.D <= 128) return launch_mode<T, 16>(p, bwd, s);
  if (p.D <= 2 * kMaxPairs) return launch_mode<T, 32>(p, bwd, s);
  const long long items = (long long)p.T * p.B * (p.NQ + p.NK);
  if (!bwd) {
    const long long most = 32LL * sm_count();
    return launch_dependent(rotary_any_kernel<T, false>, (unsigned)(items < most ? items : most), 32, 0, s,
                            (const RotaryParams)p);
  }
  const int grid = (int)(items < kRotaryParts ? items : kRotaryParts);
  const int e = launch_dependent(rotary_any_kernel<T, true>, (unsigned)grid, 32, p.qw ? 8 * (size_t)p.D : 0, s,
                                 (const RotaryParams)p);
  return e != 0 || !p.qw ? e : reduce_dw(p, grid, grid, 0, s);
}

}  // namespace

int launch_rotary(RotaryParams p, bool bf16, bool bwd, cudaStream_t s) {
  return bf16 ? launch_t<__nv_bfloat16>(p, bwd, s) : launch_t<float>(p, bwd, s);
}

}  // namespace srnn
