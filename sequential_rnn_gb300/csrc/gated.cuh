// Arithmetic of the gated recurrence's kernels: both sides of a sigmoid, maps.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "lm.h"
#include "num.cuh"

namespace srnn {

constexpr int kRunTokens = kGatedRun;                  // tokens of a run
constexpr int kRunWarps = 8;                           // runs of a CTA side by side
constexpr int kRunChunk = kRunTokens * kRunWarps;      // tokens of a CTA's round
constexpr int kGatedCluster = 16;                      // CTAs of a cluster, at most

template <class T>
__device__ __forceinline__ float exp_of(float x);  // x <= 0
template <>
__device__ __forceinline__ float exp_of<float>(float x) { return expf(x); }
// for bf16 gates: the product's rounding leaves a relative error of |x| 2^-24
template <>
__device__ __forceinline__ float exp_of<__nv_bfloat16>(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
  return y;
}
__device__ __forceinline__ float reciprocal(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// s = sigmoid(x), c = sigmoid(-x): the smaller one from e^-|x|, the larger one as 1 less it, so that both are good to
// a few units of their own last place (a memory of n tokens needs 1 - a to better than 1 / n); sl = s c
template <class T, int V>
__device__ __forceinline__ void sigmoids(const Num<V>& x, Num<V>& s, Num<V>& c, Num<V>* slope = nullptr) {
  Num<V> e, r;
#pragma unroll
  for (int v = 0; v < V; ++v) e.set(v, exp_of<T>(-fabsf(x.get(v))));
  const Num<V> d = e + Num<V>(1.f);
#pragma unroll
  for (int v = 0; v < V; ++v) r.set(v, reciprocal(d.get(v)));
  const Num<V> low = e * r, high = minus(Num<V>(1.f), low);
  if (slope) *slope = low * high;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const bool up = x.get(v) > 0.f;
    s.set(v, up ? high.get(v) : low.get(v));
    c.set(v, up ? low.get(v) : high.get(v));
  }
}
template <class T, int V>
__device__ __forceinline__ Num<V> sigmoid(const Num<V>& x) {
  Num<V> s, c;
  sigmoids<T>(x, s, c);
  return s;
}

// c -> a c + u of one channel
struct Map {
  float a, u;
};
}  // namespace srnn
