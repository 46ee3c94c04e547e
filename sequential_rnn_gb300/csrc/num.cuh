// One fp32 number, or two that one instruction adds and multiplies.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

namespace srnn {

// V fp32 numbers; a pair is added and multiplied by one instruction
template <int V>
struct Num;
template <>
struct Num<1> {
  float x;
  __device__ Num() {}
  __device__ explicit Num(float a) : x(a) {}
  __device__ float get(int) const { return x; }
  __device__ void set(int, float a) { x = a; }
};
template <>
struct Num<2> {
  float2 x;
  __device__ Num() {}
  __device__ explicit Num(float a) : x(make_float2(a, a)) {}
  __device__ float get(int i) const { return i ? x.y : x.x; }
  __device__ void set(int i, float a) { (i ? x.y : x.x) = a; }
};
__device__ __forceinline__ uint64_t bits(const Num<2>& a) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x.x), "f"(a.x.y));
  return r;
}
__device__ __forceinline__ Num<2> of_bits(uint64_t r) {
  Num<2> a;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x.x), "=f"(a.x.y) : "l"(r));
  return a;
}
__device__ __forceinline__ Num<1> fma(const Num<1>& a, const Num<1>& b, const Num<1>& c) { return Num<1>(fmaf(a.x, b.x, c.x)); }
__device__ __forceinline__ Num<1> operator*(const Num<1>& a, const Num<1>& b) { return Num<1>(a.x * b.x); }
__device__ __forceinline__ Num<1> operator+(const Num<1>& a, const Num<1>& b) { return Num<1>(a.x + b.x); }
__device__ __forceinline__ Num<2> fma(const Num<2>& a, const Num<2>& b, const Num<2>& c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
  return of_bits(r);
}
__device__ __forceinline__ Num<2> operator*(const Num<2>& a, const Num<2>& b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
  return of_bits(r);
}
__device__ __forceinline__ Num<2> operator+(const Num<2>& a, const Num<2>& b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
  return of_bits(r);
}
template <int V>
__device__ __forceinline__ Num<V> minus(const Num<V>& a, const Num<V>& b) { return fma(b, Num<V>(-1.f), a); }

}  // namespace srnn
