// What the linear-attention kernels share: the place of a CTA, powers of the
// decay, and the scan over the segments of the token axis.
//
// A long sequence is cut into segments so that its heads fill the GPU: one
// launch sums each segment's own contribution to the state (from zero), the scan
// turns these into the state at the start of every segment, and the main launch
// runs all segments at once.
#pragma once
#include <cstdint>

#include "lm.h"

namespace srnn {

// 16 bytes to shared memory, zeros where not `valid`
__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
// 0 as long as every value of the packed pairs seen is finite (0 times an infinity or NaN is NaN, and NaN stays)
__device__ __forceinline__ uint32_t seen_finite(uint32_t seen, uint32_t pair) {
  asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(seen) : "r"(pair), "r"(0u));
  return seen;
}
// largest magnitude of three, NaN if one is
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// lambda^n, n >= 0 (lg = log2 lambda, possibly -inf)
__device__ __forceinline__ float pw(float lg, int n) { return n == 0 ? 1.f : exp2f(lg * (float)n); }

struct Where {
  int job, b, h, bh, vt, seg;
};
__device__ __forceinline__ Where where_of(const LinAttnParams& p, int VT, int segs) {
  Where w;
  int i = blockIdx.x;
  w.seg = i % segs;
  i /= segs;
  w.vt = i % VT;
  i /= VT;
  w.bh = i % (p.B * p.NH);
  w.job = i / (p.B * p.NH);
  w.b = w.bh / p.NH;
  w.h = w.bh % p.NH;
  return w;
}
__device__ __forceinline__ int row_len(const LinAttnParams& p, int b) {
  if (p.lens == nullptr) return p.T;
  const int n = p.lens[b];
  return n < 0 ? 0 : (n > p.T ? p.T : n);
}
// segment states (slot s: the state segment s starts from): [segment][pass][head of a row][v tile] tiles of `tile` values
__device__ __forceinline__ float* seg_state(const LinAttnParams& p, const Where& w, int seg, int VT,
                                            int tile) {
  return p.ws + ((((long long)seg * p.npass + w.job) * p.B * p.NH + w.bh) * VT + w.vt) * tile;
}

// Contributions of segments 0 .. nseg - 2 (in slots 1 ..) -> the states that the
// segments start from, in place; slot 0 gets the initial state, so that the main
// launch reads no initial state that it may be writing as the final one.  Order maps a place in a workspace tile to (dk, v).
template <class Order>
__global__ void __launch_bounds__(256)
    linattn_scan_kernel(const __grid_constant__ LinAttnParams p, int seg_tokens) {
  constexpr int TILE = Order::TILE, PER = TILE / 256;  // blocks of 256 per tile
  depend_launch();
  const int VT = Order::tiles(p);
  const int e = (blockIdx.x % PER) * 256 + threadIdx.x;
  int i = blockIdx.x / PER;
  Where w;
  w.vt = i % VT;
  i /= VT;
  w.bh = i % (p.B * p.NH);
  w.job = i / (p.B * p.NH);
  w.b = w.bh / p.NH;
  w.h = w.bh % p.NH;
  w.seg = 0;
  const LinAttnPass& ps = p.pass[w.job];
  const int len = row_len(p, w.b);
  const int n = len > 0 ? (len - 1) / seg_tokens : 0;  // segments that another one follows
  const float lam = pw(p.log_decay[w.h] * 1.4426950408889634f, seg_tokens);
  int dk, v;
  Order::at(p, w.vt, e, dk, v);
  const float* in = ps.init ? ps.init + (long long)w.bh * p.DK * p.DV : nullptr;
  float s = in ? in[ps.init_t ? (long long)v * p.DK + dk : (long long)dk * p.DV + v] : 0.f;
  float* ws = seg_state(p, w, 0, VT, TILE) + e;
  depend_wait();  // for the segments' contributions
  *ws = s;
  const long long step = (long long)p.npass * p.B * p.NH * VT * TILE;
  ws += step;
  for (int k = 0; k < n; k += 32) {  // the loads of 32 segments in flight
    float x[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) x[j] = k + j < n ? ws[(k + j) * step] : 0.f;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      s = fmaf(lam, s, x[j]);
      if (k + j < n) ws[(k + j) * step] = s;
    }
  }
}

}  // namespace srnn
