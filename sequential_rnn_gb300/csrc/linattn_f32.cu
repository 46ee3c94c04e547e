// Linear attention with a decay for each head, fp32: the precision path.  The
// same passes as linattn.cu, with fp32 multiply-adds throughout.
//
// One CTA per (pass, row, head, 32 columns of the state, segment), chunks of 32
// tokens staged in shared memory, the state [DK, 32] there too.  Each thread
// owns a 2 x 2 piece of the scores and of the output, and DK / 8 elements of
// the state.
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "linattn.cuh"
#include "lm.h"
#include "ptx.cuh"

namespace srnn {
namespace {

constexpr int kC32 = 32, kV32 = 32, kT32 = 256;

template <int DK>
struct La32Cfg {
  static constexpr int LD = DK + 4;  // row pitch of x and a: 16-byte rows, banks shifted row by row
  static constexpr uint32_t FLOATS = 2 * kC32 * LD + kC32 * kV32 + kC32 * (kC32 + 1) + DK * kV32 + 3 * kC32;
  static constexpr uint32_t SMEM = FLOATS * 4;
};
template <int DK>
struct RowOrder {
  static constexpr int TILE = DK * kV32;
  static __device__ __forceinline__ int tiles(const LinAttnParams& p) { return p.DV / kV32; }
  static __device__ __forceinline__ void at(const LinAttnParams&, int tile, int e, int& dk, int& v) {
    dk = e / kV32;
    v = tile * kV32 + e % kV32;
  }
};

template <int DK, bool STATE_ONLY>
__global__ void __launch_bounds__(kT32)
    linattn_f32_kernel(const __grid_constant__ LinAttnParams p) {
  using C = La32Cfg<DK>;
  extern __shared__ __align__(16) float sm[];
  float* X = sm;
  float* A = X + kC32 * C::LD;
  float* V = A + kC32 * C::LD;
  float* P = V + kC32 * kV32;
  float* S = P + kC32 * (kC32 + 1);
  float* pws = S + DK * kV32;  // lambda^m, m = 0 .. 32
  float* wj = pws + kC32 + 1;  // weight of token j in the state's update
  const int tid = threadIdx.x;
  if (STATE_ONLY || p.nseg == 1) {  // the call's first kernel
    depend_wait();
    depend_launch();
  }
  const int VT = p.DV / kV32;
  const Where w = where_of(p, VT, STATE_ONLY ? p.nseg - 1 : p.nseg);
  const LinAttnPass& ps = p.pass[w.job];
  const int len = row_len(p, w.b);
  const int nch = (p.T + kC32 - 1) / kC32;
  const int c0 = w.seg * p.seg_chunks;
  const int c1 = c0 + p.seg_chunks < nch ? c0 + p.seg_chunks : nch;
  const int lch = (len + kC32 - 1) / kC32;
  const int cend = c1 < lch ? c1 : lch;
  if (STATE_ONLY && (long long)c1 * kC32 >= len) return;
  const float lg = p.log_decay[w.h] * 1.4426950408889634f;
  const bool rev = ps.reverse != 0;
  if (!STATE_ONLY && blockIdx.x == 0 && tid == 0 && p.clear) *p.status = 0;
  const float* gx = static_cast<const float*>(ps.x) + w.b * ps.xs[1] + w.h * ps.xs[2];
  const float* ga = static_cast<const float*>(ps.a) + w.b * ps.as[1] + w.h * ps.as[2];
  const float* gc = static_cast<const float*>(ps.c) + w.b * ps.cs[1] + w.h * ps.cs[2] + w.vt * kV32;
  float* gout = static_cast<float*>(ps.out) + w.b * ps.os[1] + w.h * ps.os[2] + w.vt * kV32;

  if (STATE_ONLY) {
    for (int e = tid; e < DK * kV32; e += kT32) S[e] = 0.f;
  } else if (p.nseg > 1) {
    depend_wait();  // for the scan
    const float* src = seg_state(p, w, w.seg, VT, DK * kV32);
    if (w.seg == 0 || c0 < cend)
      for (int e = tid; e < DK * kV32; e += kT32) S[e] = src[e];
  } else {
    const float* in = ps.init ? ps.init + (long long)w.bh * DK * p.DV : nullptr;
    for (int e = tid; e < DK * kV32; e += kT32) {
      const int dk = e / kV32, v = w.vt * kV32 + e % kV32;
      S[e] = in ? in[ps.init_t ? (long long)v * DK + dk : (long long)dk * p.DV + v] : 0.f;
    }
  }
  if (tid <= kC32) pws[tid] = pw(lg, tid);

  for (int c = c0; c < cend; ++c) {
    const int n = len - c * kC32 < kC32 ? len - c * kC32 : kC32;
    __syncthreads();
    for (int e = tid; e < kC32 * (DK / 4); e += kT32) {
      const int row = e / (DK / 4), col = 4 * (e % (DK / 4));
      const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
      const int r = c * kC32 + row;
      const long long t = rev ? len - 1 - r : r;
      const bool ok = row < n;
      if (!STATE_ONLY)
        *reinterpret_cast<float4*>(X + row * C::LD + col) =
            ok ? *reinterpret_cast<const float4*>(gx + t * ps.xs[0] + col) : z;
      *reinterpret_cast<float4*>(A + row * C::LD + col) =
          ok ? *reinterpret_cast<const float4*>(ga + t * ps.as[0] + col) : z;
    }
    for (int e = tid; e < kC32 * (kV32 / 4); e += kT32) {
      const int row = e / (kV32 / 4), col = 4 * (e % (kV32 / 4));
      const int r = c * kC32 + row;
      const long long t = rev ? len - 1 - r : r;
      *reinterpret_cast<float4*>(V + row * kV32 + col) =
          row < n ? *reinterpret_cast<const float4*>(gc + t * ps.cs[0] + col)
                  : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (tid < kC32) wj[tid] = tid < n ? ps.upd * pw(lg, n - 1 - tid + ps.shift) : 0.f;
    __syncthreads();
    const int i0 = 2 * (tid / 16), j0 = 2 * (tid % 16);  // this thread's 2 x 2 pieces
    if (!STATE_ONLY) {
      float s00 = 0.f, s01 = 0.f, s10 = 0.f, s11 = 0.f;
      if (j0 <= i0 + 1)
#pragma unroll 4
        for (int d = 0; d < DK; d += 4) {
          const float4 x0 = *reinterpret_cast<const float4*>(X + i0 * C::LD + d);
          const float4 x1 = *reinterpret_cast<const float4*>(X + (i0 + 1) * C::LD + d);
          const float4 a0 = *reinterpret_cast<const float4*>(A + j0 * C::LD + d);
          const float4 a1 = *reinterpret_cast<const float4*>(A + (j0 + 1) * C::LD + d);
          s00 = fmaf(x0.x, a0.x, fmaf(x0.y, a0.y, fmaf(x0.z, a0.z, fmaf(x0.w, a0.w, s00))));
          s01 = fmaf(x0.x, a1.x, fmaf(x0.y, a1.y, fmaf(x0.z, a1.z, fmaf(x0.w, a1.w, s01))));
          s10 = fmaf(x1.x, a0.x, fmaf(x1.y, a0.y, fmaf(x1.z, a0.z, fmaf(x1.w, a0.w, s10))));
          s11 = fmaf(x1.x, a1.x, fmaf(x1.y, a1.y, fmaf(x1.z, a1.z, fmaf(x1.w, a1.w, s11))));
        }
      auto put = [&](int i, int j, float v) {
        P[i * (kC32 + 1) + j] = j <= i ? v * (ps.intra * pws[i - j]) : 0.f;
      };
      put(i0, j0, s00);
      put(i0, j0 + 1, s01);
      put(i0 + 1, j0, s10);
      put(i0 + 1, j0 + 1, s11);
      __syncthreads();
      float o[2][2] = {{0.f, 0.f}, {0.f, 0.f}}, u[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll 4
      for (int d = 0; d < DK; ++d) {
        const float x0 = X[i0 * C::LD + d], x1 = X[(i0 + 1) * C::LD + d];
        const float2 s = *reinterpret_cast<const float2*>(S + d * kV32 + j0);
        u[0][0] = fmaf(x0, s.x, u[0][0]);
        u[0][1] = fmaf(x0, s.y, u[0][1]);
        u[1][0] = fmaf(x1, s.x, u[1][0]);
        u[1][1] = fmaf(x1, s.y, u[1][1]);
      }
      for (int j = 0; j <= i0 + 1; ++j) {
        const float p0 = P[i0 * (kC32 + 1) + j], p1 = P[(i0 + 1) * (kC32 + 1) + j];
        const float2 v = *reinterpret_cast<const float2*>(V + j * kV32 + j0);
        if (j <= i0) {
          o[0][0] = fmaf(p0, v.x, o[0][0]);
          o[0][1] = fmaf(p0, v.y, o[0][1]);
        }
        o[1][0] = fmaf(p1, v.x, o[1][0]);
        o[1][1] = fmaf(p1, v.y, o[1][1]);
      }
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        const int i = i0 + a;
        if (i >= n) continue;
        const float f = ps.inter * pws[i + 1 - ps.shift];
        const int r = c * kC32 + i;
        const long long t = rev ? len - 1 - r : r;
        *reinterpret_cast<float2*>(gout + t * ps.os[0] + j0) =
            make_float2(fmaf(f, u[a][0], o[a][0]), fmaf(f, u[a][1], o[a][1]));
      }
      __syncthreads();  // S was read
    }
    // state: thread (dk group, v): rows dk = tid / 32 + 8 m, column tid % 32
    const int v = tid & 31, d0 = tid >> 5;
    const float wS = pws[n];
    float add[DK / 8];
#pragma unroll
    for (int m = 0; m < DK / 8; ++m) add[m] = 0.f;
    for (int j = 0; j < n; ++j) {
      const float cv = V[j * kV32 + v] * wj[j];
#pragma unroll
      for (int m = 0; m < DK / 8; ++m) add[m] = fmaf(A[j * C::LD + d0 + 8 * m], cv, add[m]);
    }
#pragma unroll
    for (int m = 0; m < DK / 8; ++m) {
      float* s = S + (d0 + 8 * m) * kV32 + v;
      *s = fmaf(wS, *s, add[m]);
    }
  }
  __syncthreads();

  if (STATE_ONLY) {
    float* dst = seg_state(p, w, w.seg + 1, VT, DK * kV32);
    for (int e = tid; e < DK * kV32; e += kT32) dst[e] = S[e];
    return;
  }
  if (ps.fin != nullptr &&
      ((len > c0 * kC32 && (long long)len <= (long long)c1 * kC32) || (len == 0 && w.seg == 0))) {
    float* f = ps.fin + (long long)w.bh * DK * p.DV + w.vt * kV32;
    for (int e = tid; e < DK * kV32; e += kT32) f[(long long)(e / kV32) * p.DV + e % kV32] = S[e];
  }
  const int rlo = len > c0 * kC32 ? len : c0 * kC32, rhi = c1 * kC32 < p.T ? c1 * kC32 : p.T;
  for (int e = tid; e < (rhi - rlo) * kV32; e += kT32)
    gout[(long long)(rlo + e / kV32) * ps.os[0] + e % kV32] = 0.f;
}

template <int DK>
int launch_dk(const LinAttnParams& p, cudaStream_t s) {
  using C = La32Cfg<DK>;
  static int prep_main[64][5], prep_state[64][5];
  int e = prepare_launch(prep_main, linattn_f32_kernel<DK, false>, C::SMEM, kT32, 1);
  if (e != 0) return e;
  const long long base = (long long)p.npass * p.B * p.NH * (p.DV / kV32);
  if (base * p.nseg * (DK * kV32 / 256) > 0x7fffffffLL) return (int)cudaErrorInvalidValue;
  if (p.nseg > 1) {
    e = prepare_launch(prep_state, linattn_f32_kernel<DK, true>, C::SMEM, kT32, 1);
    if (e != 0) return e;
    e = launch_dependent(linattn_f32_kernel<DK, true>, (unsigned)(base * (p.nseg - 1)), kT32, C::SMEM, s, p);
    if (e != 0) return e;
    e = launch_dependent(linattn_scan_kernel<RowOrder<DK>>, (unsigned)(base * (DK * kV32 / 256)), 256, 0, s, p,
                         p.seg_chunks * kC32);
    if (e != 0) return e;
  }
  return launch_dependent(linattn_f32_kernel<DK, false>, (unsigned)(base * p.nseg), kT32, C::SMEM, s, p);
}

}  // namespace

int launch_linattn_f32(const LinAttnParams& p, cudaStream_t s) {
  switch (p.DK) {
    case 32: return launch_dk<32>(p, s);
    case 64: return launch_dk<64>(p, s);
    case 128: return launch_dk<128>(p, s);
    case 256: return launch_dk<256>(p, s);
    default: return (int)cudaErrorInvalidValue;
  }
}

}  // namespace srnn
