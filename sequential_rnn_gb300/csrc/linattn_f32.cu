// Linear attention with a decay for each head, fp32: the precision path.  The
// same passes as linattn.cu, with fp32 multiply-adds throughout.
//
// One CTA per (pass, row, head, 64 or 32 columns of the state, segment), chunks of 32 tokens (the scores, which every
// CTA of a head makes for itself, grow with the chunk) staged in shared memory, the state [DK, DVT] there too.
// Bound by the multiply-adds: a thread owns up to 4 x 4 of each product, so that eight 16-byte loads feed
// 64 of them (with 2 x 2, a load to each two, the kernel took 2.6 times as long).  Measured: 16 x 1024 tokens, 12 x 64,
// 217 us, gradient 393; 4 x 2001, 6 x 128 205 and 526; 4 x 4096, 4 x 256 1109 (19 TFLOP/s of fp32's 75) and 3112.
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "linattn.cuh"
#include "lm.h"
#include "ptx.cuh"

namespace srnn {
namespace {

constexpr int kC32 = 32;  // tokens per chunk

template <int DK_, int DVT_>
struct La32Cfg {
  static constexpr int DK = DK_, DVT = DVT_;
  static constexpr int NT = 128;
  static constexpr int OCC = DK <= 64 ? 4 : (DK == 128 ? 2 : 1);
  static constexpr int STAGES = DK <= 128 ? 1 : 2;  // with one CTA on an SM, the next chunk's copies run ahead
  static constexpr int LD = DK + 4;   // row pitch of x and a: 16-byte rows, banks shifted row by row
  static constexpr int LP = kC32 + 4;  // and of the scores
  static constexpr int RS = kC32 / (NT / 16);  // scores: rows of a thread (beside two columns)
  static constexpr int CT = DVT / 4, RT = NT / CT;  // threads side by side over the columns (4 each), and over rows
  static constexpr int RO = kC32 / RT;          // output: rows of a thread
  static constexpr int M = DK >= 4 * RT ? DK / (4 * RT) : 1;  // state: blocks of 4 rows of a thread
  static constexpr int STAGE = 2 * kC32 * LD + kC32 * DVT;    // x, a, c
  static constexpr uint32_t SMEM = (STAGES * STAGE + kC32 * LP + DK * DVT + 3 * kC32) * 4;
};
template <class C>
struct RowOrder {
  static constexpr int TILE = C::DK * C::DVT;
  static __device__ __forceinline__ int tiles(const LinAttnParams& p) { return p.DV / C::DVT; }
  static __device__ __forceinline__ void at(const LinAttnParams&, int tile, int e, int& dk, int& v) {
    dk = e / C::DVT;
    v = tile * C::DVT + e % C::DVT;
  }
};

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void fma4(float (&d)[4], float a, const float4& b) {
  d[0] = fmaf(a, b.x, d[0]);
  d[1] = fmaf(a, b.y, d[1]);
  d[2] = fmaf(a, b.z, d[2]);
  d[3] = fmaf(a, b.w, d[3]);
}
__device__ __forceinline__ float dot4(const float4& a, const float4& b, float c) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, c))));
}

template <class C, bool STATE_ONLY>
__global__ void __launch_bounds__(C::NT, C::OCC)
    linattn_f32_kernel(const __grid_constant__ LinAttnParams p) {
  constexpr int DK = C::DK, DVT = C::DVT, NT = C::NT, LD = C::LD, LP = C::LP, RS = C::RS, RO = C::RO, M = C::M;
  extern __shared__ __align__(16) float sm[];
  float* P = sm + C::STAGES * C::STAGE;
  float* S = P + kC32 * LP;
  float* pws = S + DK * DVT;   // lambda^m, m = 0 .. 32
  float* wj = pws + kC32 + 1;  // weight of token j in the state's update
  const int tid = threadIdx.x;
  if (STATE_ONLY || p.nseg == 1) depend_wait();  // the call's first kernel
  if (STATE_ONLY) depend_launch();
  const int VT = p.DV / DVT;
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
  const float* gc = static_cast<const float*>(ps.c) + w.b * ps.cs[1] + w.h * ps.cs[2] + w.vt * DVT;
  float* gout = static_cast<float*>(ps.out) + w.b * ps.os[1] + w.h * ps.os[2] + w.vt * DVT;

  auto load_rows = [&](float* dst, int pitch, int width, const float* src, long long stride, int c) {
    const uint32_t to = smem_u32(dst);
    for (int e = tid; e < kC32 * (width / 4); e += NT) {
      const int row = e / (width / 4), col = 4 * (e % (width / 4)), r = c * kC32 + row;
      const bool ok = r < len;
      const long long t = ok ? (rev ? len - 1 - r : r) : 0;
      cp_async16_zfill(to + (row * pitch + col) * 4, src + t * stride + col, ok);
    }
  };
  auto load_chunk = [&](int c, int st) {
    float* X = sm + st * C::STAGE;
    if (!STATE_ONLY) load_rows(X, LD, DK, gx, ps.xs[0], c);
    load_rows(X + kC32 * LD, LD, DK, ga, ps.as[0], c);
    load_rows(X + 2 * kC32 * LD, DVT, DVT, gc, ps.cs[0], c);
  };
  if (C::STAGES == 2 && c0 < cend) {
    load_chunk(c0, 0);
    cp_async_commit();
  }

  if (STATE_ONLY) {
    for (int e = tid; e < DK * DVT; e += NT) S[e] = 0.f;
  } else if (p.nseg > 1) {
    depend_wait();  // for the scan
    const float* src = seg_state(p, w, w.seg, VT, DK * DVT);
    if (w.seg == 0 || c0 < cend)
      for (int e = tid; e < DK * DVT; e += NT) S[e] = src[e];
  } else {
    const float* in = ps.init ? ps.init + (long long)w.bh * DK * p.DV : nullptr;
    for (int e = tid; e < DK * DVT; e += NT) {
      const int dk = e / DVT, v = w.vt * DVT + e % DVT;
      S[e] = in ? in[ps.init_t ? (long long)v * DK + dk : (long long)dk * p.DV + v] : 0.f;
    }
  }
  if (tid <= kC32) pws[tid] = pw(lg, tid);

  const int v0 = 4 * (tid % C::CT), rt = tid / C::CT;  // this thread's columns, and its place over the rows
  for (int c = c0; c < cend; ++c) {
    const int n = len - c * kC32 < kC32 ? len - c * kC32 : kC32;
    const int st = C::STAGES == 2 ? (c - c0) & 1 : 0;
    const float *X = sm + st * C::STAGE, *A = X + kC32 * LD, *V = A + kC32 * LD;
    __syncthreads();  // the chunk before has been read
    if (C::STAGES == 1)
      load_chunk(c, 0);
    else if (c + 1 < cend)
      load_chunk(c + 1, st ^ 1);
    cp_async_commit();
    if (tid < kC32) wj[tid] = tid < n ? ps.upd * pw(lg, n - 1 - tid + ps.shift) : 0.f;
    cp_async_wait<C::STAGES - 1>();
    __syncthreads();
    if (!STATE_ONLY) {
      {  // scores: rows i0 .., columns tid % 16 and 16 more
        const int i0 = RS * (tid / 16), j0 = tid % 16;
        float s[RS][2];
#pragma unroll
        for (int i = 0; i < RS; ++i) s[i][0] = s[i][1] = 0.f;
        if (j0 < i0 + RS)
#pragma unroll 4
          for (int d = 0; d < DK; d += 4) {
            const float4 a0 = ld4(A + j0 * LD + d), a1 = ld4(A + (j0 + 16) * LD + d);
#pragma unroll
            for (int i = 0; i < RS; ++i) {
              const float4 x = ld4(X + (i0 + i) * LD + d);
              s[i][0] = dot4(x, a0, s[i][0]);
              s[i][1] = dot4(x, a1, s[i][1]);
            }
          }
#pragma unroll
        for (int i = 0; i < RS; ++i)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int j = j0 + 16 * k, lag = i0 + i - j;
            P[(i0 + i) * LP + j] = lag >= 0 ? s[i][k] * (ps.intra * pws[lag]) : 0.f;
          }
      }
      __syncthreads();
      const int i0 = RO * rt;
      float o[RO][4];
#pragma unroll
      for (int i = 0; i < RO; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
#pragma unroll 2
      for (int d = 0; d < DK; d += 4) {
        const float4 s0 = ld4(S + d * DVT + v0), s1 = ld4(S + (d + 1) * DVT + v0), s2 = ld4(S + (d + 2) * DVT + v0),
                     s3 = ld4(S + (d + 3) * DVT + v0);
#pragma unroll
        for (int i = 0; i < RO; ++i) {
          const float4 x = ld4(X + (i0 + i) * LD + d);
          fma4(o[i], x.x, s0);
          fma4(o[i], x.y, s1);
          fma4(o[i], x.z, s2);
          fma4(o[i], x.w, s3);
        }
      }
#pragma unroll
      for (int i = 0; i < RO; ++i) {
        const float f = ps.inter * pws[i0 + i + 1 - ps.shift];
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][k] *= f;
      }
      int j = 0;
      for (; j + 4 <= i0; j += 4) {
        const float4 c_0 = ld4(V + j * DVT + v0), c_1 = ld4(V + (j + 1) * DVT + v0), c_2 = ld4(V + (j + 2) * DVT + v0),
                     c_3 = ld4(V + (j + 3) * DVT + v0);
#pragma unroll
        for (int i = 0; i < RO; ++i) {
          const float4 q = ld4(P + (i0 + i) * LP + j);
          fma4(o[i], q.x, c_0);
          fma4(o[i], q.y, c_1);
          fma4(o[i], q.z, c_2);
          fma4(o[i], q.w, c_3);
        }
      }
      for (; j < i0 + RO; ++j) {  // (a token's own row must not meet later ones, which may not be finite)
        const float4 cj = ld4(V + j * DVT + v0);
#pragma unroll
        for (int i = 0; i < RO; ++i)
          if (j <= i0 + i) fma4(o[i], P[(i0 + i) * LP + j], cj);
      }
#pragma unroll
      for (int i = 0; i < RO; ++i) {
        if (i0 + i >= n) continue;
        const int r = c * kC32 + i0 + i;
        const long long t = rev ? len - 1 - r : r;
        *reinterpret_cast<float4*>(gout + t * ps.os[0] + v0) = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
      }
      __syncthreads();  // S was read
    }
    if (4 * rt < DK) {  // state: rows 4 rt .., and every 4 RT further
      const float wS = pws[n];
      float add[M][4][4];
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) add[m][i][0] = add[m][i][1] = add[m][i][2] = add[m][i][3] = 0.f;
#pragma unroll 2
      for (int j = 0; j < n; ++j) {
        const float wt = wj[j];
        float4 cj = ld4(V + j * DVT + v0);
        cj.x *= wt, cj.y *= wt, cj.z *= wt, cj.w *= wt;
#pragma unroll
        for (int m = 0; m < M; ++m) {
          const float4 a = ld4(A + j * LD + 4 * rt + 4 * C::RT * m);
          fma4(add[m][0], a.x, cj);
          fma4(add[m][1], a.y, cj);
          fma4(add[m][2], a.z, cj);
          fma4(add[m][3], a.w, cj);
        }
      }
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float* at = S + (4 * rt + 4 * C::RT * m + i) * DVT + v0;
          float4 s = ld4(at);
          s.x = fmaf(wS, s.x, add[m][i][0]);
          s.y = fmaf(wS, s.y, add[m][i][1]);
          s.z = fmaf(wS, s.z, add[m][i][2]);
          s.w = fmaf(wS, s.w, add[m][i][3]);
          *reinterpret_cast<float4*>(at) = s;
        }
    }
  }
  cp_async_wait<0>();
  __syncthreads();

  if (STATE_ONLY) {
    float* dst = seg_state(p, w, w.seg + 1, VT, DK * DVT);
    for (int e = tid; e < DK * DVT; e += NT) dst[e] = S[e];
    return;
  }
  if (ps.fin != nullptr &&
      ((len > c0 * kC32 && (long long)len <= (long long)c1 * kC32) || (len == 0 && w.seg == 0))) {
    float* f = ps.fin + (long long)w.bh * DK * p.DV + w.vt * DVT;
    for (int e = tid; e < DK * DVT; e += NT) f[(long long)(e / DVT) * p.DV + e % DVT] = S[e];
  }
  // (not before: the next kernel's CTAs would take the places that this one's leave free, three on some SMs, and keep
  // them: 8 x 2048 gradients one after the other 133 us each instead of 100)
  depend_launch();
  const int rlo = len > c0 * kC32 ? len : c0 * kC32, rhi = c1 * kC32 < p.T ? c1 * kC32 : p.T;
  for (long long e = tid; e < (long long)(rhi - rlo) * C::CT; e += NT)
    *reinterpret_cast<float4*>(gout + (long long)(rlo + e / C::CT) * ps.os[0] + 4 * (e % C::CT)) =
        make_float4(0.f, 0.f, 0.f, 0.f);
}

template <int DK, int DVT>
int launch_cfg(const LinAttnParams& p, cudaStream_t s) {
  using C = La32Cfg<DK, DVT>;
  static int prep_main[64][5], prep_state[64][5];
  int e = prepare_launch(prep_main, linattn_f32_kernel<C, false>, C::SMEM, C::NT, 1);
  if (e != 0) return e;
  const long long base = (long long)p.npass * p.B * p.NH * (p.DV / DVT);
  if (base * p.nseg * (DK * DVT / 256) > 0x7fffffffLL) return (int)cudaErrorInvalidValue;
  if (p.nseg > 1) {
    e = prepare_launch(prep_state, linattn_f32_kernel<C, true>, C::SMEM, C::NT, 1);
    if (e != 0) return e;
    e = launch_dependent(linattn_f32_kernel<C, true>, (unsigned)(base * (p.nseg - 1)), C::NT, C::SMEM, s, p);
    if (e != 0) return e;
    e = launch_dependent(linattn_scan_kernel<RowOrder<C>>, (unsigned)(base * (DK * DVT / 256)), 256, 0, s, p,
                         p.seg_chunks * kC32);
    if (e != 0) return e;
  }
  return launch_dependent(linattn_f32_kernel<C, false>, (unsigned)(base * p.nseg), C::NT, C::SMEM, s, p);
}
template <int DK>
int launch_dk(const LinAttnParams& p, cudaStream_t s) {
  return p.DV % 64 == 0 ? launch_cfg<DK, 64>(p, s) : launch_cfg<DK, 32>(p, s);
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
