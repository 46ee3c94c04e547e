// Linear attention, one token for each row out of a cache of states:
//   S <- lambda S + k v^T,   o = scale q S        S [DK, DV] fp32, in place
// Bound by the state's bytes (8 DK DV a row and head, read and written once).
// One CTA per (row, head, 64 or 32 columns): a thread owns four neighbouring
// columns of every (256 / column groups)-th row of S; the partial sums of q S meet in
// shared memory.  64 rows of 12 heads, 64 x 64: 4.7 us with the call, 5.5 TB/s; a thread's rows of S are loaded in batches
// (one after the other, each load waited for the store before it).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "lm.h"
#include "ptx.cuh"

namespace srnn {
namespace {

__device__ __forceinline__ float in1(const float* p) { return *p; }
__device__ __forceinline__ float in1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void out1(float* p, float v) { *p = v; }
__device__ __forceinline__ void out1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <class T, int DK, int VC>
__global__ void __launch_bounds__(128) linattn_step_kernel(const LinAttnStepParams p) {
  constexpr int G = VC / 4, R = 128 / G;  // column groups, rows of S side by side
  __shared__ float qk[2][DK];
  __shared__ float4 part[R][G];
  const int VT = p.DV / VC;
  const int vt = blockIdx.x % VT, bh = blockIdx.x / VT, b = bh / p.NH, h = bh % p.NH;
  const int tid = threadIdx.x, g = tid % G, r0 = tid / G;
  T* o = static_cast<T*>(p.o) + ((long long)b * p.NH + h) * p.DV + vt * VC;
  depend_launch();
  depend_wait();
  const int slot = p.slots ? p.slots[b] : b;
  if (slot < 0 || slot >= p.nslots) {  // a row without a state
    if (tid < VC) out1(o + tid, 0.f);
    return;
  }
  float4* S = reinterpret_cast<float4*>(p.state + (((long long)slot * p.NH + h) * DK) * p.DV + vt * VC) + g;
  const int pitch = p.DV / 4;
  // the thread's rows of S in batches, each loaded whole before its first store
  constexpr int ROWS = DK / R, BATCH = ROWS < 8 ? ROWS : 8;
  float4 s[BATCH];
  auto load = [&](int i0) {
#pragma unroll
    for (int i = 0; i < BATCH; ++i) s[i] = S[(long long)(r0 + (i0 + i) * R) * pitch];
  };
  load(0);
  const T* q = static_cast<const T*>(p.q) + b * p.qs[0] + h * p.qs[1];
  const T* k = static_cast<const T*>(p.k) + b * p.ks[0] + h * p.ks[1];
  const T* v = static_cast<const T*>(p.v) + b * p.vs[0] + h * p.vs[1] + vt * VC;
  for (int i = tid; i < DK; i += 128) {
    qk[0][i] = in1(q + i) * p.scale;
    qk[1][i] = in1(k + i);
  }
  const float lam = expf(p.log_decay[h]);
  float4 v4;
  v4.x = in1(v + 4 * g), v4.y = in1(v + 4 * g + 1), v4.z = in1(v + 4 * g + 2), v4.w = in1(v + 4 * g + 3);
  __syncthreads();
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < ROWS; i0 += BATCH) {
    if (i0) load(i0);
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int d = r0 + (i0 + i) * R;
      const float kd = qk[1][d], qd = qk[0][d];
      float4 x = s[i];
      x.x = fmaf(lam, x.x, kd * v4.x);
      x.y = fmaf(lam, x.y, kd * v4.y);
      x.z = fmaf(lam, x.z, kd * v4.z);
      x.w = fmaf(lam, x.w, kd * v4.w);
      S[(long long)d * pitch] = x;
      acc.x = fmaf(qd, x.x, acc.x);
      acc.y = fmaf(qd, x.y, acc.y);
      acc.z = fmaf(qd, x.z, acc.z);
      acc.w = fmaf(qd, x.w, acc.w);
    }
  }
  part[r0][g] = acc;
  __syncthreads();
  if (tid < VC) {
    float s = 0.f;
    for (int r = 0; r < R; ++r) s += reinterpret_cast<const float*>(&part[r][tid / 4])[tid & 3];
    out1(o + tid, s);
  }
}

template <class T, int DK>
int launch_t(const LinAttnStepParams& p, cudaStream_t s) {
  const long long rows = (long long)p.B * p.NH;
  if (p.DV % 64 == 0)
    return launch_dependent(linattn_step_kernel<T, DK, 64>, (unsigned)(rows * (p.DV / 64)), 128, 0, s, p);
  return launch_dependent(linattn_step_kernel<T, DK, 32>, (unsigned)(rows * (p.DV / 32)), 128, 0, s, p);
}
template <class T>
int launch_dk(const LinAttnStepParams& p, cudaStream_t s) {
  switch (p.DK) {
    case 32: return launch_t<T, 32>(p, s);
    case 64: return launch_t<T, 64>(p, s);
    case 128: return launch_t<T, 128>(p, s);
    case 256: return launch_t<T, 256>(p, s);
    default: return (int)cudaErrorInvalidValue;
  }
}

}  // namespace

int launch_linattn_step(const LinAttnStepParams& p, bool bf16, cudaStream_t s) {
  return bf16 ? launch_dk<__nv_bfloat16>(p, s) : launch_dk<float>(p, s);
}

}  // namespace srnn
