// Gated linear recurrence: the cells without a recurrent matrix.  For each row and channel, with a = sigmoid(f):
//   G = 2 (f, z)        c_t = a c_{t-1} + (1 - a) z_t          y_t = c_t
//   G = 3 (f, z, o)     the same                               y_t = sigmoid(o_t) c_t
//   G = 4 (i, f, z, o)  c_t = a c_{t-1} + sigmoid(i_t) z_t     y_t = sigmoid(o_t) c_t
// Wx [T, B, NH, G D] gate-major, as for the other cells.  A step is the map c -> a c + u, and maps compose:
// (A, U) followed by (a, u) is (a A, a U + u).  So time is cut: a warp takes runs of 8 tokens of 64 channels (two
// neighbouring ones a thread), keeps their gates in registers, and makes the run's map from them; a CTA's eight
// warps exchange their maps in shared memory, the CTAs of a cluster theirs in distributed shared memory, and every
// warp goes through its run again from the state at its start.  Each value is read and written once; maps
// are composed in one order, whatever the timing.
//
// The gradient is the same with time reversed: with e_t = dy_t sigmoid(o_t), dc_t = e_t + a_{t+1} dc_{t+1}.  Every
// run's state is recomputed from the one at its start, which the forward pass leaves (4 bytes for 8 tokens).
//
// Sums, states and gates are fp32; results are rounded once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "lm.h"
#include "ptx.cuh"

namespace srnn {
namespace {

constexpr int kS = kGatedRun;     // tokens of a run
constexpr int kWarps = 8;         // runs of a CTA side by side
constexpr int kChunk = kS * kWarps;
constexpr int kMaxCluster = 16;

// V neighbouring channels of one token
template <class T, int V>
struct Raw;
template <>
struct Raw<__nv_bfloat16, 2> {
  uint32_t v;
  __device__ void load(const void* p) { v = *static_cast<const uint32_t*>(p); }
  __device__ void zero() { v = 0u; }
  __device__ float get(int i) const { return i ? bf16_hi(v) : bf16_lo(v); }
  static __device__ void store(void* p, const float (&x)[2]) { *static_cast<uint32_t*>(p) = pack_bf16x2(x[0], x[1]); }
};
template <>
struct Raw<__nv_bfloat16, 1> {
  uint16_t v;
  __device__ void load(const void* p) { v = *static_cast<const uint16_t*>(p); }
  __device__ void zero() { v = 0; }
  __device__ float get(int) const { return bf16_to_f32(v); }
  static __device__ void store(void* p, const float (&x)[1]) {
    *static_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(x[0]);
  }
};
template <>
struct Raw<float, 2> {
  float2 v;
  __device__ void load(const void* p) { v = *static_cast<const float2*>(p); }
  __device__ void zero() { v = make_float2(0.f, 0.f); }
  __device__ float get(int i) const { return i ? v.y : v.x; }
  static __device__ void store(void* p, const float (&x)[2]) { *static_cast<float2*>(p) = make_float2(x[0], x[1]); }
};
template <>
struct Raw<float, 1> {
  float v;
  __device__ void load(const void* p) { v = *static_cast<const float*>(p); }
  __device__ void zero() { v = 0.f; }
  __device__ float get(int) const { return v; }
  static __device__ void store(void* p, const float (&x)[1]) { *static_cast<float*>(p) = x[0]; }
};

// s = sigmoid(x) and c = sigmoid(-x): the smaller one from e^-|x|, the larger one as 1 less it, so that both are good to
// a few units of their own last place (a memory of n tokens needs 1 - a to better than 1 / n)
__device__ __forceinline__ void sigmoids(float x, float& s, float& c) {
  const float e = expf(-fabsf(x));
  const float low = __fdividef(e, 1.f + e), high = 1.f - low;
  const bool up = x > 0.f;
  s = up ? high : low;
  c = up ? low : high;
}
__device__ __forceinline__ float sigmoid1(float x) {
  float s, c;
  sigmoids(x, s, c);
  return s;
}

template <int V>
struct Map {  // c -> a c + u
  float a[V], u[V];
};
template <int V>
struct Shared {
  Map<V> part[2][kWarps][32];
  Map<V> all[2][kMaxCluster][32];
};

// what a thread works on
template <class T, int G, int V>
struct Where {
  int b, t0, rank, warp, lane, len, steps;
  bool on;
  long long wx, wstep, ch, ystep;  // elements: token 0's first gate, tokens apart; the channel in [B, N], tokens apart

  __device__ explicit Where(const GatedParams& p) {
    rank = (int)(blockIdx.x % p.cs);
    const unsigned id = blockIdx.x / p.cs;
    b = (int)(id / p.tiles);
    warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int c = (int)(id % p.tiles * 32 + lane) * V;
    on = c < p.N;
    wstep = (long long)p.B * p.N * G, ystep = (long long)p.B * p.N;
    wx = ((long long)b * p.N + c / p.D * p.D) * G + c % p.D;
    ch = (long long)b * p.N + c;
    steps = p.cs * kChunk;
  }
  // (after what writes the lengths)
  __device__ void lengths(const GatedParams& p) {
    len = p.T;
    if (p.lens) {
      const int n = p.lens[b];
      len = n < 0 ? 0 : n < p.T ? n : p.T;
    }
  }
  __device__ int rounds() const { return (int)((len + (long long)steps - 1) / steps); }
};

// Composes the maps of a CTA's warps, then those of the cluster's CTAs, in the order of time (REV: against it).  h: the
// state the round begins with, replaced by the one it ends with; returns the state before this warp's run.
template <int V, bool REV>
__device__ __forceinline__ void carry(Shared<V>& sh, int buf, const Map<V>& mine, int warp, int lane, int rank, int cs,
                                      float (&h)[V], float (&start)[V]) {
  sh.part[buf][warp][lane] = mine;
  __syncthreads();
  Map<V> before, total;
#pragma unroll
  for (int v = 0; v < V; ++v) total.a[v] = 1.f, total.u[v] = 0.f;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    const int w = REV ? kWarps - 1 - i : i;
    if (w == warp) before = total;
    const Map<V> m = sh.part[buf][w][lane];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      total.u[v] = fmaf(m.a[v], total.u[v], m.u[v]);
      total.a[v] *= m.a[v];
    }
  }
  float in[V];
  if (cs == 1) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      in[v] = h[v];
      h[v] = fmaf(total.a[v], h[v], total.u[v]);
    }
  } else {
    // warp w hands the CTA's map to the CTAs w, w + 8; the buffer's last readers were done before the round between
    const uint32_t at = smem_u32(&sh.all[buf][rank][lane]);
    for (int r = warp; r < cs; r += kWarps) {
      const uint32_t to = mapa(at, (uint32_t)r);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 4 * v), "f"(total.a[v]) : "memory");
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 4 * (V + v)), "f"(total.u[v]) : "memory");
      }
    }
    cluster_sync();
    for (int i = 0; i < cs; ++i) {
      const int r = REV ? cs - 1 - i : i;
      const Map<V> m = sh.all[buf][r][lane];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (r == rank) in[v] = h[v];
        h[v] = fmaf(m.a[v], h[v], m.u[v]);
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) start[v] = fmaf(before.a[v], in[v], before.u[v]);
}

template <class T, int G, int V>
__global__ void __launch_bounds__(32 * kWarps) gated_fwd_kernel(const GatedParams p) {
  constexpr int F = G == 4 ? 1 : 0, Z = F + 1, O = F + 2;  // the gates' places
  __shared__ Shared<V> sh;
  depend_launch();
  Where<T, G, V> w(p);
  const T* wx = static_cast<const T*>(p.wx) + w.wx;
  T* y = static_cast<T*>(p.y) + w.ch;
  depend_wait();
  w.lengths(p);
  float h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = p.state0 && w.on ? p.state0[w.ch + v] : 0.f;
  const int rounds = w.rounds();
  if (p.cs > 1) cluster_sync();  // every CTA has begun before another one writes to its shared memory
  for (int k = 0; k < rounds; ++k) {
    const int t0 = k * w.steps + w.rank * kChunk + w.warp * kS;
    const int n = w.on ? min(kS, w.len - t0) : 0;  // tokens that count (none: 0 or less)
    Raw<T, V> raw[G][kS];
#pragma unroll
    for (int s = 0; s < kS; ++s) {
      const T* at = wx + (t0 + s) * w.wstep;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        raw[g][s].zero();
        if (s < n) raw[g][s].load(at + (long long)g * p.D);
      }
    }
    float a[kS][V], u[kS][V];
    Map<V> m;
#pragma unroll
    for (int v = 0; v < V; ++v) m.a[v] = 1.f, m.u[v] = 0.f;
#pragma unroll
    for (int s = 0; s < kS; ++s)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float gain;
        sigmoids(raw[F][s].get(v), a[s][v], gain);
        if (G == 4) gain = sigmoid1(raw[0][s].get(v));
        u[s][v] = gain * raw[Z][s].get(v);
        if (s >= n) a[s][v] = 1.f, u[s][v] = 0.f;
        m.u[v] = fmaf(a[s][v], m.u[v], u[s][v]);
        m.a[v] *= a[s][v];
      }
    float c[V];
    carry<V, false>(sh, k & 1, m, w.warp, w.lane, w.rank, p.cs, h, c);
    if (p.stash && n > 0)
#pragma unroll
      for (int v = 0; v < V; ++v) p.stash[t0 / kS * w.ystep + w.ch + v] = c[v];
#pragma unroll
    for (int s = 0; s < kS; ++s) {
      float out[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        c[v] = fmaf(a[s][v], c[v], u[s][v]);
        out[v] = G == 2 ? c[v] : sigmoid1(raw[G == 2 ? 0 : O][s].get(v)) * c[v];
        if (s >= n) out[v] = 0.f;
      }
      if (w.on && t0 + s < p.T) Raw<T, V>::store(y + (t0 + s) * w.ystep, out);
    }
  }
  if (!w.on) return;
  const float none[V] = {};
  for (long long t = (long long)rounds * w.steps + w.rank * kChunk + w.warp * kS; t < p.T; t += w.steps)
    for (int s = 0; s < kS && t + s < p.T; ++s) Raw<T, V>::store(y + (t + s) * w.ystep, none);
  if (p.stateT && w.rank == 0 && w.warp == 0)
#pragma unroll
    for (int v = 0; v < V; ++v) p.stateT[w.ch + v] = h[v];
}

template <class T, int G, int V>
__global__ void __launch_bounds__(32 * kWarps) gated_bwd_kernel(const GatedParams p) {
  constexpr int F = G == 4 ? 1 : 0, Z = F + 1, O = G == 2 ? 0 : F + 2;
  __shared__ Shared<V> sh;
  depend_launch();
  Where<T, G, V> w(p);
  const T* wx = static_cast<const T*>(p.wx) + w.wx;
  T* dwx = static_cast<T*>(p.dwx) + w.wx;
  const T* dy = static_cast<const T*>(p.dy) + w.ch;
  depend_wait();
  w.lengths(p);
  float d[V];  // gradient of the state after the round's last token
#pragma unroll
  for (int v = 0; v < V; ++v) d[v] = p.dstateT && w.on ? p.dstateT[w.ch + v] : 0.f;
  const int rounds = w.rounds();
  if (p.cs > 1) cluster_sync();
  for (int k = rounds - 1; k >= 0; --k) {
    const int t0 = k * w.steps + w.rank * kChunk + w.warp * kS;
    const int n = w.on ? min(kS, w.len - t0) : 0;
    Raw<T, V> raw[G][kS], up[kS];
#pragma unroll
    for (int s = 0; s < kS; ++s) {
      const T* at = wx + (t0 + s) * w.wstep;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        raw[g][s].zero();
        if (s < n) raw[g][s].load(at + (long long)g * p.D);
      }
      up[s].zero();
      if (s < n) up[s].load(dy + (t0 + s) * w.ystep);
    }
    float c[kS][V];  // states before each token
#pragma unroll
    for (int v = 0; v < V; ++v) c[0][v] = n > 0 ? p.stash[t0 / kS * w.ystep + w.ch + v] : 0.f;
    float a[kS][V], b[kS][V];  // sigmoid(f), sigmoid(-f)
    Map<V> m;
#pragma unroll
    for (int v = 0; v < V; ++v) m.a[v] = 1.f, m.u[v] = 0.f;
#pragma unroll
    for (int s = kS - 1; s >= 0; --s)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        sigmoids(raw[F][s].get(v), a[s][v], b[s][v]);
        float e = up[s].get(v);
        if (G != 2) e *= sigmoid1(raw[O][s].get(v));
        if (s >= n) a[s][v] = 1.f, e = 0.f;
        m.u[v] = a[s][v] * (m.u[v] + e);
        m.a[v] *= a[s][v];
      }
    float q[V];
    carry<V, true>(sh, k & 1, m, w.warp, w.lane, w.rank, p.cs, d, q);
#pragma unroll
    for (int s = 0; s + 1 < kS; ++s)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float gain = G == 4 ? sigmoid1(raw[0][s].get(v)) : b[s][v];
        c[s + 1][v] = fmaf(a[s][v], c[s][v], gain * raw[Z][s].get(v));
      }
#pragma unroll
    for (int s = kS - 1; s >= 0; --s) {
      float g[G][V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float z = raw[Z][s].get(v), slope = a[s][v] * b[s][v];
        float e = up[s].get(v), os = 1.f, oc = 0.f, is = b[s][v], ic = 0.f;
        if (G != 2) sigmoids(raw[O][s].get(v), os, oc);
        if (G == 4) sigmoids(raw[0][s].get(v), is, ic);
        const float dc = fmaf(e, os, q[v]);
        g[Z][v] = dc * is;
        g[F][v] = dc * (G == 4 ? c[s][v] : c[s][v] - z) * slope;
        if (G == 4) g[0][v] = dc * z * (is * ic);
        if (G != 2) g[O][v] = e * fmaf(a[s][v], c[s][v], is * z) * (os * oc);
        if (s < n) q[v] = a[s][v] * dc;
        if (s >= n)
#pragma unroll
          for (int j = 0; j < G; ++j) g[j][v] = 0.f;
      }
      if (w.on && t0 + s < p.T)
#pragma unroll
        for (int j = 0; j < G; ++j) Raw<T, V>::store(dwx + (t0 + s) * w.wstep + (long long)j * p.D, g[j]);
    }
  }
  if (!w.on) return;
  const float none[V] = {};
  for (long long t = (long long)rounds * w.steps + w.rank * kChunk + w.warp * kS; t < p.T; t += w.steps)
    for (int s = 0; s < kS && t + s < p.T; ++s)
#pragma unroll
      for (int j = 0; j < G; ++j) Raw<T, V>::store(dwx + (t + s) * w.wstep + (long long)j * p.D, none);
  if (p.dstate0 && w.rank == 0 && w.warp == 0)
#pragma unroll
    for (int v = 0; v < V; ++v) p.dstate0[w.ch + v] = d[v];
}

// One token of each row against a cache of states: a thread for V channels of a row.
template <class T, int G, int V>
__global__ void __launch_bounds__(128) gated_step_kernel(const GatedStepParams p) {
  constexpr int F = G == 4 ? 1 : 0, Z = F + 1, O = G == 2 ? 0 : F + 2;
  depend_launch();
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x, per = p.N / V;
  if (i >= per * p.B) return;  // (nothing is touched: no need to wait)
  const int b = (int)(i / per), c = (int)(i % per) * V;
  const T* wx = static_cast<const T*>(p.wx) + ((long long)b * p.N + c / p.D * p.D) * G + c % p.D;
  depend_wait();
  const int slot = p.slots ? p.slots[b] : b;
  float out[V] = {};
  if (slot >= 0 && slot < p.nslots) {
    Raw<T, V> raw[G];
#pragma unroll
    for (int g = 0; g < G; ++g) raw[g].load(wx + (long long)g * p.D);
    float* state = p.state + (long long)slot * p.N + c;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float a, gain;
      sigmoids(raw[F].get(v), a, gain);
      if (G == 4) gain = sigmoid1(raw[0].get(v));
      const float h = fmaf(a, state[v], gain * raw[Z].get(v));
      state[v] = h;
      out[v] = G == 2 ? h : sigmoid1(raw[O].get(v)) * h;
    }
  }
  Raw<T, V>::store(static_cast<T*>(p.y) + (long long)b * p.N + c, out);
}

template <class... A>
int launch_cluster(void (*kern)(A...), unsigned grid, int cs, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cs;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cs > 1 ? 2 : 1;
  return (int)cudaLaunchKernelEx(&cfg, kern, args...);
}

template <class T, int G, int V>
int launch_gv(GatedParams& p, bool bwd, cudaStream_t s) {
  p.tiles = (p.N + 32 * V - 1) / (32 * V);
  const long long tiles = (long long)p.tiles * p.B, want = 2LL * sm_count();
  p.cs = 1;
  while (p.cs < 8 && tiles * p.cs < want && p.cs * kChunk < p.T) p.cs *= 2;
  if (tiles * p.cs > 0x7fffffff) return (int)cudaErrorInvalidConfiguration;
  return launch_cluster(bwd ? gated_bwd_kernel<T, G, V> : gated_fwd_kernel<T, G, V>, (unsigned)(tiles * p.cs), p.cs, s,
                        (const GatedParams)p);
}
template <class T, int G>
int launch_g(GatedParams& p, bool bwd, bool pairs, cudaStream_t s) {
  return pairs ? launch_gv<T, G, 2>(p, bwd, s) : launch_gv<T, G, 1>(p, bwd, s);
}
template <class T>
int launch_t(GatedParams& p, int gates, bool bwd, cudaStream_t s) {
  auto ok = [](const void* x, size_t n) { return reinterpret_cast<uintptr_t>(x) % n == 0; };
  const bool pairs = p.D % 2 == 0 && ok(p.wx, 2 * sizeof(T)) && ok(p.y, 2 * sizeof(T)) && ok(p.dy, 2 * sizeof(T)) &&
                     ok(p.dwx, 2 * sizeof(T));
  switch (gates) {
    case 2: return launch_g<T, 2>(p, bwd, pairs, s);
    case 3: return launch_g<T, 3>(p, bwd, pairs, s);
    default: return launch_g<T, 4>(p, bwd, pairs, s);
  }
}

template <class T, int G>
int step_g(const GatedStepParams& p, bool pairs, cudaStream_t s) {
  const long long n = (long long)p.B * p.N / (pairs ? 2 : 1), grid = (n + 127) / 128;
  if (grid > 0x7fffffff) return (int)cudaErrorInvalidConfiguration;
  return launch_dependent(pairs ? gated_step_kernel<T, G, 2> : gated_step_kernel<T, G, 1>, (unsigned)grid, 128, 0, s, p);
}
template <class T>
int step_t(const GatedStepParams& p, int gates, cudaStream_t s) {
  const bool pairs = p.D % 2 == 0 && (reinterpret_cast<uintptr_t>(p.wx) | reinterpret_cast<uintptr_t>(p.y)) % (2 * sizeof(T)) == 0;
  switch (gates) {
    case 2: return step_g<T, 2>(p, pairs, s);
    case 3: return step_g<T, 3>(p, pairs, s);
    default: return step_g<T, 4>(p, pairs, s);
  }
}

}  // namespace

int launch_gated(GatedParams p, int gates, bool bf16, bool bwd, cudaStream_t s) {
  return bf16 ? launch_t<__nv_bfloat16>(p, gates, bwd, s) : launch_t<float>(p, gates, bwd, s);
}
int launch_gated_step(const GatedStepParams& p, int gates, bool bf16, cudaStream_t s) {
  return bf16 ? step_t<__nv_bfloat16>(p, gates, s) : step_t<float>(p, gates, s);
}

}  // namespace srnn
