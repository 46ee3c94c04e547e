// Gated linear recurrence: the cells without a recurrent matrix.  For each row and channel, with a = sigmoid(f):
//   G = 2 (f, z)        c_t = a c_{t-1} + (1 - a) z_t          y_t = c_t
//   G = 3 (f, z, o)     the same                               y_t = sigmoid(o_t) c_t
//   G = 4 (i, f, z, o)  c_t = a c_{t-1} + sigmoid(i_t) z_t     y_t = sigmoid(o_t) c_t
// Wx [T, B, NH, G D] gate-major, as for the other cells.  A step is the map c -> a c + u, and maps compose:
// (A, U) followed by (a, u) is (a A, a U + u).  So time is cut: a warp takes runs of 8 tokens of 64 channels (two
// neighbouring ones a thread; one, of 32, where the head size is odd), keeps their gates in registers, and makes the run's map
// from them; the CTA's threads of one channel compose the maps of its eight warps -- and those of the cluster's CTAs,
// exchanged in distributed shared memory -- and every warp goes through its run again from the state at its start.  Each
// value is read and written once; maps are composed in one order, whatever the timing.
//
// The gradient is the same with time reversed: with e_t = dy_t sigmoid(o_t), dc_t = e_t + a_{t+1} dc_{t+1}.  Every
// run's state is recomputed from the one at its start, which the forward pass leaves (4 bytes for 8 tokens).
//
// Sums, states and gates are fp32; results are rounded once.  gated_tile.cu does the same on tiles that TMA brings, where sizes
// allow it and there is more than one round; here any size runs, bound by latency: 1024 x 16 tokens of 5 x 33 heads, fz, 10.7 us
// (gradient 15.0), of which bytes are 2.4.  Single tokens are bound by the launch (16 x 768: 1.5 us issued back to back).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "gated.cuh"
#include "kernels.h"
#include "lm.h"
#include "ptx.cuh"

namespace srnn {
namespace {

constexpr int kS = kRunTokens, kWarps = kRunWarps, kChunk = kRunChunk, kMaxCluster = 8;

// V neighbouring channels of one token
template <class T, int V>
struct Raw;
template <>
struct Raw<__nv_bfloat16, 2> {
  uint32_t v;
  __device__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint32_t*>(p); }
  __device__ void zero() { v = 0u; }
  __device__ Num<2> get() const {
    Num<2> r;
    r.x = make_float2(bf16_lo(v), bf16_hi(v));
    return r;
  }
  static __device__ void store(__nv_bfloat16* p, const Num<2>& a) { *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(a.x.x, a.x.y); }
};
template <>
struct Raw<__nv_bfloat16, 1> {
  uint16_t v;
  __device__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint16_t*>(p); }
  __device__ void zero() { v = 0; }
  __device__ Num<1> get() const { return Num<1>(bf16_to_f32(v)); }
  static __device__ void store(__nv_bfloat16* p, const Num<1>& a) { *p = __float2bfloat16_rn(a.x); }
};
template <>
struct Raw<float, 2> {
  float2 v;
  __device__ void load(const float* p) { v = *reinterpret_cast<const float2*>(p); }
  __device__ void zero() { v = make_float2(0.f, 0.f); }
  __device__ Num<2> get() const {
    Num<2> r;
    r.x = v;
    return r;
  }
  static __device__ void store(float* p, const Num<2>& a) { *reinterpret_cast<float2*>(p) = a.x; }
};
template <>
struct Raw<float, 1> {
  float v;
  __device__ void load(const float* p) { v = *p; }
  __device__ void zero() { v = 0.f; }
  __device__ Num<1> get() const { return Num<1>(v); }
  static __device__ void store(float* p, const Num<1>& a) { *p = a.x; }
};

template <int V>
struct Shared {
  alignas(16) Map part[kWarps][32 * V];
  alignas(16) Map all[2][kMaxCluster][32 * V];
  alignas(16) float start[kWarps][32 * V];
};

// what a thread works on
template <class T, int G, int V>
struct Where {
  int b, rank, warp, lane, len, steps, first;  // first: its run's first token of the first round
  bool on;
  long long wx, wstep, ch, ystep;  // elements: token 0's first gate, tokens apart; the channel in [B, N], tokens apart
  long long at;                    // [B, N]: the channel whose state this thread carries from round to round, or -1

  __device__ explicit Where(const GatedParams& p) {
    rank = (int)(blockIdx.x % p.cs);
    const unsigned id = blockIdx.x / p.cs;
    b = (int)(id / p.tiles);
    warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int c0 = (int)(id % p.tiles) * 32 * V, mine = c0 + lane * V, own = c0 + (int)threadIdx.x;
    on = mine < p.N;
    const int c = on ? mine : p.N - V;  // (a thread past the last channel reads another one's values and writes none)
    wstep = (long long)p.B * p.N * G, ystep = (long long)p.B * p.N;
    wx = ((long long)b * p.N + c / p.D * p.D) * G + c % p.D;
    ch = (long long)b * p.N + c;
    at = threadIdx.x < 32 * V && own < p.N ? (long long)b * p.N + own : -1;
    steps = p.cs * kChunk;
    first = rank * kChunk + warp * kS;
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

// The state before this warp's run from the runs' maps m: the CTA's threads of one channel each compose the maps of its
// warps, then those of the cluster's CTAs, in the order of time (REV: against it).  h: the state of thread's own channel
// (Where::at), at the round's beginning; replaced by that at its end.
template <int V, bool REV>
__device__ __forceinline__ Num<V> carry(Shared<V>& sh, int buf, const Num<V>& ma, const Num<V>& mu, int warp, int lane,
                                        int rank, int cs, float& h) {
  Map m[V];
#pragma unroll
  for (int v = 0; v < V; ++v) m[v].a = ma.get(v), m[v].u = mu.get(v);
  if constexpr (V == 2)
    *reinterpret_cast<float4*>(&sh.part[warp][2 * lane]) = make_float4(m[0].a, m[0].u, m[1].a, m[1].u);
  else
    sh.part[warp][lane] = m[0];
  __syncthreads();
  const int c = threadIdx.x;
  const bool fold = c < 32 * V;
  float in = h;
  if (cs > 1) {
    if (fold) {
      Map t{1.f, 0.f};
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        const Map x = sh.part[REV ? kWarps - 1 - i : i][c];
        t.u = fmaf(x.a, t.u, x.u);
        t.a *= x.a;
      }
      const uint32_t to = smem_u32(&sh.all[buf][rank][c]);
      for (int r = 0; r < cs; ++r)
        asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(mapa(to, (uint32_t)r)), "f"(t.a), "f"(t.u) : "memory");
    }
    // (the buffer's readers of two rounds ago were done before the round between)
    __syncwarp();
    cluster_sync();
    if (fold)
      for (int i = 0; i < cs; ++i) {
        const int r = REV ? cs - 1 - i : i;
        const Map x = sh.all[buf][r][c];
        if (r == rank) in = h;
        h = fmaf(x.a, h, x.u);
      }
  }
  if (fold) {
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      const int w = REV ? kWarps - 1 - i : i;
      const Map x = sh.part[w][c];
      sh.start[w][c] = in;
      in = fmaf(x.a, in, x.u);
    }
    if (cs == 1) h = in;
  }
  __syncthreads();
  Num<V> s;
  if constexpr (V == 2)
    s.x = *reinterpret_cast<const float2*>(&sh.start[warp][2 * lane]);
  else
    s.x = sh.start[warp][lane];
  return s;
}

template <class T, int G, int V>
struct Run {  // a run's raw values
  Raw<T, V> x[G][kS];
  // n: tokens of it that count
  __device__ __forceinline__ void load(const T* wx, long long wstep, int D, int n) {
    if (n >= kS) {
#pragma unroll
      for (int s = 0; s < kS; ++s)
#pragma unroll
        for (int g = 0; g < G; ++g) x[g][s].load(wx + s * wstep + (long long)g * D);
    } else {
#pragma unroll
      for (int s = 0; s < kS; ++s)
#pragma unroll
        for (int g = 0; g < G; ++g) {
          x[g][s].zero();
          if (s < n) x[g][s].load(wx + s * wstep + (long long)g * D);
        }
    }
  }
};

template <class T, int G, int V>
__global__ void __launch_bounds__(32 * kWarps) gated_fwd_kernel(const GatedParams p) {
  constexpr int F = G == 4 ? 1 : 0, Z = F + 1, O = G == 2 ? 0 : F + 2;  // the gates' places
  __shared__ Shared<V> sh;
  depend_launch();
  Where<T, G, V> w(p);
  const T* wx = static_cast<const T*>(p.wx) + w.wx + w.first * w.wstep;
  T* y = static_cast<T*>(p.y) + w.ch + w.first * w.ystep;
  depend_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
  w.lengths(p);
  float h = p.state0 && w.at >= 0 ? p.state0[w.at] : 0.f;
  const int rounds = w.rounds();
  __syncwarp();  // (the barrier takes a warp's lanes together)
  if (p.cs > 1) cluster_sync();  // every CTA has begun before another one writes to its shared memory
  Run<T, G, V> raw;
  if (rounds > 0) raw.load(wx, w.wstep, p.D, w.len - w.first);
  int t0 = w.first;
  for (int k = 0; k < rounds; ++k) {
    const int n = w.len - t0;  // tokens from the run's first on that count (none: 0 or less)
    Num<V> a[kS], u[kS], ma(1.f), mu(0.f);
    Raw<T, V> o[kS];
#pragma unroll
    for (int s = 0; s < kS; ++s) {
      Num<V> gain;
      sigmoids<T>(raw.x[F][s].get(), a[s], gain);
      if (G == 4) gain = sigmoid<T>(raw.x[0][s].get());
      u[s] = gain * raw.x[Z][s].get();
      if (G != 2) o[s] = raw.x[O][s];
      if (s >= n) a[s] = Num<V>(1.f), u[s] = Num<V>(0.f);
      mu = fma(a[s], mu, u[s]);
      ma = ma * a[s];
    }
    wx += w.steps * w.wstep;
    if (k + 1 < rounds) raw.load(wx, w.wstep, p.D, n - w.steps);  // the next round's
    Num<V> c = carry<V, false>(sh, k & 1, ma, mu, w.warp, w.lane, w.rank, p.cs, h);
    if (p.stash && w.on && n > 0)
      Raw<float, 1>::store(p.stash + t0 / kS * w.ystep + w.ch, Num<1>(c.get(0))),
          V == 2 ? Raw<float, 1>::store(p.stash + t0 / kS * w.ystep + w.ch + 1, Num<1>(c.get(V - 1))) : (void)0;
    const int room = w.on ? p.T - t0 : 0;
#pragma unroll
    for (int s = 0; s < kS; ++s) {
      c = fma(a[s], c, u[s]);
      Num<V> out = c;
      if (G != 2) out = sigmoid<T>(o[s].get()) * c;
      if (s >= n) out = Num<V>(0.f);
      if (s < room) Raw<T, V>::store(y + s * w.ystep, out);
    }
    y += w.steps * w.ystep;
    t0 += w.steps;
  }
  if (w.on)
    for (long long t = t0; t < p.T; t += w.steps, y += w.steps * w.ystep)
      for (int s = 0; s < kS && t + s < p.T; ++s) Raw<T, V>::store(y + s * w.ystep, Num<V>(0.f));
  if (p.stateT && w.rank == 0 && w.at >= 0) p.stateT[w.at] = h;
}

template <class T, int G, int V>
__global__ void __launch_bounds__(32 * kWarps) gated_bwd_kernel(const GatedParams p) {
  constexpr int F = G == 4 ? 1 : 0, Z = F + 1, O = G == 2 ? 0 : F + 2;
  __shared__ Shared<V> sh;
  depend_launch();
  Where<T, G, V> w(p);
  depend_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
  w.lengths(p);
  float h = p.dstateT && w.at >= 0 ? p.dstateT[w.at] : 0.f;  // gradient of the state after the round's last token
  const int rounds = w.rounds();
  __syncwarp();
  if (p.cs > 1) cluster_sync();
  for (int k = rounds - 1; k >= 0; --k) {
    const int t0 = k * w.steps + w.first, n = w.len - t0;
    const T* wx = static_cast<const T*>(p.wx) + w.wx + t0 * w.wstep;
    const T* dy = static_cast<const T*>(p.dy) + w.ch + t0 * w.ystep;
    Run<T, G, V> raw;
    Run<T, 1, V> up;
    raw.load(wx, w.wstep, p.D, n);
    up.load(dy, w.ystep, 0, n);
    Num<V> c[kS];  // states before each token
#pragma unroll
    for (int v = 0; v < V; ++v) c[0].set(v, n > 0 ? p.stash[t0 / kS * w.ystep + w.ch + v] : 0.f);
    Num<V> a[kS], b[kS], ma(1.f), mu(0.f);  // sigmoid(f), sigmoid(-f)
#pragma unroll
    for (int s = kS - 1; s >= 0; --s) {
      sigmoids<T>(raw.x[F][s].get(), a[s], b[s]);
      Num<V> e = up.x[0][s].get();
      if (G != 2) e = e * sigmoid<T>(raw.x[O][s].get());
      if (s >= n) a[s] = Num<V>(1.f), e = Num<V>(0.f);
      mu = a[s] * (mu + e);
      ma = ma * a[s];
    }
    Num<V> q = carry<V, true>(sh, k & 1, ma, mu, w.warp, w.lane, w.rank, p.cs, h);
#pragma unroll
    for (int s = 0; s + 1 < kS; ++s) {
      const Num<V> gain = G == 4 ? sigmoid<T>(raw.x[0][s].get()) : b[s];
      c[s + 1] = fma(a[s], c[s], gain * raw.x[Z][s].get());
    }
    T* dwx = static_cast<T*>(p.dwx) + w.wx + t0 * w.wstep;
    const int room = w.on ? p.T - t0 : 0;
#pragma unroll
    for (int s = kS - 1; s >= 0; --s) {
      Num<V> g[G];
      const Num<V> z = raw.x[Z][s].get(), e = up.x[0][s].get();
      Num<V> os, oc, is = b[s], ic, si, so;
      Num<V> dc = e + q;
      if (G != 2) {
        sigmoids<T>(raw.x[O][s].get(), os, oc, &so);
        dc = fma(e, os, q);
      }
      if (G == 4) sigmoids<T>(raw.x[0][s].get(), is, ic, &si);
      g[Z] = dc * is;
      g[F] = dc * (G == 4 ? c[s] : minus(c[s], z)) * (a[s] * b[s]);
      if (G == 4) g[0] = dc * z * si;
      if (G != 2) g[O] = e * fma(a[s], c[s], is * z) * so;
      if (s < n) q = a[s] * dc;
      if (s >= n)
#pragma unroll
        for (int j = 0; j < G; ++j) g[j] = Num<V>(0.f);
      if (s < room)
#pragma unroll
        for (int j = 0; j < G; ++j) Raw<T, V>::store(dwx + s * w.wstep + (long long)j * p.D, g[j]);
    }
  }
  if (w.on) {
    long long t = (long long)rounds * w.steps + w.first;
    T* dwx = static_cast<T*>(p.dwx) + w.wx + t * w.wstep;
    for (; t < p.T; t += w.steps, dwx += w.steps * w.wstep)
      for (int s = 0; s < kS && t + s < p.T; ++s)
#pragma unroll
        for (int j = 0; j < G; ++j) Raw<T, V>::store(dwx + s * w.wstep + (long long)j * p.D, Num<V>(0.f));
  }
  if (p.dstate0 && w.rank == 0 && w.at >= 0) p.dstate0[w.at] = h;
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
  Num<V> out(0.f);
  if (slot >= 0 && slot < p.nslots) {
    Raw<T, V> raw[G];
#pragma unroll
    for (int g = 0; g < G; ++g) raw[g].load(wx + (long long)g * p.D);
    float* state = p.state + (long long)slot * p.N + c;
    Num<V> h, a, gain;
#pragma unroll
    for (int v = 0; v < V; ++v) h.set(v, state[v]);
    sigmoids<T>(raw[F].get(), a, gain);
    if (G == 4) gain = sigmoid<T>(raw[0].get());
    h = fma(a, h, gain * raw[Z].get());
#pragma unroll
    for (int v = 0; v < V; ++v) state[v] = h.get(v);
    out = h;
    if (G != 2) out = sigmoid<T>(raw[O].get()) * h;
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
int launch_gv(GatedParams& p, bool bwd, cudaStream_t s, GatedInfo* info) {
  p.tiles = (p.N + 32 * V - 1) / (32 * V);
  // CTAs along time until each SM has two (4000 tokens of 2 x 33, fz: 43.5 us by one CTA, 22.6 by four, 12.7 by eight)
  const long long tiles = (long long)p.tiles * p.B, want = 2LL * sm_count();
  p.cs = 1;
  while (p.cs < 8 && tiles * p.cs < want && p.cs * kChunk < p.T) p.cs *= 2;
  if (tiles * p.cs > 0x7fffffff) return (int)cudaErrorInvalidConfiguration;
  if (info) {
    *info = GatedInfo{(int)(tiles * p.cs), 32 * kWarps, p.cs, 0, 0, 0, 0};
    return 0;
  }
  return launch_cluster(bwd ? gated_bwd_kernel<T, G, V> : gated_fwd_kernel<T, G, V>, (unsigned)(tiles * p.cs), p.cs, s,
                        (const GatedParams)p);
}
template <class T, int G>
int launch_g(GatedParams& p, bool bwd, bool pairs, cudaStream_t s, GatedInfo* info) {
  return pairs ? launch_gv<T, G, 2>(p, bwd, s, info) : launch_gv<T, G, 1>(p, bwd, s, info);
}
template <class T>
int launch_t(GatedParams& p, int gates, bool bwd, cudaStream_t s, GatedInfo* info) {
  auto ok = [](const void* x, size_t n) { return reinterpret_cast<uintptr_t>(x) % n == 0; };
  const bool pairs = p.D % 2 == 0 && ok(p.wx, 2 * sizeof(T)) && ok(p.y, 2 * sizeof(T)) && ok(p.dy, 2 * sizeof(T)) &&
                     ok(p.dwx, 2 * sizeof(T));
  switch (gates) {
    case 2: return launch_g<T, 2>(p, bwd, pairs, s, info);
    case 3: return launch_g<T, 3>(p, bwd, pairs, s, info);
    default: return launch_g<T, 4>(p, bwd, pairs, s, info);
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

int launch_gated(GatedParams p, int gates, bool bf16, bool bwd, cudaStream_t s, GatedInfo* info) {
  if (gated_takes_tiles(p, bf16)) {
    const int e = launch_gated_tile(p, gates, bf16, bwd, s, info);
    if (e != kGatedNoTile || p.withhold) return e;
  }
  return bf16 ? launch_t<__nv_bfloat16>(p, gates, bwd, s, info) : launch_t<float>(p, gates, bwd, s, info);
}
int launch_gated_step(const GatedStepParams& p, int gates, bool bf16, cudaStream_t s) {
  return bf16 ? step_t<__nv_bfloat16>(p, gates, s) : step_t<float>(p, gates, s);
}

}  // namespace srnn
