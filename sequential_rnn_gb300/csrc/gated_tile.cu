// Gated linear recurrence on tiles that TMA brings: head sizes that are multiples of 16 bytes, more than 64 tokens (the
// mathematics and the other sizes: gated.cu).
//
// A CTA takes 64 (or 32) channels of a head of one row, and goes through time in rounds of 64 (128) tokens; the CTAs of a cluster take
// neighbouring rounds at once.  A control warp keeps a ring of tiles [tokens][gates][channels] filled.  Eight warps (four of fp32)
// take a run of 8 tokens each: gates and the run's map c -> A c + U in registers, the map handed to
// one more warp, which composes the maps in the order of time -- those of the cluster's CTAs after
// exchanging them by st.async -- and hands every run the state at its start; then the run once more, its results written into
// the tile it came from, from where TMA stores them.  Nothing is read twice and no thread forms an address per token.
//
// Bound by neither bytes nor issue slots alone (24 instructions an element, 44-54% of the slots): 16384 tokens of one row of
// 12 x 64, fz, bf16 take 20 us (3.8 TB/s), rounds one after the other in 240 CTAs on 152 SMs, of which 64 hold one and the
// others two; 1024 x 16, fzo, 23.7 us (4.5 TB/s) with the states for the gradient, and the gradient 38.9 (4.7 TB/s; 384 CTAs
// in 304 places).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "gated.cuh"
#include "kernels.h"
#include "lm.h"
#include "ptx.cuh"
#include "tc.cuh"

namespace srnn {
namespace {

constexpr int kS = kRunTokens;
constexpr int kReady = 1, kStart = 3;           // named barriers, a pair of each: maps there, starts there
// c -> a c + u of two neighbouring channels, as 16 bytes of shared memory
struct Map2 {
  Num<2> a, u;
};
__device__ __forceinline__ void put(float4* at, const Num<2>& a, const Num<2>& u) {
  *at = make_float4(a.x.x, a.x.y, u.x.x, u.x.y);
}
__device__ __forceinline__ Map2 get(const float4* at) {
  const float4 v = *at;
  Map2 m;
  m.a.x = make_float2(v.x, v.y);
  m.u.x = make_float2(v.z, v.w);
  return m;
}

struct TileMaps {
  CUtensorMap wx;                 // [T, B, NH G, D], box [TOKENS, 1, G, X]
  CUtensorMap out;                // y, or dWx by runs
  CUtensorMap dy, stash;          // gradient alone: box [TOKENS, 1, 1, X], [RUNS, 1, 1, X]
};

// X: channels of a tile, 64 or 32; a warp takes 64 / X runs at once, PL lanes each.  W warps for runs: four for fp32, whose
// tiles would otherwise leave room for one CTA on an SM (training, 2001 x 4 tokens of
// 6 x 128, ifzo: 79 us with eight, 67 with four)
template <class T, int G, bool BWD, int X, bool AHEAD>
struct Tile {
  static constexpr int W = sizeof(T) == 4 ? 4 : 8, THREADS = 32 * (W + 2), TALK = 32 * (W + 1);  // TALK: of runs and maps
  static constexpr int PL = X / 2, RUNS = W * 64 / X, TOKENS = RUNS * kS;
  static constexpr uint32_t ROW = X * sizeof(T), TOK = G * ROW, MAPS = X * 8;  // bytes; of a run's maps
  static constexpr uint32_t WX = TOKENS * TOK, DY = BWD ? TOKENS * ROW : 0, ST = BWD ? RUNS * X * 4 : 0;
  static constexpr uint32_t STAGE = WX + DY + ST;
  static constexpr int BUF = AHEAD ? 2 : 1, MOST = AHEAD ? 4 : 3;
  static constexpr uint32_t REST = BUF * (RUNS * MAPS + RUNS * X * 4) + 256 + 128 + 8 * MAPS, ROOM = 224 * 1024;
  // CTAs of an SM, as registers (64 a thread for three with W = 8, 96 for two; 112 and 168 with W = 4) and shared memory allow
  static constexpr bool THREE = !AHEAD && (W == 8 ? !BWD : G < 4 || !BWD) && 3 * (2 * STAGE + REST) <= ROOM;
  static constexpr int CTAS = THREE ? 3 : 2 * ((AHEAD ? 3 : 2) * STAGE + REST) <= ROOM ? 2 : 1;
  static constexpr int FIT = (int)((ROOM / CTAS - REST) / STAGE), STAGES = FIT > MOST ? MOST : FIT;
  static_assert(STAGES >= (AHEAD ? 3 : 2), "the tile of a round ahead needs the stage of two rounds before");
  static constexpr uint32_t PART = STAGES * STAGE, START = PART + BUF * RUNS * MAPS, BARS = START + BUF * RUNS * X * 4,
                            ALL = BARS + 256;
  static constexpr uint32_t smem(int cs) { return ALL + (cs > 1 ? 2 * cs * MAPS : 0) + 128; }
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, int c0, int c1, int c2, int c3, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(src)
               : "memory");
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void bar_arrive(uint32_t id, uint32_t n) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(n) : "memory"); }

// A bounded wait.  Nobody leaves its loop early (the named barriers count on everyone): after one wait has run out the
// others do not wait any more, and what the call writes is not valid.
struct Wait {
  int* status;
  unsigned long long limit_ns;
  volatile int* gave_up;
  template <bool CLUSTER = false>
  __device__ __forceinline__ void on(uint32_t bar, uint32_t parity) const {
    auto there = [&] { return CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity); };
    if (there()) return;
    const uint64_t t0 = globaltimer_ns();
    while (!*gave_up && !there())
      if (globaltimer_ns() - t0 > limit_ns) {
        *gave_up = 1;
        atomicOr(status, kStatusTimeout);
      }
  }
};

// two neighbouring channels in shared memory
template <class T>
__device__ __forceinline__ Num<2> get2(uint32_t at);
template <>
__device__ __forceinline__ Num<2> get2<__nv_bfloat16>(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at));
  Num<2> r;
  r.x = make_float2(bf16_lo(v), bf16_hi(v));
  return r;
}
template <>
__device__ __forceinline__ Num<2> get2<float>(uint32_t at) {
  Num<2> r;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(r.x.x), "=f"(r.x.y) : "r"(at));
  return r;
}
template <class T>
__device__ __forceinline__ void put2(uint32_t at, const Num<2>& a);
template <>
__device__ __forceinline__ void put2<__nv_bfloat16>(uint32_t at, const Num<2>& a) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(pack_bf16x2(a.x.x, a.x.y)) : "memory");
}
template <>
__device__ __forceinline__ void put2<float>(uint32_t at, const Num<2>& a) {
  asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(a.x.x), "f"(a.x.y) : "memory");
}

// One run of a round, forward: maps first, results second.  FULL: all its tokens count (else the first n do).
template <class T, int G, int X, bool FULL>
struct Forward {
  using C = Tile<T, G, false, X, false>;  // (the layout is that of both)
  static constexpr int F = G == 4 ? 1 : 0, Z = F + 1, O = G == 2 ? 0 : F + 2;
  static __device__ __forceinline__ void maps(uint32_t x, int n, Num<2> (&a)[kS], Num<2> (&u)[kS], Num<2>& ma, Num<2>& mu) {
    ma = Num<2>(1.f), mu = Num<2>(0.f);
#pragma unroll
    for (int s = 0; s < kS; ++s) {
      Num<2> gain;
      sigmoids<T>(get2<T>(x + s * C::TOK + F * C::ROW), a[s], gain);
      if (G == 4) gain = sigmoid<T>(get2<T>(x + s * C::TOK));
      u[s] = gain * get2<T>(x + s * C::TOK + Z * C::ROW);
      if (!FULL && s >= n) a[s] = Num<2>(1.f), u[s] = Num<2>(0.f);
      mu = fma(a[s], mu, u[s]);
      ma = ma * a[s];
    }
  }
  // y of token s goes where value s G^0 of the run was: rows of one gate behind one another, each past what is still read
  static __device__ __forceinline__ void results(uint32_t x, int n, const Num<2> (&a)[kS], const Num<2> (&u)[kS], Num<2> c) {
#pragma unroll
    for (int s = 0; s < kS; ++s) {
      c = fma(a[s], c, u[s]);
      Num<2> y = c;
      if (G != 2) y = sigmoid<T>(get2<T>(x + s * C::TOK + O * C::ROW)) * c;
      if (!FULL && s >= n) y = Num<2>(0.f);
      put2<T>(x + s * C::ROW, y);
    }
  }
};

template <class T, int G, int X, bool FULL>
struct Backward {
  using C = Tile<T, G, true, X, false>;
  static constexpr int F = G == 4 ? 1 : 0, Z = F + 1, O = G == 2 ? 0 : F + 2;
  static __device__ __forceinline__ void maps(uint32_t x, uint32_t dy, int n, Num<2> (&a)[kS], Num<2> (&b)[kS], Num<2>& ma,
                                              Num<2>& mu) {
    ma = Num<2>(1.f), mu = Num<2>(0.f);
#pragma unroll
    for (int s = kS - 1; s >= 0; --s) {
      sigmoids<T>(get2<T>(x + s * C::TOK + F * C::ROW), a[s], b[s]);
      Num<2> e = get2<T>(dy + s * C::ROW);
      if (G != 2) e = e * sigmoid<T>(get2<T>(x + s * C::TOK + O * C::ROW));
      if (!FULL && s >= n) a[s] = Num<2>(1.f), e = Num<2>(0.f);
      mu = a[s] * (mu + e);
      ma = ma * a[s];
    }
  }
  // c0: the state before the run; q: the gradient of the state after it
  static __device__ __forceinline__ void results(uint32_t x, uint32_t dy, int n, const Num<2> (&a)[kS],
                                                 const Num<2> (&b)[kS], const Num<2>& c0, Num<2> q) {
    Num<2> c[kS];
    c[0] = c0;
#pragma unroll
    for (int s = 0; s + 1 < kS; ++s) {
      const Num<2> gain = G == 4 ? sigmoid<T>(get2<T>(x + s * C::TOK)) : b[s];
      c[s + 1] = fma(a[s], c[s], gain * get2<T>(x + s * C::TOK + Z * C::ROW));
    }
#pragma unroll
    for (int s = kS - 1; s >= 0; --s) {
      const uint32_t at = x + s * C::TOK;
      Num<2> g[G];
      const Num<2> z = get2<T>(at + Z * C::ROW), e = get2<T>(dy + s * C::ROW);
      Num<2> os, oc, is = b[s], ic, si, so;
      Num<2> dc = e + q;
      if (G != 2) {
        sigmoids<T>(get2<T>(at + O * C::ROW), os, oc, &so);
        dc = fma(e, os, q);
      }
      if (G == 4) sigmoids<T>(get2<T>(at), is, ic, &si);
      g[Z] = dc * is;
      g[F] = dc * (G == 4 ? c[s] : minus(c[s], z)) * (a[s] * b[s]);
      if (G == 4) g[0] = dc * z * si;
      if (G != 2) g[O] = e * fma(a[s], c[s], is * z) * so;
      if (FULL || s < n) q = a[s] * dc;
#pragma unroll
      for (int j = 0; j < G; ++j) put2<T>(at + j * C::ROW, !FULL && s >= n ? Num<2>(0.f) : g[j]);
    }
  }
};

// AHEAD: a run's maps are made a round ahead of its results, while the maps of the round before are on their way
template <class T, int G, bool BWD, int X, bool AHEAD>
__global__ void __launch_bounds__((Tile<T, G, BWD, X, AHEAD>::THREADS), (Tile<T, G, BWD, X, AHEAD>::CTAS))
    gated_tile_kernel(const GatedParams p, const __grid_constant__ TileMaps maps) {
  using C = Tile<T, G, BWD, X, AHEAD>;
  constexpr int PL = C::PL;
  extern __shared__ char dyn[];
  __shared__ int gave_up_s;
  const uint32_t sm = (smem_u32(dyn) + 127u) & ~127u;
  char* const sp = dyn + (sm - smem_u32(dyn));
  float4* const part = reinterpret_cast<float4*>(sp + C::PART);    // maps of the runs: [RUNS][PL pairs of channels]
  float2* const start = reinterpret_cast<float2*>(sp + C::START);  // states before them: the same
  float4* const all = reinterpret_cast<float4*>(sp + C::ALL);      // maps of the CTAs: [2][cs][PL]
  const uint32_t full = sm + C::BARS, empty = full + 8 * C::STAGES, swap = empty + 8 * C::STAGES;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, cs = p.cs;
  const int rank = (int)(blockIdx.x % cs);
  const unsigned id = blockIdx.x / cs;
  const int b = (int)(id / p.tiles), tile = (int)(id % p.tiles), per = (p.D + X - 1) / X;
  const int head = tile / per, c0 = tile % per * X, pl = lane % PL, sub = lane / PL;
  depend_launch();
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::STAGES; ++i) mbar_init(full + 8 * i, 1), mbar_init(empty + 8 * i, C::RUNS);
    for (int i = 0; i < 2; ++i) mbar_init(swap + 8 * i, 1);
    gave_up_s = 0;
    fence_mbar_init();
    fence_async_smem();
  }
  __syncthreads();
  depend_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
  const Wait wait{p.status, p.timeout_ns, &gave_up_s};
  int len = p.T;
  if (p.lens) len = min(max(p.lens[b], 0), p.T);
  const int step = cs * C::TOKENS, rounds = (len + step - 1) / step;
  __syncwarp();
  if (cs > 1) cluster_sync();  // every CTA's barriers are there
  auto round_of = [&](int i) { return BWD ? rounds - 1 - i : i; };
  auto state_at = [&] { return c0 + 2 * pl < p.D ? (long long)b * p.N + (long long)head * p.D + c0 + 2 * pl : -1; };

  if (warp == C::W + 1) {  // ---- copies
    if (lane == 0) {
      tma_prefetch_map(&maps.wx);
      tma_prefetch_map(&maps.out);
      int i = 0;
      for (; i < rounds && !p.withhold; ++i) {
        const int st = i % C::STAGES;
        if (i >= C::STAGES) wait.on(empty + 8 * st, (i / C::STAGES - 1) & 1);
        if (gave_up_s) break;
        const uint32_t at = sm + st * C::STAGE, bar = full + 8 * st;
        const int t0 = round_of(i) * step + rank * C::TOKENS;
        mbar_arrive_expect_tx(bar, C::STAGE);
        tma_load_4d(at, &maps.wx, c0, head * G, b, t0, bar);
        if (BWD) {
          tma_load_4d(at + C::WX, &maps.dy, c0, head, b, t0, bar);
          tma_load_4d(at + C::WX + C::DY, &maps.stash, c0, head, b, t0 / kS, bar);
        }
      }
      if (gave_up_s)  // what was asked for lands before the CTA leaves
        for (int j = i < C::STAGES ? 0 : i - C::STAGES; j < i; ++j) {
          const uint64_t since = globaltimer_ns();
          while (!mbar_try_wait(full + 8 * (j % C::STAGES), (j / C::STAGES) & 1) && globaltimer_ns() - since < 10000000ull) {
          }
        }
    }
    __syncwarp();
  } else if (warp == C::W) {  // ---- maps: two channels a thread, the lanes of one `sub` W runs that follow one another
    const float* from = BWD ? p.dstateT : p.state0;
    const long long at = state_at();
    Num<2> h(0.f);
    if (from && at >= 0) h.x = make_float2(from[at], from[at + 1]);
    auto other = [&](const Num<2>& x) {  // of the lane with the same channels
      Num<2> y;
      y.x = make_float2(__shfl_xor_sync(0xffffffffu, x.x.x, 16), __shfl_xor_sync(0xffffffffu, x.x.y, 16));
      return y;
    };
    struct Runs {
      Map2 m[C::W], t, first;  // the lane's runs; composed: all of the CTA's, those of the lane before it
    };
    auto read = [&](int i, Runs& r) {
      const int buf = AHEAD ? i & 1 : 0;
#pragma unroll
      for (int w = 0; w < C::W; ++w) {
        const int run = sub * C::W + w;
        r.m[w] = get(part + (buf * C::RUNS + (BWD ? C::RUNS - 1 - run : run)) * PL + pl);
      }
      if (cs == 1 && PL == 32) return;
      r.t = r.m[0];
#pragma unroll
      for (int w = 1; w < C::W; ++w) {
        r.t.u = fma(r.m[w].a, r.t.u, r.m[w].u);
        r.t.a = r.m[w].a * r.t.a;
      }
      if constexpr (PL == 16) {
        const Map2 o{other(r.t.a), other(r.t.u)}, last = sub ? r.t : o;
        r.first = sub ? o : r.t;
        r.t.u = fma(last.a, r.first.u, last.u);
        r.t.a = last.a * r.first.a;
      }
    };
    // A CTA sends round i after it has the maps of round i - 1 from every CTA, which had then read all of round i - 2.  (The
    // lanes meet at named barriers between one round and the next.)
    auto send = [&](int i, const Runs& r) {
      if (cs == 1 || gave_up_s) return;
      const int buf = i % 2;
      const uint32_t bar = swap + 8 * buf, slot = smem_u32(&all[(buf * cs + rank) * PL + pl]);
      const uint32_t v[4] = {__float_as_uint(r.t.a.x.x), __float_as_uint(r.t.a.x.y), __float_as_uint(r.t.u.x.x),
                             __float_as_uint(r.t.u.x.y)};
      if (lane == 0) mbar_arrive_expect_tx(bar, cs * C::MAPS);
      for (int k = sub; k < cs; k += 32 / PL) st_async_v4(mapa(slot, (uint32_t)k), v, mapa(bar, (uint32_t)k));
    };
    auto tell_starts = [&](int i, const Runs& r) {
      Num<2> in = h;
      if (cs > 1) {
        const int buf = i % 2;
        wait.on<true>(swap + 8 * buf, (i / 2) & 1);
        const float4* x = all + buf * cs * PL + pl;
#pragma unroll 4
        for (int j = 0; j < cs; ++j) {
          const int k = BWD ? cs - 1 - j : j;
          const Map2 y = get(x + k * PL);
          if (k == rank) in = h;
          h = fma(y.a, h, y.u);
        }
      } else if (PL == 16) {
        h = fma(r.t.a, h, r.t.u);
      }
      if (PL == 16 && sub) in = fma(r.first.a, in, r.first.u);
      const int buf = AHEAD ? i & 1 : 0;
#pragma unroll
      for (int w = 0; w < C::W; ++w) {
        const int run = sub * C::W + w;
        start[(buf * C::RUNS + (BWD ? C::RUNS - 1 - run : run)) * PL + pl] = in.x;
        in = fma(r.m[w].a, in, r.m[w].u);
      }
      if (cs == 1 && PL == 32) h = in;
      __syncwarp();
      bar_arrive(kStart + buf, C::TALK);
    };
    for (int i = 0; i < rounds; ++i) {
      __syncwarp();
      bar_sync(kReady + (AHEAD ? i & 1 : 0), C::TALK);
      Runs r;
      read(i, r);
      send(i, r);
      tell_starts(i, r);
    }
    part[lane] = make_float4(h.x.x, h.x.y, 0.f, 0.f);  // (this warp's alone by now)
  } else {  // ---- runs
    const int run = warp * (32 / PL) + sub;
    const uint32_t base = sm + run * kS * C::TOK, mine = base + pl * 2 * sizeof(T);
    const long long ystep = (long long)p.B * p.N;
    const bool on = c0 + 2 * pl < p.D, tell = pl == 0;  // tell: the lane that speaks for the run
    float* const stash = p.stash + (long long)b * p.N + (long long)head * p.D + c0 + 2 * pl;
    struct Gates {  // of a round
      Num<2> a[kS], u[kS];
    };
    auto first_token = [&](int i) { return round_of(i) * step + rank * C::TOKENS + run * kS; };
    auto is_whole = [&](int n) { return PL == 32 ? n >= kS : (bool)__all_sync(0xffffffffu, n >= kS); };
    int out = -1;  // the stage whose results are on their way out
    auto begin = [&](int i, Gates& g) {
      const int st = i % C::STAGES, n = len - first_token(i);
      const uint32_t x = mine + st * C::STAGE;
      const bool whole = is_whole(n);
      wait.on(full + 8 * st, (i / C::STAGES) & 1);
      Num<2> ma, mu;
      if constexpr (BWD) {
        const uint32_t dy = sm + st * C::STAGE + C::WX + run * kS * C::ROW + pl * 2 * sizeof(T);
        if (whole)
          Backward<T, G, X, true>::maps(x, dy, n, g.a, g.u, ma, mu);
        else
          Backward<T, G, X, false>::maps(x, dy, n, g.a, g.u, ma, mu);
      } else {
        if (whole)
          Forward<T, G, X, true>::maps(x, n, g.a, g.u, ma, mu);
        else
          Forward<T, G, X, false>::maps(x, n, g.a, g.u, ma, mu);
      }
      const int buf = AHEAD ? i & 1 : 0;
      put(part + (buf * C::RUNS + run) * PL + pl, ma, mu);
      __syncwarp();
      bar_arrive(kReady + buf, C::TALK);
      if (out >= 0 && tell) {
        bulk_wait_read_all();
        mbar_arrive(empty + 8 * out);
      }
      out = -1;
    };
    auto finish = [&](int i, const Gates& g) {
      const int st = i % C::STAGES, t0 = first_token(i), n = len - t0, buf = AHEAD ? i & 1 : 0;
      const uint32_t x = mine + st * C::STAGE;
      const bool whole = is_whole(n);
      __syncwarp();
      bar_sync(kStart + buf, C::TALK);
      Num<2> c;
      c.x = start[(buf * C::RUNS + run) * PL + pl];
      if constexpr (BWD) {
        const uint32_t dy = sm + st * C::STAGE + C::WX + run * kS * C::ROW + pl * 2 * sizeof(T);
        const Num<2> before = get2<float>(sm + st * C::STAGE + C::WX + C::DY + (run * X + 2 * pl) * 4);
        if (whole)
          Backward<T, G, X, true>::results(x, dy, n, g.a, g.u, before, c);
        else
          Backward<T, G, X, false>::results(x, dy, n, g.a, g.u, before, c);
      } else {
        if (p.stash && on && n > 0) *reinterpret_cast<float2*>(stash + t0 / kS * ystep) = c.x;
        if (whole)
          Forward<T, G, X, true>::results(x, n, g.a, g.u, c);
        else
          Forward<T, G, X, false>::results(x, n, g.a, g.u, c);
      }
      fence_async_smem();
      __syncwarp();
      if (tell) {
        if (t0 < p.T) tma_store_4d(&maps.out, c0, BWD ? head * G : head, b, t0, base + st * C::STAGE);
        bulk_commit();
      }
      out = st;
    };
    if constexpr (AHEAD) {
      Gates even, odd;
      if (rounds > 0) begin(0, even);
      for (int i = 0; i < rounds; i += 2) {
        if (i + 1 < rounds) begin(i + 1, odd);
        finish(i, even);
        if (i + 1 >= rounds) break;
        if (i + 2 < rounds) begin(i + 2, even);
        finish(i + 1, odd);
      }
    } else {
      Gates g;
      for (int i = 0; i < rounds; ++i) {
        begin(i, g);
        finish(i, g);
      }
    }
    // rows of zeros behind the last round: from a run's place in the first stage, which nothing uses any more
    if (rounds * (long long)step < p.T) {
      if (tell) bulk_wait_read_all();
      __syncwarp();
#pragma unroll
      for (int s = 0; s < kS; ++s)
#pragma unroll
        for (int j = 0; j < (BWD ? G : 1); ++j) put2<T>(mine + (BWD ? s * C::TOK + j * C::ROW : s * C::ROW), Num<2>(0.f));
      fence_async_smem();
      __syncwarp();
      if (tell) {
        for (long long t = (long long)rounds * step + rank * C::TOKENS + run * kS; t < p.T; t += step)
          tma_store_4d(&maps.out, c0, BWD ? head * G : head, b, (int)t, base);
        bulk_commit();
      }
    }
    if (tell) bulk_wait_all();
  }
  __syncwarp();
  if (cs > 1) {
    __syncthreads();
    cluster_sync();  // (every CTA has read the initial state, whose place the final one may take)
    if (gave_up_s) {  // (maps that other CTAs sent after this one had given up land)
      const uint64_t since = globaltimer_ns();
      while (globaltimer_ns() - since < 100000ull) __nanosleep(1000);
    }
  }
  float* const to = BWD ? p.dstate0 : p.stateT;
  const long long at = state_at();
  if (warp == C::W && to && rank == 0 && sub == 0 && at >= 0) to[at] = part[lane].x, to[at + 1] = part[lane].y;
}

}  // namespace

// ------------------------------------------------------------- host side --
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn();  // tc_gemm.cu

namespace {

// [T, B, heads, D] contiguous, boxes of `rows` tokens, `h` heads and `x` channels
bool encode(CUtensorMap* map, const void* ptr, bool bf16, long long D, long long heads, long long B, long long T, uint32_t x,
            uint32_t h, uint32_t rows) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr || reinterpret_cast<uintptr_t>(ptr) % 16 != 0) return false;
  const cuuint64_t es = bf16 ? 2 : 4, d = (cuuint64_t)D * es;
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)B, (cuuint64_t)T};
  const cuuint64_t strides[3] = {d, d * heads, d * heads * B};
  const cuuint32_t box[4] = {x, h, 1, rows}, ones[4] = {1, 1, 1, 1};
  return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, const_cast<void*>(ptr), dims,
            strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class T, int G, bool BWD, int X, bool AHEAD>
struct Variant {
  using C = Tile<T, G, BWD, X, AHEAD>;
  static constexpr auto kernel = gated_tile_kernel<T, G, BWD, X, AHEAD>;

  static void attributes(cudaLaunchAttribute (&attr)[2], int cs) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cs;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  }
  // the kernel's attributes, once a device; a cudaError_t value.  (Where the device cannot hold a cluster of the largest
  // size, active() says so, and there are smaller ones.)
  static int prepare() {
    static int prep[64][5];
    const int e = prepare_launch(prep, kernel, C::smem(kGatedCluster), C::THREADS, kGatedCluster);
    return e == -1 ? prepare_launch(prep, kernel, C::smem(kGatedCluster), C::THREADS, 1) : e;
  }
  // Shared memory of a launch of which `each` CTAs come to an SM: so much that no more of them fit one (a cluster's would pack two
  // or three to it); 0: what they need.
  static uint32_t smem_for(int cs, int each) {
    const uint32_t need = C::smem(cs), spread = each > 0 ? 226 * 1024 / (each + 1) + 1024 : 0;
    return spread > need ? spread : need;
  }
  // clusters of cs CTAs with smem_for(cs, each) that the device holds at once (0: none, or not to be had)
  static int active(int cs, int each, int dev) {
    static int known[64][kGatedCluster + 1][C::CTAS];  // one more than it, once asked for
    if (dev >= 64) return 0;
    int& k = known[dev][cs][each];
    if (k == 0) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(cs);
      cfg.blockDim = dim3(C::THREADS);
      cfg.dynamicSmemBytes = smem_for(cs, each);
      cudaLaunchAttribute attr[2];
      attributes(attr, cs);
      cfg.attrs = attr + 1;
      cfg.numAttrs = 1;
      int n = 0;
      if (prepare() != 0 || cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) n = 0;
      k = n + 1;
    }
    return k - 1;
  }
  // Few CTAs are spread evenly over the SMs (one row of 16384 tokens of 2 x 64, ifzo: gradient 25.1 us against 32.5), unless the
  // clusters then do not all fit at once, which keep to the SMs of one group (12 of 12 CTAs, 16384 tokens of 12 x 32, fz: 25.4 us one
  // to an SM, of which 8 fit, 17.6 packed).
  static int each_of(int cs, long long clusters, int dev) {
    const long long each = (clusters * cs + sm_count() - 1) / sm_count();
    if (each >= C::CTAS) return 0;
    return cs == 1 || active(cs, (int)each, dev) >= clusters ? (int)each : 0;
  }
  static int launch(GatedParams p, int cs, cudaStream_t s, GatedInfo* info) {
    const bool bf16 = sizeof(T) == 2;
    const long long NH = p.N / p.D;
    TileMaps m;
    if (!info) {
      bool ok = encode(&m.wx, p.wx, bf16, p.D, NH * G, p.B, p.T, X, G, C::TOKENS);
      if (BWD)
        ok = ok && encode(&m.out, p.dwx, bf16, p.D, NH * G, p.B, p.T, X, G, kS) &&
             encode(&m.dy, p.dy, bf16, p.D, NH, p.B, p.T, X, 1, C::TOKENS) &&
             encode(&m.stash, p.stash, false, p.D, NH, p.B, (p.T + kS - 1) / kS, X, 1, C::RUNS);
      else
        ok = ok && encode(&m.out, p.y, bf16, p.D, NH, p.B, p.T, X, 1, kS) && reinterpret_cast<uintptr_t>(p.stash) % 8 == 0;
      if (!ok) return kGatedNoTile;
    }
    p.tiles = (int)(NH * ((p.D + X - 1) / X));
    p.cs = cs;
    const long long clusters = (long long)p.tiles * p.B, ctas = clusters * cs;
    if (ctas > 0x7fffffff) return (int)cudaErrorInvalidConfiguration;
    const int e = prepare();
    if (e != 0) return e;
    int dev = 0;
    cudaGetDevice(&dev);
    const int each = each_of(cs, clusters, dev);
    const uint32_t smem = smem_for(cs, each);
    if (info) {
      const int held = cs > 1 ? active(cs, each, dev) : (each ? each : C::CTAS) * sm_count();
      *info = GatedInfo{(int)ctas, C::THREADS, cs, X, AHEAD, (int)smem, held};
      return 0;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attributes(attr, cs);
    cfg.attrs = attr;
    cfg.numAttrs = cs > 1 ? 2 : 1;
    return (int)cudaLaunchKernelEx(&cfg, kernel, (const GatedParams)p, (const TileMaps)m);
  }
};

// Which of them, and how many CTAs along time: the one whose rounds end first.  A round of bf16 runs of two gates takes
// 0.76 us where maps are made ahead, else 0.80 (CTAs by themselves) or 1.13 (clusters), and 0.46 more for each other
// CTA on the SM.  Other gates, types and the gradient take 1.5 to 2 times as long, roughly alike, so that only the
// wave's 0.3 us weigh too much there; the gradient's and fp32's choices were not timed against all others.  What does
// not fit the device at once runs after it.
struct Plan {
  double cost = 1e30;
  int variant = 0, cs = 1, dev = 0, sms = sm_count();
  Plan() { cudaGetDevice(&dev); }
  template <class V>
  void consider(int variant_, const GatedParams& p, bool ahead) {
    using C = typename V::C;
    const long long tiles = (long long)(p.N / p.D) * ((p.D + 2 * C::PL - 1) / (2 * C::PL)) * p.B;
    const int chunks = (p.T + C::TOKENS - 1) / C::TOKENS;
    for (int c = 1; c <= kGatedCluster && c <= chunks; ++c) {
      const long long room = c == 1 ? (long long)C::CTAS * sms : V::active(c, 0, dev);
      if (room < 1) continue;
      auto wave = [&](long long clusters) {
        if (clusters == 0) return 0.0;
        const long long each = (clusters * c + sms - 1) / sms;
        const double k = (double)(each < C::CTAS ? each : C::CTAS);
        return (chunks + c - 1) / c * ((ahead ? 0.76 : c == 1 ? 0.80 : 1.13) + 0.46 * (k - 1)) + 0.3;
      };
      const double t = (double)(tiles / room) * wave(room) + wave(tiles % room);
      if (t < cost) cost = t, variant = variant_, cs = c;
    }
  }
};
template <class T, int G, bool BWD>
int launch_planned(const GatedParams& p, cudaStream_t s, GatedInfo* info) {
  Plan plan;
  plan.consider<Variant<T, G, BWD, 64, false>>(0, p, false);
  plan.consider<Variant<T, G, BWD, 32, false>>(1, p, false);
  constexpr bool AHEAD = !BWD && sizeof(T) == 2;  // (the others lack registers or shared memory for it)
  if constexpr (AHEAD) {
    plan.consider<Variant<T, G, BWD, 64, true>>(2, p, true);
    plan.consider<Variant<T, G, BWD, 32, true>>(3, p, true);
  }
  switch (plan.variant) {
    case 0: return Variant<T, G, BWD, 64, false>::launch(p, plan.cs, s, info);
    case 1: return Variant<T, G, BWD, 32, false>::launch(p, plan.cs, s, info);
    case 2: return Variant<T, G, BWD, 64, AHEAD>::launch(p, plan.cs, s, info);
    default: return Variant<T, G, BWD, 32, AHEAD>::launch(p, plan.cs, s, info);
  }
}
template <class T, int G>
int launch_dir(const GatedParams& p, bool bwd, cudaStream_t s, GatedInfo* info) {
  return bwd ? launch_planned<T, G, true>(p, s, info) : launch_planned<T, G, false>(p, s, info);
}
template <class T>
int launch_t(const GatedParams& p, int gates, bool bwd, cudaStream_t s, GatedInfo* info) {
  switch (gates) {
    case 2: return launch_dir<T, 2>(p, bwd, s, info);
    case 3: return launch_dir<T, 3>(p, bwd, s, info);
    default: return launch_dir<T, 4>(p, bwd, s, info);
  }
}

}  // namespace

// (up to 64 tokens, one round, they are no faster than gated.cu's kernels, 16 rows of 12 x 64, fz: 2.95 us against 2.99; with 128
// 3.6 against 7.0)
bool gated_takes_tiles(const GatedParams& p, bool bf16) { return p.D % (bf16 ? 8 : 4) == 0 && p.T >= kGatedTileTokens; }

int launch_gated_tile(const GatedParams& p, int gates, bool bf16, bool bwd, cudaStream_t s, GatedInfo* info) {
  return bf16 ? launch_t<__nv_bfloat16>(p, gates, bwd, s, info) : launch_t<float>(p, gates, bwd, s, info);
}

}  // namespace srnn
