// Linear attention with a decay for each head, bf16, head sizes that are a
// multiple of 64: the chunked passes of linattn.cu on the 5th-generation tensor
// cores (tcgen05, accumulators in TMEM), chunks of 128 tokens, in two kernels.
//
//   states   S <- lambda^n S + a^T (weighted c), chunk by chunk; leaves the state at
//            every chunk's start (bf16, an operand of the next kernel) and the final one
//   outputs  out = mask(x a^T) c + decay (x S), all chunks at once
//
// Split in two, only the cheap part (one product of the three) is sequential, and the
// outputs fill the GPU with independent CTAs whose loads, MMAs and epilogues overlap one
// another's; the chunk states cost 2 Dk Dv bytes per 128 tokens and head, written and
// read once, mostly inside L2.
//
// The states' CTA holds 128 (or 64) x 64 of S in fp32 registers.  c times its weight is split into
// three bf16 terms (24 bits), so that the state does not lose to operand rounding what fp32
// keeps; the three products of a chunk accumulate from zero, smallest first, in TMEM, and the
// sum joins the decayed state in round-to-nearest.
// Shared-memory tiles are rows of 64 values (128 bytes, 128-byte swizzle): the same tile
// is a K-major operand (scores) and an MN-major one (state update, P c, x S).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "linattn.cuh"
#include "lm.h"
#include "ptx.cuh"
#include "tc.cuh"

namespace srnn {
namespace {

constexpr int kTC = 128;                     // tokens per chunk
constexpr int kTT = 256;                     // threads per CTA
constexpr uint32_t kBlkBytes = kTC * 128;    // 128 rows x 64 columns

__device__ __forceinline__ void zfill16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// offset of 16-byte chunk ch (of all blocks) of row r
__device__ __forceinline__ uint32_t blk_at(int r, int ch) {
  return (uint32_t)(ch >> 3) * kBlkBytes + (uint32_t)(r * 128 + (((ch & 7) ^ (r & 7)) << 4));
}

struct TcWait {
  int* status;
  unsigned long long limit_ns;
  volatile int* abort_flag;
};
// mbarrier wait bounded in time: a wait that runs out sets the status word and the
// CTA's abort flag
__device__ __forceinline__ bool tc_wait(uint32_t bar, uint32_t parity, const TcWait& w) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*w.abort_flag) return false;
    if (globaltimer_ns() - t0 > w.limit_ns) {
      *w.abort_flag = 1;
      atomicOr(w.status, kStatusTimeout);
      return false;
    }
  }
}

// 128 rows (tokens r0 ..) x D columns of a strided operand into swizzled blocks
template <int D>
__device__ __forceinline__ void load_rows(uint32_t dst, const __nv_bfloat16* src, long long stride,
                                          int r0, int len, bool rev) {
  constexpr int CH = D / 8;
#pragma unroll
  for (int i = 0; i < kTC * CH / kTT; ++i) {
    const int e = threadIdx.x + i * kTT, row = e / CH, ch = e % CH, r = r0 + row;
    const bool ok = r < len;
    const long long t = ok ? (rev ? len - 1 - r : r) : 0;
    zfill16(dst + blk_at(row, ch), src + t * stride + ch * 8, ok);
  }
}

template <int DK>
struct StCfg {
  static constexpr int DKB = DK < 128 ? DK : 128;   // state rows (dk) per CTA
  static constexpr int MB = DK / DKB;
  static constexpr uint32_t A = (DKB / 64) * kBlkBytes;
  static constexpr int NA = 3;                      // buffers of a: two chunks ahead
  // sets of c's three terms.  With two, a chunk's terms are made while the one before is
  // multiplied; with 64 state rows one set, so that two CTAs fit on an SM.
  static constexpr int NT = DKB == 128 ? 2 : 1;
  static constexpr int OCC = DKB == 128 ? 1 : 2;
  // (with 64 state rows the MMA's other 64 rows read the tile behind a, and are not used)
  static constexpr uint32_t SMEM = NA * A + NT * 3 * kBlkBytes + 1024;
  static constexpr int TILE = DKB * 64;
};

// workspace order of a state tile: quad by quad, the active threads' float4 side by side
template <int DK>
struct TcOrder {
  static constexpr int TILE = StCfg<DK>::TILE;
  static __device__ __forceinline__ int tiles(const LinAttnParams& p) {
    return StCfg<DK>::MB * (p.DV / 64);
  }
  static __device__ __forceinline__ void at(const LinAttnParams& p, int tile, int e, int& dk, int& v) {
    constexpr int DKB = StCfg<DK>::DKB;
    const int vts = p.DV / 64, th = (e / 4) % (2 * DKB);
    dk = (tile / vts) * DKB + th % DKB;
    v = (tile % vts) * 64 + 32 * (th / DKB) + 4 * (e / (8 * DKB)) + (e & 3);
  }
};

// STATE_ONLY: a segment's own contribution to the state, from zero, into the workspace.
template <int DK, bool STATE_ONLY>
__global__ void __launch_bounds__(kTT, StCfg<DK>::OCC)
    linattn_states_kernel(const __grid_constant__ LinAttnParams p) {
  using C = StCfg<DK>;
  constexpr int DKB = C::DKB;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ int abort_flag_s;
  __shared__ uint32_t tslot_s;
  __shared__ __align__(8) uint64_t bar_s;
  const uint32_t sm = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sC = sm + C::NA * C::A;
  const uint32_t bar = smem_u32(&bar_s);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int vts = p.DV / 64;
  const Where w = where_of(p, C::MB * vts, STATE_ONLY ? p.nseg - 1 : p.nseg);
  const LinAttnPass& ps = p.pass[w.job];
  const int mb = w.vt / vts, vt = w.vt % vts;
  const int len = row_len(p, w.b);
  const int nch = (p.T + kTC - 1) / kTC;
  const int c0 = w.seg * p.seg_chunks;
  const int c1 = c0 + p.seg_chunks < nch ? c0 + p.seg_chunks : nch;
  const int lch = (len + kTC - 1) / kTC;
  const int cend = c1 < lch ? c1 : lch;
  if (STATE_ONLY && (long long)c1 * kTC >= len) return;
  if (!STATE_ONLY && c0 >= cend && w.seg != 0) return;  // nothing to add, nothing to leave
  const float lg = p.log_decay[w.h] * 1.4426950408889634f;
  const bool rev = ps.reverse != 0;
  const TcWait tw{p.status, p.timeout_ns, &abort_flag_s};

  if (tid == 0) {
    mbar_init(bar, 1);
    abort_flag_s = 0;
    fence_mbar_init();
    fence_async_smem();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(&tslot_s), 64);
    tmem_relinquish();
  }
  const __nv_bfloat16* ga =
      static_cast<const __nv_bfloat16*>(ps.a) + w.b * ps.as[1] + w.h * ps.as[2] + mb * DKB;
  const __nv_bfloat16* gc =
      static_cast<const __nv_bfloat16*>(ps.c) + w.b * ps.cs[1] + w.h * ps.cs[2] + vt * 64;

  // c of a chunk: rows tid / 8 + 32 i, 16-byte chunk tid % 8
  uint4 cr[4];
  auto load_c = [&](int c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = c * kTC + tid / 8 + 32 * i;
      const long long t = rev ? len - 1 - r : r;
      cr[i] = r < len ? *reinterpret_cast<const uint4*>(gc + t * ps.cs[0] + (tid % 8) * 8)
                      : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  auto load_a = [&](int c) {
    if (c < cend) load_rows<DKB>(sm + ((c - c0) % C::NA) * C::A, ga, ps.as[0], c * kTC, len, rev);
    cp_async_commit();
  };
  if (c0 < cend) load_c(c0);
  load_a(c0);
  load_a(c0 + 1);

  // ---- the state at the segment's start: row dk = 32 q + lane, 32 columns --
  const int q = warp & 3, half = warp >> 2;
  const bool owner = 32 * q < DKB;
  const int dk = 32 * q + lane, th = half * DKB + dk;
  float S[32];
#pragma unroll
  for (int j = 0; j < 32; ++j) S[j] = 0.f;
  if (!STATE_ONLY && owner) {
    if (p.nseg > 1) {
      const float4* src = reinterpret_cast<const float4*>(seg_state(p, w, w.seg, C::MB * vts, C::TILE));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 f = src[i * 2 * DKB + th];
        S[4 * i] = f.x, S[4 * i + 1] = f.y, S[4 * i + 2] = f.z, S[4 * i + 3] = f.w;
      }
    } else if (ps.init != nullptr) {
      const int gk = mb * DKB + dk, gv = vt * 64 + 32 * half;
      const float* in = ps.init + (long long)w.bh * DK * p.DV;
      if (ps.init_t) {
#pragma unroll
        for (int j = 0; j < 32; ++j) S[j] = in[(long long)(gv + j) * DK + gk];
      } else {
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 f = *reinterpret_cast<const float4*>(in + (long long)gk * p.DV + gv + j);
          S[j] = f.x, S[j + 1] = f.y, S[j + 2] = f.z, S[j + 3] = f.w;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tslot_s;

  constexpr uint32_t idesc = idesc_bf16_f32(128, 64, true, true);
  float wj[4];
  int wn = -1;
  // weighted c of chunk c (in cr) in three bf16 terms; then the next chunk's c on its way
  auto make_terms = [&](int c) {
    const int n = len - c * kTC < kTC ? len - c * kTC : kTC;
    if (wn != n) {
      wn = n;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = tid / 8 + 32 * i;
        wj[i] = j < n ? ps.upd * pw(lg, n - 1 - j + ps.shift) : 0.f;
      }
    }
    const uint32_t set = sC + ((c - c0) % C::NT) * (3 * kBlkBytes);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t in[4] = {cr[i].x, cr[i].y, cr[i].z, cr[i].w};
      uint32_t t[3][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float x0 = bf16_lo(in[k]) * wj[i], x1 = bf16_hi(in[k]) * wj[i];
        t[0][k] = pack_bf16x2(x0, x1);
        x0 -= bf16_lo(t[0][k]);
        x1 -= bf16_hi(t[0][k]);
        t[1][k] = pack_bf16x2(x0, x1);
        x0 -= bf16_lo(t[1][k]);
        x1 -= bf16_hi(t[1][k]);
        t[2][k] = pack_bf16x2(x0, x1);
      }
      const uint32_t at = set + blk_at(tid / 8 + 32 * i, tid % 8);
#pragma unroll
      for (int m = 0; m < 3; ++m)
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at + m * kBlkBytes), "r"(t[m][0]),
                     "r"(t[m][1]), "r"(t[m][2]), "r"(t[m][3])
                     : "memory");
    }
    if (c + 1 < cend) load_c(c + 1);
  };
  if (c0 < cend) make_terms(c0);
  for (int c = c0; c < cend; ++c) {
    const int it = c - c0, n = len - c * kTC < kTC ? len - c * kTC : kTC;
    cp_async_wait<1>();   // this chunk's a (the next one's may be on its way)
    fence_async_smem();
    tc_fence_before();    // (this CTA's reads of the previous sum)
    __syncthreads();
    if (tid == 0) {
      tc_fence_after();
      const uint32_t sA = sm + (it % C::NA) * C::A, set = sC + (it % C::NT) * (3 * kBlkBytes);
#pragma unroll
      for (int term = 2; term >= 0; --term)
#pragma unroll
        for (int ks = 0; ks < kTC / 16; ++ks)
          umma_bf16(tmem, sdesc_sw128(sA + ks * 2048, kBlkBytes, 1024),
                    sdesc_sw128(set + term * kBlkBytes + ks * 2048, kBlkBytes, 1024), idesc,
                    (term != 2 || ks != 0) ? 1u : 0u);
      umma_commit(bar);
    }
    load_a(c + 2);  // into the buffer that the previous chunk's MMAs have read
    if (!STATE_ONLY && owner) {  // the state at this chunk's start
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.chunk_states) +
                           ((((long long)w.job * p.B * p.NH + w.bh) * nch + c) * DK + mb * DKB + dk) * p.DV +
                           vt * 64 + 32 * half;
#pragma unroll
      for (int j = 0; j < 32; j += 8)
        *reinterpret_cast<uint4*>(dst + j) =
            make_uint4(pack_bf16x2(S[j], S[j + 1]), pack_bf16x2(S[j + 2], S[j + 3]),
                       pack_bf16x2(S[j + 4], S[j + 5]), pack_bf16x2(S[j + 6], S[j + 7]));
    }
    if (C::NT == 2 && c + 1 < cend) make_terms(c + 1);
    const float wS = pw(lg, n);
    if (!tc_wait(bar, it & 1, tw)) break;
    tc_fence_after();
    if (owner) {
      uint32_t r[32];
      tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + 32 * half, r);
      tmem_wait_ld();
      tmem_reg_fence(r);
#pragma unroll
      for (int j = 0; j < 32; ++j) S[j] = fmaf(wS, S[j], __uint_as_float(r[j]));
    }
    if (C::NT == 1 && c + 1 < cend) make_terms(c + 1);
  }
  cp_async_wait<0>();

  if (owner) {
    if (STATE_ONLY) {
      float4* dst = reinterpret_cast<float4*>(seg_state(p, w, w.seg + 1, C::MB * vts, C::TILE));
#pragma unroll
      for (int i = 0; i < 8; ++i)
        dst[i * 2 * DKB + th] = make_float4(S[4 * i], S[4 * i + 1], S[4 * i + 2], S[4 * i + 3]);
    } else if (ps.fin != nullptr &&
               ((len > c0 * kTC && (long long)len <= (long long)c1 * kTC) || (len == 0 && w.seg == 0))) {
      float* f = ps.fin + ((long long)w.bh * DK + mb * DKB + dk) * p.DV + vt * 64 + 32 * half;
#pragma unroll
      for (int j = 0; j < 32; j += 4)
        *reinterpret_cast<float4*>(f + j) = make_float4(S[j], S[j + 1], S[j + 2], S[j + 3]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 64);
  }
}

template <int DK>
struct OutCfg {
  static constexpr uint32_t X = (DK / 64) * kBlkBytes;
  // x and a of one tile.  Scores in bf16 (32 KB) take the place of a once it has been multiplied
  // (with 64 columns of a, its 16 KB and 16 KB more).
  static constexpr int NXA = DK <= 128 ? 2 : 1;        // tiles of x and a: the next one is loaded early
  static constexpr uint32_t XTRA = X < 2 * kBlkBytes ? kBlkBytes : 0;
  static constexpr uint32_t S = DK * 128;              // DK rows x 64 columns of the state
  static constexpr int NCS = DK >= 128 ? 2 : 1;        // c and state tiles of 64 columns
  // with 256 columns the second state tile lies in a's upper half, free after the scores
  static constexpr uint32_t CS = DK == 256 ? 2 * kBlkBytes + S : NCS * (kBlkBytes + S);
  static constexpr uint32_t SMEM = NXA * 2 * X + XTRA + CS + 1024;
  static constexpr int OCC = DK == 64 ? 2 : 1;
  static constexpr int NO = OCC == 1 ? 2 : 1;          // sums (P c and x S) in TMEM
  static constexpr uint32_t TMEM = OCC == 1 ? 512 : 256;
};

// A persistent CTA walks (row, head, chunk, pass) tiles, the passes of a chunk side by
// side on the grid, since they read the same tokens.
template <int DK>
__global__ void __launch_bounds__(kTT, OutCfg<DK>::OCC)
    linattn_outputs_kernel(const __grid_constant__ LinAttnParams p, int tiles) {
  using C = OutCfg<DK>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ int abort_flag_s;
  __shared__ uint32_t tslot_s;
  __shared__ __align__(8) uint64_t bar_s;
  __shared__ float pows[kTC];  // intra lambda^m
  const uint32_t sm = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sXtra = sm + C::NXA * 2 * C::X, sCS = sXtra + C::XTRA;
  const uint32_t bar = smem_u32(&bar_s);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q = warp & 3, half = warp >> 2, row = 32 * q + lane;
  const int nch = (p.T + kTC - 1) / kTC;
  const int vts = p.DV / 64;
  const TcWait tw{p.status, p.timeout_ns, &abort_flag_s};

  struct Tile {
    int job, b, h, bh, c, len;
  };
  auto tile_of = [&](int idx) {
    Tile t;
    t.job = idx % p.npass;
    idx /= p.npass;
    t.c = idx % nch;
    t.bh = idx / nch;
    t.b = t.bh / p.NH;
    t.h = t.bh % p.NH;
    t.len = row_len(p, t.b);
    return t;
  };
  auto load_xa = [&](const Tile& t, int buf) {
    const LinAttnPass& ps = p.pass[t.job];
    const uint32_t d = sm + buf * (2 * C::X);
    const __nv_bfloat16* gx = static_cast<const __nv_bfloat16*>(ps.x) + t.b * ps.xs[1] + t.h * ps.xs[2];
    const __nv_bfloat16* ga = static_cast<const __nv_bfloat16*>(ps.a) + t.b * ps.as[1] + t.h * ps.as[2];
    load_rows<DK>(d, gx, ps.xs[0], t.c * kTC, t.len, ps.reverse != 0);
    load_rows<DK>(d + C::X, ga, ps.as[0], t.c * kTC, t.len, ps.reverse != 0);
  };
  auto s_at = [&](int buf) {  // state tile, and c tile behind the first one
    return DK == 256 && buf == 1 ? sm + C::X + 2 * kBlkBytes : sCS + buf * (kBlkBytes + C::S);
  };
  auto c_at = [&](int buf) { return buf == 0 ? sCS + C::S : (DK == 256 ? sCS + C::S + kBlkBytes : sCS + 2 * C::S + kBlkBytes); };
  auto load_cs = [&](const Tile& t, int v, int buf) {
    const LinAttnPass& ps = p.pass[t.job];
    const __nv_bfloat16* gc = static_cast<const __nv_bfloat16*>(ps.c) + t.b * ps.cs[1] + t.h * ps.cs[2];
    const __nv_bfloat16* gs = static_cast<const __nv_bfloat16*>(p.chunk_states) +
                              (((long long)t.job * p.B * p.NH + t.bh) * nch + t.c) * DK * p.DV;
    const uint32_t sS = s_at(buf);
    load_rows<64>(c_at(buf), gc + 64 * v, ps.cs[0], t.c * kTC, t.len, ps.reverse != 0);
#pragma unroll
    for (int i = 0; i < DK * 8 / kTT; ++i) {
      const int e = tid + i * kTT, k = e / 8, ch = e % 8;
      zfill16(sS + (uint32_t)(k * 128 + ((ch ^ (k & 7)) << 4)), gs + (long long)k * p.DV + 64 * v + ch * 8, true);
    }
  };
  // the first tile at or after idx that holds tokens; the others get their zeros here
  auto next_tile = [&](int idx, Tile& t) {
    for (; idx < tiles; idx += gridDim.x) {
      t = tile_of(idx);
      if (t.len > t.c * kTC) break;
      const LinAttnPass& ps = p.pass[t.job];
      const int r = t.c * kTC + row;
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(ps.out) + t.b * ps.os[1] + t.h * ps.os[2] +
                         (long long)r * ps.os[0] + 32 * half;
      if (r < p.T)
        for (int v = 0; v < vts; ++v)
#pragma unroll
          for (int j = 0; j < 32; j += 8)
            *reinterpret_cast<uint4*>(o + 64 * v + j) = make_uint4(0u, 0u, 0u, 0u);
    }
    return idx;
  };

  Tile t, tn;
  int idx = next_tile(blockIdx.x, t);
  if (idx >= tiles) return;
  load_xa(t, 0);
  cp_async_commit();
  if (tid == 0) {
    mbar_init(bar, 1);
    abort_flag_s = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(&tslot_s), C::TMEM);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tslot_s;
  const uint32_t mylanes = (uint32_t)(q * 32) << 16;
  uint32_t phase = 0;
  constexpr int kNext = C::NXA == 2 ? 1 : 0, kPre = C::NCS == 2 ? 1 : 0;  // copy groups behind the one awaited
  bool ok = true;
  for (int k = 0; ok && idx < tiles; ++k) {
    const int buf = C::NXA == 2 ? (k & 1) : 0;
    const uint32_t sX = sm + buf * (2 * C::X), sA = sX + C::X;
    const LinAttnPass& ps = p.pass[t.job];
    const int r0 = t.c * kTC, n = t.len - r0 < kTC ? t.len - r0 : kTC;
    const float lg = p.log_decay[t.h] * 1.4426950408889634f;
    load_cs(t, 0, 0);
    cp_async_commit();
    const int nidx = next_tile(idx + gridDim.x, tn);
    if (C::NXA == 2) {
      if (nidx < tiles) load_xa(tn, buf ^ 1);
      cp_async_commit();
    }
    if (tid < kTC) pows[tid] = ps.intra * pw(lg, tid);
    const float fr = ps.inter * pw(lg, row + 1 - ps.shift);
    cp_async_wait<1 + kNext>();
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    if (tid == 0) {  // scores
      tc_fence_after();
      constexpr uint32_t idesc = idesc_bf16_f32(128, 128, false, false);
#pragma unroll
      for (int ks = 0; ks < DK / 16; ++ks) {
        const uint32_t o = (uint32_t)(ks / 4) * kBlkBytes + (ks % 4) * 32;
        umma_bf16(tmem, sdesc_sw128(sX + o, 16, 1024), sdesc_sw128(sA + o, 16, 1024), idesc, ks != 0);
      }
      umma_commit(bar);
    }
    if (!tc_wait(bar, phase, tw)) break;
    phase ^= 1;
    tc_fence_after();
    // decay and mask; 32-column blocks `half` and `half + 2` of this thread's row
#pragma unroll
    for (int jb = 0; jb < 2; ++jb) {
      const int blk = half + 2 * jb;  // columns 32 blk ..
      uint32_t pk[16];
      if (blk <= q) {
        uint32_t s[32];
        tmem_ld32(tmem + mylanes + 32 * blk, s);
        tmem_wait_ld();
        tmem_reg_fence(s);
        const float* pm = pows + (row - 32 * blk);
        float v[32];
        if (blk < q) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(s[j]) * pm[-j];
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = j <= lane ? __uint_as_float(s[j]) * pm[-min(j, lane)] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) pk[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) pk[j] = 0u;
      }
      // block 0 (columns 0 .. 63) in a's place, block 1 behind it or in the extra space
      const uint32_t d = jb == 0 || C::XTRA == 0 ? sA + blk_at(row, 4 * blk) : sXtra + blk_at(row, 4 * (blk - 2));
#pragma unroll
      for (int i = 0; i < 4; ++i)
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(
                         (d & ~127u) | (((d & 127u) ^ (uint32_t)(i << 4)))),
                     "r"(pk[4 * i]), "r"(pk[4 * i + 1]), "r"(pk[4 * i + 2]), "r"(pk[4 * i + 3])
                     : "memory");
    }
    __nv_bfloat16* orow =
        static_cast<__nv_bfloat16*>(ps.out) + t.b * ps.os[1] + t.h * ps.os[2] +
        (long long)(row < n && ps.reverse ? t.len - 1 - r0 - row : r0 + row) * ps.os[0] + 32 * half;
    // 64 columns at a time: the MMAs of one tile run during the epilogue of the one before
    for (int v = 0; v <= vts; ++v) {
      if (v > 0) {
        if (!tc_wait(bar, phase, tw)) {
          ok = false;
          break;
        }
        phase ^= 1;
        tc_fence_after();
      }
      if (v < vts) {
        if (C::NCS == 2) {
          if (v + 1 < vts) load_cs(t, v + 1, (v + 1) & 1);
          cp_async_commit();
          if (v == 0) cp_async_wait<kNext + kPre>();
          else cp_async_wait<kPre>();
        } else {
          if (v > 0) {
            load_cs(t, v, 0);
            cp_async_commit();
            cp_async_wait<0>();
          } else {
            cp_async_wait<kNext>();
          }
        }
        fence_async_smem();
        tc_fence_before();  // (reads of the sums that these MMAs overwrite)
        __syncthreads();
        if (tid == 0) {
          tc_fence_after();
          constexpr uint32_t idesc = idesc_bf16_f32(128, 64, false, true);
          const uint32_t tO = tmem + 128 + (v % C::NO) * 128, cb = C::NCS == 2 ? (v & 1) : 0;
          const uint32_t sS = s_at(cb), sC = c_at(cb);
#pragma unroll
          for (int ks = 0; ks < DK / 16; ++ks)
            umma_bf16(tO + 64, sdesc_sw128(sX + (uint32_t)(ks / 4) * kBlkBytes + (ks % 4) * 32, 16, 1024),
                      sdesc_sw128(sS + ks * 2048, kBlkBytes, 1024), idesc, ks != 0);
#pragma unroll
          for (int ks = 0; ks < kTC / 16; ++ks)
            umma_bf16(tO, sdesc_sw128((ks < 4 ? sA : (C::XTRA ? sXtra : sA + kBlkBytes)) + (ks % 4) * 32, 16, 1024),
                      sdesc_sw128(sC + ks * 2048, kBlkBytes, 1024), idesc, ks != 0);
          umma_commit(bar);
        }
      } else if (C::NXA == 1) {  // x and a have been multiplied for the last time
        if (nidx < tiles) load_xa(tn, 0);
        cp_async_commit();
      }
      const int e = v - (C::NO == 2 ? 1 : 0);  // columns whose sums are complete
      if (C::NO == 1 && v < vts) {
        if (!tc_wait(bar, phase, tw)) {
          ok = false;
          break;
        }
        tc_fence_after();
      }
      if (e < 0 || e >= vts) continue;
      const uint32_t tO = tmem + 128 + (e % C::NO) * 128 + mylanes + 32 * half;
      uint32_t o[32], s[32];
      tmem_ld32(tO, o);
      tmem_ld32(tO + 64, s);
      tmem_wait_ld();
      tmem_reg_fence(o);
      tmem_reg_fence(s);
      if (r0 + row < p.T) {
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
          uint32_t pk[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int x = j + 2 * i;
            pk[i] = row < n ? pack_bf16x2(fmaf(fr, __uint_as_float(s[x]), __uint_as_float(o[x])),
                                          fmaf(fr, __uint_as_float(s[x + 1]), __uint_as_float(o[x + 1])))
                            : 0u;
          }
          *reinterpret_cast<uint4*>(orow + 64 * e + j) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
      }
    }
    t = tn;
    idx = nidx;
  }
  cp_async_wait<0>();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM);
  }
}

template <int DK>
int launch_dk(const LinAttnParams& p, cudaStream_t s) {
  using C = StCfg<DK>;
  static int prep_main[64][5], prep_state[64][5], prep_out[64][5];
  int e = prepare_launch(prep_main, linattn_states_kernel<DK, false>, C::SMEM, kTT, 1);
  if (e != 0) return e;
  e = prepare_launch(prep_out, linattn_outputs_kernel<DK>, OutCfg<DK>::SMEM, kTT, 1);
  if (e != 0) return e;
  const long long nch = ((long long)p.T + kTC - 1) / kTC;
  const long long base = (long long)p.npass * p.B * p.NH * C::MB * (p.DV / 64);
  const long long outs = (long long)p.npass * p.B * p.NH * nch;
  if (base * p.nseg * (C::TILE / 256) > 0x7fffffffLL || outs > 0x3fffffffLL)
    return (int)cudaErrorInvalidValue;
  if (p.nseg > 1) {
    e = prepare_launch(prep_state, linattn_states_kernel<DK, true>, C::SMEM, kTT, 1);
    if (e != 0) return e;
    linattn_states_kernel<DK, true><<<(unsigned)(base * (p.nseg - 1)), kTT, C::SMEM, s>>>(p);
    linattn_scan_kernel<TcOrder<DK>>
        <<<(unsigned)(base * (C::TILE / 256)), 256, 0, s>>>(p, p.seg_chunks * kTC);
  }
  linattn_states_kernel<DK, false><<<(unsigned)(base * p.nseg), kTT, C::SMEM, s>>>(p);
  if (outs > 0) {
    const long long cap = (long long)sm_count() * OutCfg<DK>::OCC;
    linattn_outputs_kernel<DK>
        <<<(unsigned)(outs < cap ? outs : cap), kTT, OutCfg<DK>::SMEM, s>>>(p, (int)outs);
  }
  return (int)cudaGetLastError();
}

}  // namespace

int launch_linattn_tc(const LinAttnParams& p, cudaStream_t s) {
  if (cudaMemsetAsync(p.status, 0, sizeof(int), s) != cudaSuccess) return (int)cudaErrorUnknown;
  switch (p.DK) {
    case 64: return launch_dk<64>(p, s);
    case 128: return launch_dk<128>(p, s);
    case 256: return launch_dk<256>(p, s);
    default: return (int)cudaErrorInvalidValue;
  }
}

}  // namespace srnn
