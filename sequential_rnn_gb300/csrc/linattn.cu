// Linear attention with a decay for each head, bf16: the chunked form and its
// gradient on the tensor cores.
//
//   S_t = lambda S_{t-1} + k_t v_t^T,   o_t = scale q_t S_t        (S [Dk, Dv], per head)
//
// A chunk of C = 64 tokens starts from S and needs three products:
//   o_i = scale (sum_{j<=i} lambda^(i-j) (q_i.k_j) v_j + lambda^(i+1) q_i S)
//   S  <- lambda^C S + sum_j lambda^(C-1-j) k_j v_j^T
// The gradients are the same operator with its arguments in other places:
//   dq = the operator on (do, v, k) with S^T in the place of S,
//   dk = the operator on (v, do, q) with time reversed and dS^T,
//   dv = the operator on (k, q, do) with time reversed and dS, which also leaves dS_0;
// reversed in time the state enters token r with lambda^r (its own token is not
// behind a decay) instead of lambda^(r+1), and leaves a chunk with one power more.
// One kernel serves all four ("passes", LinAttnPass: x, a, c for q, k, v), and a
// gradient launches its three passes together.
//
// A CTA takes a head of a row (of up to 64 columns of c) and walks its chunks, warps side by side over 16 rows of
// the output and 16 of the state.  Bound by latency: a chunk is a chain of copies, three products that depend on one
// another and a barrier, with 12 warps an SM (168 registers each) to fill it; the tensor cores run at 42% of
// mma.sync's rate, DRAM at 26% of its.  Measured, 12 heads of 64: 1 x 16384 tokens 56.4 us (in 37 segments), 16 x
// 1024 gradient 104.3, five ragged rows of up to 333 13.4.
//
// Rounding: the scores times their decay, and the state as an operand of q S,
// are rounded to bf16, once each (as bf16 results are); every sum is fp32.  The
// state itself stays in fp32 registers, and its update must not lose it to
// operand rounding: c_j times its weight is split into three bf16 terms (24 bits)
// and each chunk's update is summed from zero, then added to the decayed state in
// round-to-nearest (the tensor cores' own accumulation truncates).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "kernels.h"
#include "linattn.cuh"
#include "lm.h"
#include "ptx.cuh"

namespace srnn {
namespace {

constexpr int kC = 64;  // tokens per chunk

template <int DK_, int DVT_>
struct LaCfg {
  static constexpr int DK = DK_, DVT = DVT_;     // DVT: columns of c (and of the state) per CTA
  static constexpr int NW = DK <= 64 ? 4 : 8;    // warps
  static constexpr int NT = NW * 32;
  static constexpr int VG = DVT / 16;            // state rows (v): 16 per warp
  static constexpr int KG = NW / VG;             // state columns (dk) over the other warps
  static constexpr int DKW = DK / KG, NTS = DKW / 8;
  static constexpr int CG = NW / 4;              // output: 16 rows per warp, columns over CG
  static constexpr int OVC = DVT / CG, NTO = OVC / 8;
  static constexpr uint32_t XB = kC * DK * 2, CB = kC * DVT * 2;
  static constexpr uint32_t STAGE = 2 * XB + CB;
  static constexpr uint32_t SB = DVT * DK * 2;   // bf16 copy of the state, [v][dk]
  static constexpr uint32_t SMEM = 2 * STAGE + 2 * SB + 1024;  // (1024: for aligning the tiles)
  static constexpr uint32_t SMEM_STATE = 2 * (XB + CB) + 1024;
  static constexpr int OCC = DK <= 64 ? 3 : (DK == 128 ? 2 : 1);
  static constexpr int GT = NTS < 8 ? NTS : 8;  // state tiles whose update is looked at together
};

// byte offset of 16-byte chunk ch of row r in a swizzled tile of D bf16 columns
template <int D>
__device__ __forceinline__ uint32_t tile_at(int r, int ch) {
  const int x = D >= 64 ? (r & 7) : ((r >> 1) & 3);
  return (uint32_t)(r * (D * 2) + ((ch ^ x) << 4));
}

// A chunk's update of the state in fp32 multiply-adds, where d[m][r] (rows v, v + 8 (r >> 1), columns dk + 8 m + (r & 1)) is
// not finite
template <int DK, int DVT, int GT>
__device__ __forceinline__ void add_tokens(float (&d)[GT][4], uint32_t bA, uint32_t bC, int dk, int v, int n, float lg,
                                           float upd, int shift) {
  uint32_t on = 0u;
#pragma unroll
  for (int m = 0; m < GT; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (!(fabsf(d[m][r]) < INFINITY)) on |= 1u << (4 * m + r), d[m][r] = 0.f;
#pragma unroll 1
  for (int j = 0; j < n; ++j) {
    const float w = upd * pw(lg, n - 1 - j + shift);
    float c[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint16_t x;
      asm volatile("ld.shared.b16 %0, [%1];" : "=h"(x) : "r"(bC + tile_at<DVT>(j, v / 8 + k) + (v & 7) * 2));
      c[k] = bf16_to_f32(x) * w;
    }
#pragma unroll
    for (int m = 0; m < GT; ++m) {
      uint32_t a;
      asm volatile("ld.shared.b32 %0, [%1];" : "=r"(a) : "r"(bA + tile_at<DK>(j, dk / 8 + m) + (dk & 7) * 2));
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (on >> (4 * m + r) & 1u) d[m][r] = fmaf(r & 1 ? bf16_hi(a) : bf16_lo(a), c[r >> 1], d[m][r]);
    }
  }
}

// which state element register `reg` of quad i of thread t holds
template <class C>
__device__ __forceinline__ void state_of(int t, int i, int reg, int& dk, int& v) {
  const int warp = t >> 5, lane = t & 31;
  v = 16 * (warp % C::VG) + (lane >> 2) + 8 * (reg >> 1);
  dk = (warp / C::VG) * C::DKW + 8 * i + 2 * (lane & 3) + (reg & 1);
}
// workspace order of a state tile: quad by quad, the threads' float4 side by side
template <class C>
struct QuadOrder {
  static constexpr int TILE = C::DK * C::DVT;
  static __device__ __forceinline__ int tiles(const LinAttnParams& p) { return p.DV / C::DVT; }
  static __device__ __forceinline__ void at(const LinAttnParams&, int tile, int e, int& dk, int& v) {
    state_of<C>((e / 4) % C::NT, e / (4 * C::NT), e & 3, dk, v);
    v += tile * C::DVT;
  }
};

// STATE_ONLY: the segment's own contribution to the state, from zero, into the workspace.
template <class C, bool STATE_ONLY>
__global__ void __launch_bounds__(C::NT, C::OCC)
    linattn_kernel(const __grid_constant__ LinAttnParams p) {
  constexpr int DK = C::DK, DVT = C::DVT, NT = C::NT, NTS = C::NTS, NTO = C::NTO;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ float pow8[8];  // lambda^(8 m)
  const uint32_t sm = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t stage_bytes = STATE_ONLY ? C::XB + C::CB : C::STAGE;
  const uint32_t sS = sm + 2 * C::STAGE;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g0 = lane >> 2, t0 = 2 * (lane & 3);
  if (STATE_ONLY || p.nseg == 1) depend_wait();  // the call's first kernel
  if (STATE_ONLY) depend_launch();
  const int VT = p.DV / DVT;
  const Where w = where_of(p, VT, STATE_ONLY ? p.nseg - 1 : p.nseg);
  const LinAttnPass& ps = p.pass[w.job];
  const int len = row_len(p, w.b);
  const int nch = (p.T + kC - 1) / kC;
  const int c0 = w.seg * p.seg_chunks;
  const int c1 = c0 + p.seg_chunks < nch ? c0 + p.seg_chunks : nch;
  const int lch = (len + kC - 1) / kC;
  const int cend = c1 < lch ? c1 : lch;  // chunks c0 .. cend - 1 hold tokens
  if (STATE_ONLY && (long long)c1 * kC >= len) return;  // no later segment starts from it
  const float lg = p.log_decay[w.h] * 1.4426950408889634f;
  const bool rev = ps.reverse != 0;
  if (!STATE_ONLY && blockIdx.x == 0 && tid == 0 && p.clear) *p.status = 0;

  const __nv_bfloat16* gx = static_cast<const __nv_bfloat16*>(ps.x) + w.b * ps.xs[1] + w.h * ps.xs[2];
  const __nv_bfloat16* ga = static_cast<const __nv_bfloat16*>(ps.a) + w.b * ps.as[1] + w.h * ps.as[2];
  const __nv_bfloat16* gc =
      static_cast<const __nv_bfloat16*>(ps.c) + w.b * ps.cs[1] + w.h * ps.cs[2] + w.vt * DVT;

  auto load_tile = [&](auto dim, uint32_t dst, const __nv_bfloat16* src, long long stride, int c) {
    constexpr int D = decltype(dim)::value, CH = D / 8;
#pragma unroll
    for (int i = 0; i < kC * CH / NT; ++i) {
      const int e = tid + i * NT, row = e / CH, ch = e % CH, r = c * kC + row;
      const bool ok = r < len;
      const long long t = ok ? (rev ? len - 1 - r : r) : 0;
      cp_async16_zfill(dst + tile_at<D>(row, ch), src + t * stride + ch * 8, ok);
    }
  };
  using DKt = std::integral_constant<int, DK>;
  using DVt = std::integral_constant<int, DVT>;
  auto load_chunk = [&](int c, int st) {
    const uint32_t base = sm + st * stage_bytes;
    load_tile(DKt{}, base, ga, ps.as[0], c);
    load_tile(DVt{}, base + C::XB, gc, ps.cs[0], c);
    if (!STATE_ONLY) load_tile(DKt{}, base + C::XB + C::CB, gx, ps.xs[0], c);
    cp_async_commit();
  };

  if (c0 < cend) load_chunk(c0, 0);

  // ---- the state at the segment's start --------------------------------
  const int vg = warp % C::VG, kg = warp / C::VG;
  float S[NTS][4];
  if (STATE_ONLY) {
#pragma unroll
    for (int i = 0; i < NTS; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) S[i][r] = 0.f;
  } else if (p.nseg > 1 && (w.seg == 0 || c0 < cend)) {
    depend_wait();  // for the scan
    const float4* src = reinterpret_cast<const float4*>(seg_state(p, w, w.seg, VT, DK * DVT));
#pragma unroll
    for (int i = 0; i < NTS; ++i) {
      const float4 f = src[i * NT + tid];
      S[i][0] = f.x, S[i][1] = f.y, S[i][2] = f.z, S[i][3] = f.w;
    }
  } else if (p.nseg == 1) {
    const float* in = ps.init ? ps.init + (long long)w.bh * DK * p.DV : nullptr;
#pragma unroll
    for (int i = 0; i < NTS; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        int dk, v;
        state_of<C>(tid, i, r, dk, v);
        v += w.vt * DVT;
        S[i][r] = in ? in[ps.init_t ? (long long)v * DK + dk : (long long)dk * p.DV + v] : 0.f;
      }
  } else {  // a segment past the row's last token
#pragma unroll
    for (int i = 0; i < NTS; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) S[i][r] = 0.f;
  }
  // bf16 copy of the state into buffer `buf`, [v][dk]
  auto publish = [&](int buf) {
    const uint32_t d = sS + buf * C::SB + tile_at<DK>(16 * vg + g0, (kg * C::DKW) / 8) + t0 * 2;
#pragma unroll
    for (int i = 0; i < NTS; ++i) {
      const uint32_t at = d ^ (uint32_t)(i << 4);
#pragma unroll
      for (int hh = 0; hh < 2; ++hh)
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + 8 * hh * (DK * 2)),
                     "r"(pack_bf16x2(S[i][2 * hh], S[i][2 * hh + 1]))
                     : "memory");
    }
  };
  if (!STATE_ONLY) {
    publish(0);
    if (tid < 8) pow8[tid] = pw(lg, 8 * tid);
  }

  // decay factors of the scores: power i - j inside an 8 x 8 tile (d0, diagonal
  // tiles), and 8 and 16 rows further down
  float ge[2], fe[2][2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int d0 = g0 - t0 - e;
    ge[e] = ps.intra * pw(lg, d0 < 0 ? 0 : d0);
    fe[0][e] = ps.intra * pw(lg, d0 + 8);
    fe[1][e] = ps.intra * pw(lg, d0 + 16);
  }
  // weight of token j in the state's update, and of the state itself, for a chunk of n tokens
  float wj[4][4];
  float wS = 0.f;
  int wn = -1;

  const int rb = warp & 3, cg = warp >> 2;  // output rows 16 rb .., columns OVC cg ..
  const int mg = lane >> 3, l7 = lane & 7;
  // Where a thread's fragments begin in each tile.  A swizzled tile's 16-byte chunk numbers enter an address by
  // exclusive or, and its rows 8 apart swizzle alike: chunk 2 ks + m is (base ^ ks << 5), a row 8 i on is
  // + 8 i row bytes, an immediate (computed place by place, addresses were a third of the instructions).
  constexpr int RX = DK * 2, RC = DVT * 2;  // row bytes
  const uint32_t oX = tile_at<DK>(16 * rb + (lane & 15), lane >> 4);            // x, rows as A operand
  const uint32_t oA = tile_at<DK>(8 * (mg >> 1) + l7, mg & 1);                  // a, rows as B operand
  const uint32_t oS = tile_at<DK>(cg * C::OVC + 8 * (mg >> 1) + l7, mg & 1);    // state
  const uint32_t oCp = tile_at<DVT>(8 * (mg & 1) + l7, (cg * C::OVC) / 8 + (mg >> 1));   // c, columns as B operand
  const uint32_t oCu = tile_at<DVT>(8 * (mg >> 1) + l7, 2 * vg + (mg & 1));              // c, columns as A operand
  const uint32_t oAu = tile_at<DK>(8 * (mg & 1) + l7, (kg * C::DKW) / 8 + (mg >> 1));    // a, columns as B operand
  for (int c = c0; c < cend; ++c) {
    const int st = (c - c0) & 1;
    const uint32_t bA = sm + st * stage_bytes, bC = bA + C::XB, bX = bC + C::CB;
    cp_async_wait<0>();
    __syncthreads();
    if (c + 1 < cend) load_chunk(c + 1, st ^ 1);
    const int n = len - c * kC < kC ? len - c * kC : kC;

    if (!STATE_ONLY && 16 * rb < n) {
      // ---- scores x a^T (16 x 64, tiles up to the diagonal) and x S ------
      float P[8][4], O[NTO][4];
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) P[i][r] = 0.f;
#pragma unroll
      for (int i = 0; i < NTO; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) O[i][r] = 0.f;
      const uint32_t bS = sS + st * C::SB;
#pragma unroll 4
      for (int ks = 0; ks < DK / 16; ++ks) {
        uint32_t qa[4];
        ldmatrix_x4(qa, (bX + oX) ^ (uint32_t)(ks << 5));
        const uint32_t sk = (bS + oS) ^ (uint32_t)(ks << 5), ak = (bA + oA) ^ (uint32_t)(ks << 5);
#pragma unroll
        for (int i = 0; i < NTO; i += 2) {
          uint32_t sb[4];
          ldmatrix_x4(sb, sk + 8 * i * RX);
          mma_bf16_16816(O[i], qa, sb[0], sb[1]);
          mma_bf16_16816(O[i + 1], qa, sb[2], sb[3]);
        }
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          if (i <= 2 * rb) {
            uint32_t kb[4];
            ldmatrix_x4(kb, ak + 8 * i * RX);
            mma_bf16_16816(P[i], qa, kb[0], kb[1]);
            mma_bf16_16816(P[i + 1], qa, kb[2], kb[3]);
          }
        }
      }
      const int i0 = 16 * rb + g0;
      const float r0 = ps.inter * pw(lg, i0 + 1 - ps.shift), r1 = ps.inter * pw(lg, i0 + 9 - ps.shift);
#pragma unroll
      for (int i = 0; i < NTO; ++i) {
        O[i][0] *= r0;
        O[i][1] *= r0;
        O[i][2] *= r1;
        O[i][3] *= r1;
      }
      // ---- decay and mask, then times c ----------------------------------
      uint32_t pd[4];  // of the tiles on the diagonal, which come last
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        if (ks > rb) continue;
        if (ks == rb) {  // (2 ks: d0 and d0 + 8), (2 ks + 1: d0 - 8 and d0)
          float d[2][2], f[2], m[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const bool low = g0 >= t0 + e;
            d[0][e] = low ? P[2 * ks][e] * ge[e] : 0.f;
            f[e] = P[2 * ks][2 + e] * fe[0][e];
            m[e] = low ? P[2 * ks + 1][2 + e] * ge[e] : 0.f;
          }
          pd[0] = pack_bf16x2(d[0][0], d[0][1]);
          pd[1] = pack_bf16x2(f[0], f[1]);
          pd[2] = 0u;
          pd[3] = pack_bf16x2(m[0], m[1]);
        } else {
          uint32_t pa[4];
          const float m0 = pow8[2 * (rb - ks) - 1], m1 = pow8[2 * (rb - ks) - 2];
          pa[0] = pack_bf16x2(P[2 * ks][0] * (m0 * fe[0][0]), P[2 * ks][1] * (m0 * fe[0][1]));
          pa[1] = pack_bf16x2(P[2 * ks][2] * (m0 * fe[1][0]), P[2 * ks][3] * (m0 * fe[1][1]));
          pa[2] = pack_bf16x2(P[2 * ks + 1][0] * (m1 * fe[0][0]), P[2 * ks + 1][1] * (m1 * fe[0][1]));
          pa[3] = pack_bf16x2(P[2 * ks + 1][2] * (m1 * fe[1][0]), P[2 * ks + 1][3] * (m1 * fe[1][1]));
#pragma unroll
          for (int i = 0; i < NTO; i += 2) {
            uint32_t vb[4];
            ldmatrix_x4_trans(vb, ((bC + oCp) ^ (uint32_t)(i << 4)) + 16 * ks * RC);
            mma_bf16_16816(O[i], pa, vb[0], vb[1]);
            mma_bf16_16816(O[i + 1], pa, vb[2], vb[3]);
          }
        }
      }
      // On the diagonal zero scores stand for later tokens, and zero times a c that is not finite is NaN: those 16
      // rows of c are looked at first, and where one is found the tokens are taken one by one.
      uint32_t vd[NTO / 2][4], seen = 0u;
#pragma unroll
      for (int i = 0; i < NTO; i += 2) {
        ldmatrix_x4_trans(vd[i / 2], ((bC + oCp) ^ (uint32_t)(i << 4)) + 16 * rb * RC);
#pragma unroll
        for (int r = 0; r < 4; ++r) seen = seen_finite(seen, vd[i / 2][r]);
      }
      if (!__any_sync(0xffffffffu, seen != 0u)) {
#pragma unroll
        for (int i = 0; i < NTO; i += 2) {
          mma_bf16_16816(O[i], pd, vd[i / 2][0], vd[i / 2][1]);
          mma_bf16_16816(O[i + 1], pd, vd[i / 2][2], vd[i / 2][3]);
        }
      } else {
#pragma unroll 1
        for (int j = 0; j < 16; ++j) {
          const int from = (lane & 28) | ((j & 7) >> 1);  // its scores' lane; this thread's rows are g0 and g0 + 8
          const uint32_t s0 = __shfl_sync(0xffffffffu, j < 8 ? pd[0] : pd[2], from);
          const uint32_t s1 = __shfl_sync(0xffffffffu, j < 8 ? pd[1] : pd[3], from);
          const float p0 = j & 1 ? bf16_hi(s0) : bf16_lo(s0), p1 = j & 1 ? bf16_hi(s1) : bf16_lo(s1);
#pragma unroll
          for (int i = 0; i < NTO; ++i) {
            uint32_t cj;
            asm volatile("ld.shared.b32 %0, [%1];"
                         : "=r"(cj)
                         : "r"(bC + tile_at<DVT>(16 * rb + j, (cg * C::OVC) / 8 + i) + t0 * 2));
            if (j <= g0) {
              O[i][0] = fmaf(p0, bf16_lo(cj), O[i][0]);
              O[i][1] = fmaf(p0, bf16_hi(cj), O[i][1]);
            }
            if (j <= g0 + 8) {
              O[i][2] = fmaf(p1, bf16_lo(cj), O[i][2]);
              O[i][3] = fmaf(p1, bf16_hi(cj), O[i][3]);
            }
          }
        }
      }
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int r = c * kC + i0 + 8 * hh;
        if (r >= len) continue;
        const long long t = rev ? len - 1 - r : r;
        __nv_bfloat16* go = static_cast<__nv_bfloat16*>(ps.out) + t * ps.os[0] + w.b * ps.os[1] +
                            w.h * ps.os[2] + w.vt * DVT + cg * C::OVC + t0;
#pragma unroll
        for (int i = 0; i < NTO; ++i)
          *reinterpret_cast<uint32_t*>(go + 8 * i) = pack_bf16x2(O[i][2 * hh], O[i][2 * hh + 1]);
      }
    }

    // ---- state: S^T <- lambda^n S^T + (weighted c)^T a ---------------------
    if (wn != n) {
      wn = n;
      wS = pw(lg, n);
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = 16 * ks + t0 + (e & 1) + 8 * (e >> 1);
          wj[ks][e] = j < n ? ps.upd * pw(lg, n - 1 - j + ps.shift) : 0.f;
        }
    }
    uint32_t ah[4][4], am[4][4], al[4][4];
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      uint32_t vt[4];
      ldmatrix_x4_trans(vt, bC + oCu + 16 * ks * RC);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float x0 = bf16_lo(vt[r]) * wj[ks][2 * (r >> 1)];
        float x1 = bf16_hi(vt[r]) * wj[ks][2 * (r >> 1) + 1];
        ah[ks][r] = pack_bf16x2(x0, x1);
        x0 -= bf16_lo(ah[ks][r]);
        x1 -= bf16_hi(ah[ks][r]);
        am[ks][r] = pack_bf16x2(x0, x1);
        x0 -= bf16_lo(am[ks][r]);
        x1 -= bf16_hi(am[ks][r]);
        al[ks][r] = pack_bf16x2(x0, x1);
      }
    }
    constexpr int GT = C::GT;
#pragma unroll
    for (int i0 = 0; i0 < NTS; i0 += GT) {
      float d[GT][4], top = 0.f;
#pragma unroll
      for (int i = 0; i < GT; ++i) d[i][0] = d[i][1] = d[i][2] = d[i][3] = 0.f;
#pragma unroll
      for (int i = 0; i < GT; i += 2) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          uint32_t kb[4];
          ldmatrix_x4_trans(kb, ((bA + oAu) ^ (uint32_t)((i0 + i) << 4)) + 16 * ks * RX);
          mma_bf16_16816(d[i], al[ks], kb[0], kb[1]);
          mma_bf16_16816(d[i + 1], al[ks], kb[2], kb[3]);
          mma_bf16_16816(d[i], am[ks], kb[0], kb[1]);
          mma_bf16_16816(d[i + 1], am[ks], kb[2], kb[3]);
          mma_bf16_16816(d[i], ah[ks], kb[0], kb[1]);
          mma_bf16_16816(d[i + 1], ah[ks], kb[2], kb[3]);
        }
      }
      // an infinite c or a: its terms' rests are NaN, or zeros that meet it; token by token it stays what it is
#pragma unroll
      for (int i = 0; i < GT; ++i) top = max_abs3(max_abs3(top, d[i][0], d[i][1]), d[i][2], d[i][3]);
      if (__any_sync(0xffffffffu, !(top < INFINITY)))
        add_tokens<DK, DVT>(d, bA, bC, kg * C::DKW + 8 * i0 + t0, 16 * vg + g0, n, lg, ps.upd, ps.shift);
#pragma unroll
      for (int i = 0; i < GT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[i0 + i][r] = fmaf(wS, S[i0 + i][r], d[i][r]);
    }
    if (!STATE_ONLY && c + 1 < cend) publish(st ^ 1);
  }

  if (STATE_ONLY) {
    float4* dst = reinterpret_cast<float4*>(seg_state(p, w, w.seg + 1, VT, DK * DVT));
#pragma unroll
    for (int i = 0; i < NTS; ++i) dst[i * NT + tid] = make_float4(S[i][0], S[i][1], S[i][2], S[i][3]);
    return;
  }
  if (ps.fin != nullptr &&
      ((len > c0 * kC && (long long)len <= (long long)c1 * kC) || (len == 0 && w.seg == 0))) {
    float* f = ps.fin + (long long)w.bh * DK * p.DV;
#pragma unroll
    for (int i = 0; i < NTS; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        int dk, v;
        state_of<C>(tid, i, r, dk, v);
        f[(long long)dk * p.DV + w.vt * DVT + v] = S[i][r];
      }
  }
  // (not before: the next kernel's CTAs would take the places that this one's leave free, three on some SMs, and keep
  // them: 8 x 2048 gradients one after the other 133 us each instead of 100)
  depend_launch();
  // tokens that do not count: zeros
  const int rlo = len > c0 * kC ? len : c0 * kC, rhi = c1 * kC < p.T ? c1 * kC : p.T;
  constexpr int CH = DVT / 8;
  for (long long e = tid; e < (long long)(rhi - rlo) * CH; e += NT) {
    const long long t = rlo + e / CH;
    __nv_bfloat16* go = static_cast<__nv_bfloat16*>(ps.out) + t * ps.os[0] + w.b * ps.os[1] +
                        w.h * ps.os[2] + w.vt * DVT + (e % CH) * 8;
    *reinterpret_cast<uint4*>(go) = make_uint4(0u, 0u, 0u, 0u);
  }
}

template <int DK, int DVT>
int launch_cfg(const LinAttnParams& p, cudaStream_t s) {
  using C = LaCfg<DK, DVT>;
  static int prep_main[64][5], prep_state[64][5];
  int e = prepare_launch(prep_main, linattn_kernel<C, false>, C::SMEM, C::NT, 1);
  if (e != 0) return e;
  const long long base = (long long)p.npass * p.B * p.NH * (p.DV / DVT);
  if (base * p.nseg * (DK * DVT / 256) > 0x7fffffffLL) return (int)cudaErrorInvalidValue;
  if (p.nseg > 1) {
    e = prepare_launch(prep_state, linattn_kernel<C, true>, C::SMEM_STATE, C::NT, 1);
    if (e != 0) return e;
    e = launch_dependent(linattn_kernel<C, true>, (unsigned)(base * (p.nseg - 1)), C::NT, C::SMEM_STATE, s, p);
    if (e != 0) return e;
    e = launch_dependent(linattn_scan_kernel<QuadOrder<C>>, (unsigned)(base * (DK * DVT / 256)), 256, 0, s, p,
                         p.seg_chunks * kC);
    if (e != 0) return e;
  }
  return launch_dependent(linattn_kernel<C, false>, (unsigned)(base * p.nseg), C::NT, C::SMEM, s, p);
}

template <int DK>
int launch_dk(const LinAttnParams& p, cudaStream_t s) {
  // 32 columns of c a CTA also where twice the CTAs still have an SM each: a chunk's chain is shorter (5 ragged rows of
  // up to 333, 12 x 64: 18.4 -> 14.3 us); forward with 64 x 64, up to three an SM (16 rows of 200 16.3 -> 14.5, of 512
  // 28.8 -> 25.4; a gradient's passes lose by it, 8 rows of 200 19.7 / 23.2, as do 64 x 128, 12.8 / 14.0)
  const long long ctas = (long long)p.npass * p.B * p.NH * (p.DV / 32);
  const bool narrow = p.nseg == 1 && ctas <= (DK == 64 && p.DV == 64 && p.npass == 1 ? 3 : 1) * sm_count();
  return p.DV % 64 == 0 && !narrow ? launch_cfg<DK, 64>(p, s) : launch_cfg<DK, 32>(p, s);
}

}  // namespace

int launch_linattn_mma(const LinAttnParams& p, cudaStream_t s) {
  switch (p.DK) {
    case 32: return launch_dk<32>(p, s);
    case 64: return launch_dk<64>(p, s);
    case 128: return launch_dk<128>(p, s);
    case 256: return launch_dk<256>(p, s);
    default: return (int)cudaErrorInvalidValue;
  }
}

}  // namespace srnn
