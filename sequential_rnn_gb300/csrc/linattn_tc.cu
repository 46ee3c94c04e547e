// Linear attention with a decay for each head, bf16, head sizes that are a
// multiple of 64: the chunked passes of linattn.cu on the 5th-generation tensor
// cores (tcgen05, accumulators in TMEM), chunks of 128 tokens, in two kernels.
//
//   states   S <- lambda^n S + a^T (weighted c), chunk by chunk; leaves the state at
//            every chunk's start (bf16, an operand of the next kernel) and the final one
//   outputs  out = mask(x a^T) c + decay (x S), all chunks at once
//
// Split in two, only the cheap part (one product of the three) is sequential, and the
// outputs are independent tiles for a persistent grid; the chunk states cost 2 Dk Dv
// bytes per 128 tokens and head, written and read once, mostly inside L2.
//
// The states' CTA holds 128 (or 64) x 64 of S in fp32 registers.  c times its weight is split into
// three bf16 terms (by truncation: exact, all 24 bits), so that the state does not lose to operand rounding what fp32
// keeps; a chunk's products with the three accumulate from zero in TMEM, and their
// sum, smallest first, joins the decayed state in round-to-nearest.
//
// Both kernels have one control warp (one lane: TMA loads, MMA issue, buffer bookkeeping)
// and 8 or 16 compute warps (terms of c, decay and mask of the scores, state and
// output epilogues); mbarriers order them.  Tiles are rows of 64 values (128 bytes, 128-byte
// swizzle): the same tile is a K-major operand (scores) and an MN-major one (state
// update, P c, x S).  Loading through the copy engine matters: with cp.async from all threads
// the copies of a tile took longer to issue (2,000-2,600 cycles) than its MMAs to run.
//
// A pass with reversed time loads the same ascending token rows (a box that begins before
// token 0 reads zeros there): row i of a chunk is then its token 127 - i, and the mask
// and the powers of the decay run the other way.
#include <cuda.h>
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

constexpr int kTC = 128;                  // tokens per chunk
constexpr uint32_t kBlkBytes = kTC * 128; // 128 rows x 64 columns
constexpr int kAhead = 4;                 // chunks fetched into L2 ahead of their use (states)

// tensor maps: x, a, c, out of each pass [T, B, NH, D]; chunk states as rows of DV
struct TcMaps {
  CUtensorMap x[kLinAttnPasses], a[kLinAttnPasses], c[kLinAttnPasses], out[kLinAttnPasses];
  CUtensorMap s_load, s_store;
  // 0 where the operand is shared by all heads / rows (its map has one)
  int xh[kLinAttnPasses], xb[kLinAttnPasses], ah[kLinAttnPasses], ab[kLinAttnPasses];
  int ch[kLinAttnPasses], cb[kLinAttnPasses];
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int c0, int c1,
                                            int c2, int c3, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}
// the same box into L2 only
__device__ __forceinline__ void tma_prefetch_4d(const CUtensorMap* map, int c0, int c1, int c2, int c3) {
  asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(c2), "r"(c3)
               : "memory");
}
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                             uint32_t src) {
  asm volatile(
      "cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(src)
      : "memory");
}
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void sts128(uint32_t at, const uint32_t* v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3])
               : "memory");
}
// offset of 16-byte chunk ch of row r in a 64-column block
__device__ __forceinline__ uint32_t blk_at(int r, int ch) {
  return (uint32_t)(r * 128 + ((ch ^ (r & 7)) << 4));
}
template <int N>
__device__ __forceinline__ void reg_fence(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// A wait is bounded in time: one that runs out sets the status word and the CTA's
// abort flag, on which every other wait gives up.
struct TcWait {
  int* status;
  unsigned long long limit_ns;
  volatile int* abort_flag;
  __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
      if (mbar_try_wait(bar, parity)) return true;
      if (*abort_flag) return false;
      if (globaltimer_ns() - t0 > limit_ns) {
        *abort_flag = 1;
        atomicOr(status, kStatusTimeout);
        return false;
      }
    }
  }
};
// after an abort: a copy that was issued on `bar` lands before the CTA leaves
__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer_ns() - t0 > 10000000ull) break;
}
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// ---------------------------------------------------------------- states --
template <int DK_>
struct StCfg {
  static constexpr int DK = DK_;
  static constexpr int DKB = DK < 128 ? DK : 128;    // state rows (dk) per CTA
  static constexpr int MB = DK / DKB;
  static constexpr int NCW = DKB == 128 ? 16 : 8;    // compute warps
  static constexpr int THREADS = 32 * (NCW + 1);
  static constexpr int OCC = DKB == 128 ? 1 : 2;
  static constexpr int NC = 64 / (NCW / 4);          // state columns of a thread
  static constexpr uint32_t A = (DKB / 64) * kBlkBytes;
  // sets of c's three terms (and buffers of c).  With two, a chunk's terms are made while the one
  // before is multiplied; with 64 state rows one set, so that two CTAs fit on an SM.
  static constexpr int NT = DKB == 128 ? 2 : 1;
  static constexpr uint32_t sA = 0, sC = 2 * A, sT = sC + NT * kBlkBytes;
  // (with 64 state rows the MMA's other 64 rows read the tile behind a, and are not used)
  static constexpr uint32_t sS = sT + NT * 3 * kBlkBytes;  // states on their way: 32 rows x NC per warp
  static constexpr uint32_t STG = 32 * NC * 2;
  static constexpr uint32_t SMEM = sS + DKB * 128 + 1024;
  // the sums of the three terms, side by side (one MMA of N = 192 reads a once for all three:
  // with three of N = 64 a chunk's MMAs took 2,000 cycles, bound by a's shared-memory reads)
  static constexpr int ND = DKB == 128 ? 2 : 1;            // TMEM buffers
  static constexpr uint32_t TMEM = ND == 2 ? 512 : 256;
  static constexpr int TILE = DKB * 64;
};

// workspace order of a state tile: quad by quad, the owning threads' float4 side by side
template <int DK>
struct TcOrder {
  using C = StCfg<DK>;
  static constexpr int TILE = C::TILE;
  static constexpr int OWN = C::DKB * (64 / C::NC);
  static __device__ __forceinline__ int tiles(const LinAttnParams& p) { return C::MB * (p.DV / 64); }
  static __device__ __forceinline__ void at(const LinAttnParams& p, int tile, int e, int& dk, int& v) {
    const int vts = p.DV / 64, th = (e / 4) % OWN;
    dk = (tile / vts) * C::DKB + th % C::DKB;
    v = (tile % vts) * 64 + C::NC * (th / C::DKB) + 4 * (e / (4 * OWN)) + (e & 3);
  }
};

// STATE_ONLY: a segment's own contribution to the state, from zero, into the workspace.
template <int DK, bool STATE_ONLY>
__global__ void __launch_bounds__(StCfg<DK>::THREADS, StCfg<DK>::OCC)
    linattn_states_kernel(const __grid_constant__ LinAttnParams p, const __grid_constant__ TcMaps m) {
  using C = StCfg<DK>;
  constexpr int DKB = C::DKB, NC = C::NC, NCW = C::NCW, OWN = TcOrder<DK>::OWN;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ int abort_flag_s;
  __shared__ uint32_t tslot_s;
  __shared__ __align__(8) uint64_t bars_s[10];
  const uint32_t sm = (smem_u32(smem_raw) + 1023u) & ~1023u;
  // copies of a, of c; terms ready; MMAs done; sums read
  const uint32_t bar = smem_u32(bars_s);
  const uint32_t aF = bar, cF = bar + 16, tR = bar + 32, mD = bar + 48, sR = bar + 64;
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
  const int cnt = cend > c0 ? cend - c0 : 0;
  const bool rev = ps.reverse != 0;
  const TcWait wait{p.status, p.timeout_ns, &abort_flag_s};

  if (tid == 0) {
    for (int i = 0; i < 4; ++i) mbar_init(bar + 8 * i, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(tR + 8 * i, NCW);
      mbar_init(mD + 8 * i, 1);
      mbar_init(sR + 8 * i, NCW);
    }
    abort_flag_s = 0;
    fence_mbar_init();
    fence_async_smem();
  }
  if (warp == NCW) {
    tmem_alloc(smem_u32(&tslot_s), C::TMEM);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tslot_s;

  if (warp == NCW) {
    // ---------------------------------------------------------- control --
    if (lane == 0 && cnt > 0) {
      const int hA = w.h * m.ah[w.job], bA = w.b * m.ab[w.job];
      const int hC = w.h * m.ch[w.job], bC = w.b * m.cb[w.job];
      auto token = [&](int it) { return rev ? len - (c0 + it + 1) * kTC : (c0 + it) * kTC; };
      int na = 0, nc = 0;  // copies issued
      auto load_a = [&](int it) {
        if (it >= cnt) return;
        const uint32_t d = sm + C::sA + (it & 1) * C::A, f = aF + 8 * (it & 1);
        mbar_arrive_expect_tx(f, C::A);
#pragma unroll
        for (int k = 0; k < DKB / 64; ++k)
          tma_load_4d(d + k * kBlkBytes, &m.a[w.job], mb * DKB + 64 * k, hA, bA, token(it), f);
        ++na;
      };
      auto load_c = [&](int it) {
        if (it >= cnt) return;
        const uint32_t f = cF + 8 * (it % C::NT);
        mbar_arrive_expect_tx(f, kBlkBytes);
        tma_load_4d(sm + C::sC + (it % C::NT) * kBlkBytes, &m.c[w.job], vt * 64, hC, bC, token(it), f);
        ++nc;
      };
      // shared memory holds little more than a chunk ahead: the ones after it are fetched into L2
      // (a by the CTA of the first columns, c by the one of the first state rows)
      auto prefetch = [&](int it) {
        if (it >= cnt || token(it) < 0) return;
        if (vt == 0)
#pragma unroll
          for (int k = 0; k < DKB / 64; ++k)
            tma_prefetch_4d(&m.a[w.job], mb * DKB + 64 * k, hA, bA, token(it));
        if (mb == 0) tma_prefetch_4d(&m.c[w.job], vt * 64, hC, bC, token(it));
      };
      load_c(0);
      load_a(0);
      if (C::NT == 2) load_c(1);
      load_a(1);
      for (int k = 2; k < kAhead; ++k) prefetch(k);
      constexpr uint32_t idesc = idesc_bf16_f32(128, 192, true, true);
      int it = 0;
      for (; it < cnt; ++it) {
        const int d = it % C::ND;
        if (!wait(tR + 8 * (it & 1), (it >> 1) & 1)) break;
        load_c(it + C::NT);  // its buffer's terms have been made
        if (!wait(aF + 8 * (it & 1), (it >> 1) & 1)) break;
        if (it >= C::ND && !wait(sR + 8 * d, ((it - C::ND) / C::ND) & 1)) break;
        tc_fence_after();
        const uint32_t a = sm + C::sA + (it & 1) * C::A, t = sm + C::sT + (it % C::NT) * (3 * kBlkBytes);
#pragma unroll
        for (int ks = 0; ks < kTC / 16; ++ks)
          umma_bf16(tmem + d * 192, sdesc_sw128(a + ks * 2048, kBlkBytes, 1024),
                    sdesc_sw128(t + ks * 2048, kBlkBytes, 1024), idesc, ks != 0 ? 1u : 0u);
        umma_commit(mD + 8 * (it & 1));
        prefetch(it + kAhead);
        if (it >= 1) {  // the next a goes where the previous chunk's MMAs have read
          if (!wait(mD + 8 * ((it - 1) & 1), ((it - 1) >> 1) & 1)) break;
          load_a(it + 1);
        }
      }
      if (it < cnt) {
        for (int k = na - 2 < 0 ? 0 : na - 2; k < na; ++k) drain(aF + 8 * (k & 1), (k >> 1) & 1);
        for (int k = nc - C::NT < 0 ? 0 : nc - C::NT; k < nc; ++k)
          drain(cF + 8 * (k % C::NT), (k / C::NT) & 1);
      }
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------- compute --
    const float lg = p.log_decay[w.h] * 1.4426950408889634f;
    const int q = warp & 3, g = warp >> 2;
    const bool owner = 32 * q < DKB;  // of row dk = 32 q + lane, columns NC g ..
    const int dk = 32 * q + lane, th = g * DKB + dk;
    const int gk = mb * DKB + dk, gv = vt * 64 + NC * g;
    float S[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) S[j] = 0.f;
    if (!STATE_ONLY && owner) {
      if (p.nseg > 1) {
        const float4* src = reinterpret_cast<const float4*>(seg_state(p, w, w.seg, C::MB * vts, C::TILE));
#pragma unroll
        for (int i = 0; i < NC / 4; ++i) {
          const float4 f = src[i * OWN + th];
          S[4 * i] = f.x, S[4 * i + 1] = f.y, S[4 * i + 2] = f.z, S[4 * i + 3] = f.w;
        }
      } else if (ps.init != nullptr) {
        const float* in = ps.init + (long long)w.bh * DK * p.DV;
        if (ps.init_t) {
#pragma unroll
          for (int j = 0; j < NC; ++j) S[j] = in[(long long)(gv + j) * DK + gk];
        } else {
#pragma unroll
          for (int j = 0; j < NC; j += 4) {
            const float4 f = *reinterpret_cast<const float4*>(in + (long long)gk * p.DV + gv + j);
            S[j] = f.x, S[j + 1] = f.y, S[j + 2] = f.z, S[j + 3] = f.w;
          }
        }
      }
    }
    // the state at the start of chunk `it` on its way to the chunk states
    auto publish = [&](int it) {
      if (STATE_ONLY || !owner) return;
      const uint32_t stg = sm + C::sS + (g * (DKB / 32) + q) * C::STG;
      if (lane == 0) bulk_wait_read_all();
      __syncwarp();
#pragma unroll
      for (int j = 0; j < NC / 8; ++j) {
        uint32_t pk[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) pk[k] = pack_bf16x2(S[8 * j + 2 * k], S[8 * j + 2 * k + 1]);
        // 32 rows of 64 (32) bytes, 64- (32-) byte swizzle
        sts128(stg + lane * (NC * 2) + ((j ^ (NC == 32 ? (lane >> 1) & 3 : (lane >> 2) & 1)) << 4), pk);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_2d(&m.s_store, gv, ((w.job * p.B * p.NH + w.bh) * nch + c0 + it) * DK + mb * DKB + 32 * q, stg);
        bulk_commit();
      }
    };
    // c of chunk `it`, weighted, in three bf16 terms: rows tid / 8 + .., 16-byte chunk tid % 8
    constexpr int ROWS = 1024 / (32 * NCW), STEP = 4 * NCW;
    float wj[ROWS];
    int wn = -1;
    auto make_terms = [&](int it) {
      const int c = c0 + it, n = len - c * kTC < kTC ? len - c * kTC : kTC;
      if (wn != n) {
        wn = n;
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
          const int row = tid / 8 + STEP * i, j = rev ? kTC - 1 - row : row;
          wj[i] = j < n ? ps.upd * pw(lg, n - 1 - j + ps.shift) : 0.f;
        }
      }
      if (!wait(cF + 8 * (it % C::NT), (it / C::NT) & 1)) return false;
      const uint32_t src = sm + C::sC + (it % C::NT) * kBlkBytes;
      const uint32_t set = sm + C::sT + (it % C::NT) * (3 * kBlkBytes);
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        const int row = tid / 8 + STEP * i;
        const uint32_t at = blk_at(row, tid % 8);
        uint32_t in[4], t[3][4];
        lds128(in, src + at);
        if ((rev ? kTC - 1 - row : row) >= n) in[0] = in[1] = in[2] = in[3] = 0u;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float x0 = bf16_lo(in[k]) * wj[i], x1 = bf16_hi(in[k]) * wj[i];
#pragma unroll
          for (int e = 0; e < 3; ++e) {  // the leading 8 bits of the significand, three times
            t[e][k] = __byte_perm(__float_as_uint(x0), __float_as_uint(x1), 0x7632);
            x0 -= __uint_as_float(__float_as_uint(x0) & 0xffff0000u);
            x1 -= __uint_as_float(__float_as_uint(x1) & 0xffff0000u);
          }
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) sts128(set + k * kBlkBytes + at, t[k]);
      }
      if (!rev && n < kTC && len < p.T) {
        // a's rows behind the row's last token hold values that do not count: zeros
        if (!wait(aF + 8 * (it & 1), (it >> 1) & 1)) return false;
        const uint32_t z[4] = {0u, 0u, 0u, 0u};
        for (int e = tid; e < kTC * (DKB / 8); e += 32 * NCW) {
          const int row = e / (DKB / 8), ch = e % (DKB / 8);
          if (row >= n) sts128(sm + C::sA + (it & 1) * C::A + (ch / 8) * kBlkBytes + blk_at(row, ch % 8), z);
        }
      }
      fence_async_smem();
      warp_arrive(tR + 8 * (it & 1));
      return true;
    };
    bool ok = cnt == 0 || make_terms(0);
    if (cnt > 0) publish(0);
    for (int it = 0; ok && it < cnt; ++it) {
      if (C::NT == 2 && it + 1 < cnt && !make_terms(it + 1)) break;
      if (!wait(mD + 8 * (it & 1), (it >> 1) & 1)) break;
      tc_fence_after();
      const int c = c0 + it, n = len - c * kTC < kTC ? len - c * kTC : kTC;
      if (owner) {
        const float wS = pw(lg, n);
        const uint32_t t = tmem + ((uint32_t)(q * 32) << 16) + (it % C::ND) * 192 + NC * g;
#pragma unroll
        for (int h = 0; h < NC; h += 16) {
          uint32_t r0[16], r1[16], r2[16];
          tmem_ld16(t + 128 + h, r2);
          tmem_ld16(t + 64 + h, r1);
          tmem_ld16(t + h, r0);
          tmem_wait_ld();
          reg_fence(r0);
          reg_fence(r1);
          reg_fence(r2);
#pragma unroll
          for (int j = 0; j < 16; ++j)  // smallest first
            S[h + j] = fmaf(wS, S[h + j],
                            (__uint_as_float(r2[j]) + __uint_as_float(r1[j])) + __uint_as_float(r0[j]));
        }
      }
      tc_fence_before();
      warp_arrive(sR + 8 * (it % C::ND));
      if (it + 1 < cnt) {
        if (C::NT == 1 && !make_terms(it + 1)) break;
        publish(it + 1);
      }
    }
    if (!STATE_ONLY && lane == 0) bulk_wait_all();
    __syncwarp();
    if (owner) {
      if (STATE_ONLY) {
        float4* dst = reinterpret_cast<float4*>(seg_state(p, w, w.seg + 1, C::MB * vts, C::TILE));
#pragma unroll
        for (int i = 0; i < NC / 4; ++i)
          dst[i * OWN + th] = make_float4(S[4 * i], S[4 * i + 1], S[4 * i + 2], S[4 * i + 3]);
      } else if (ps.fin != nullptr && ((len > c0 * kTC && (long long)len <= (long long)c1 * kTC) ||
                                       (len == 0 && w.seg == 0))) {
        float* f = ps.fin + ((long long)w.bh * DK + gk) * p.DV + gv;
#pragma unroll
        for (int j = 0; j < NC; j += 4)
          *reinterpret_cast<float4*>(f + j) = make_float4(S[j], S[j + 1], S[j + 2], S[j + 3]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == NCW) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM);
  }
}

// --------------------------------------------------------------- outputs --
template <int DK>
struct OutCfg {
  static constexpr int NCW = DK == 64 ? 8 : 16;        // compute warps
  static constexpr int THREADS = 32 * (NCW + 1);
  static constexpr int OCC = DK == 64 ? 2 : 1;
  static constexpr int NG = NCW / 4, NC = 64 / NG;     // a thread: one row, NC of 64 output columns
  static constexpr uint32_t X = (DK / 64) * kBlkBytes;
  // x and a of one tile.  Scores in bf16 (32 KB) take the place of a once it has been multiplied
  // (with 64 columns of a, its 16 KB and 16 KB more).
  static constexpr int NXA = DK <= 128 ? 2 : 1;        // tiles of x and a
  static constexpr uint32_t XTRA = X < 2 * kBlkBytes ? kBlkBytes : 0;
  static constexpr uint32_t S = DK * 128;              // DK rows x 64 columns of the state
  static constexpr int NCS = DK >= 128 ? 2 : 1;        // c and state tiles of 64 columns
  // with 256 columns the second state tile lies in a's upper half, free after the scores
  static constexpr uint32_t sXtra = NXA * 2 * X, sCS = sXtra + XTRA;
  static constexpr uint32_t CS = DK == 256 ? 2 * kBlkBytes + S : NCS * (kBlkBytes + S);
  // outputs on their way: 32 rows x NC columns per warp; with 64 columns in x's place
  static constexpr uint32_t sO = sCS + CS;
  static constexpr uint32_t STG = 32 * NC * 2;
  static constexpr uint32_t SMEM = sO + (DK == 64 ? 0 : NCW * STG) + 1024;
  static constexpr int NO = OCC == 1 ? 2 : 1;          // sums (P c and x S) in TMEM
  static constexpr uint32_t TMEM = OCC == 1 ? 512 : 256;
  static __device__ __forceinline__ uint32_t s_at(int buf) {
    return DK == 256 && buf == 1 ? X + 2 * kBlkBytes : sCS + buf * (kBlkBytes + S);
  }
  static __device__ __forceinline__ uint32_t c_at(int buf) {
    return buf == 0 ? sCS + S : (DK == 256 ? sCS + S + kBlkBytes : sCS + 2 * S + kBlkBytes);
  }
};

// A persistent CTA walks (row, head, chunk, pass) tiles, the passes of a chunk side by
// side on the grid, since they read the same tokens.
template <int DK>
__global__ void __launch_bounds__(OutCfg<DK>::THREADS, OutCfg<DK>::OCC)
    linattn_outputs_kernel(const __grid_constant__ LinAttnParams p, const __grid_constant__ TcMaps m,
                           int tiles) {
  using C = OutCfg<DK>;
  constexpr int NCW = C::NCW, NG = C::NG, NC = C::NC;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ int abort_flag_s;
  __shared__ uint32_t tslot_s;
  __shared__ __align__(8) uint64_t bars_s[14];
  const uint32_t sm = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t bar = smem_u32(bars_s);
  // x and a loaded; c and state loaded; scores done; scores written (and read from TMEM);
  // sums done; sums read; staging in x read; c's rows behind the last token zeroed
  const uint32_t xF = bar, cF = bar + 16, sc = bar + 32, pW = bar + 40, oD = bar + 48, oR = bar + 64,
                 xR = bar + 80, cZ = bar + 88;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nch = (p.T + kTC - 1) / kTC;
  const int vts = p.DV / 64;
  const TcWait wait{p.status, p.timeout_ns, &abort_flag_s};

  // tiles in the order pass, chunk, head, row (fastest first); a step of the grid is added digit by
  // digit (the divisions of a place cost 700 cycles a tile)
  struct Tile {
    int job, c, h, b, len;
  };
  auto digits = [&](int idx) {
    Tile t;
    t.job = idx % p.npass;
    idx /= p.npass;
    t.c = idx % nch;
    idx /= nch;
    t.h = idx % p.NH;
    t.b = idx / p.NH;
    return t;
  };
  const Tile stride = digits((int)gridDim.x);
  auto advance = [&](Tile& t) {  // (past the last tile b is past the last row: not to be read)
    t.job += stride.job;
    t.c += stride.c;
    t.h += stride.h;
    t.b += stride.b;
    if (t.job >= p.npass) t.job -= p.npass, ++t.c;
    if (t.c >= nch) t.c -= nch, ++t.h;
    if (t.h >= p.NH) t.h -= p.NH, ++t.b;
  };
  // first token of a tile's rows; whether rows of c have to be zeroed
  auto token_of = [&](const Tile& t) { return p.pass[t.job].reverse ? t.len - (t.c + 1) * kTC : t.c * kTC; };
  auto ragged = [&](const Tile& t) {
    return !p.pass[t.job].reverse && t.len < p.T && t.len < (t.c + 1) * kTC;
  };

  if (tid == 0) {
    for (int i = 0; i < 5; ++i) mbar_init(bar + 8 * i, 1);
    mbar_init(pW, NCW);
    for (int i = 0; i < 2; ++i) {
      mbar_init(oD + 8 * i, 1);
      mbar_init(oR + 8 * i, NCW);
    }
    mbar_init(xR, NCW);
    mbar_init(cZ, NCW);
    abort_flag_s = 0;
    fence_mbar_init();
    fence_async_smem();
  }
  if (warp == NCW) {
    tmem_alloc(smem_u32(&tslot_s), C::TMEM);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tslot_s;

  if (warp == NCW) {
    // ---------------------------------------------------------- control --
    if (lane == 0) {
      Tile at = digits(blockIdx.x);
      int at_idx = blockIdx.x;
      auto next_tile = [&](Tile& t) {  // the next one that holds tokens
        for (; at_idx < tiles; at_idx += gridDim.x, advance(at)) {
          t = at;
          t.len = row_len(p, t.b);
          if (t.len > t.c * kTC) break;
        }
        const int idx = at_idx;
        at_idx += gridDim.x;
        advance(at);
        return idx < tiles ? idx : tiles;
      };
      uint32_t nx[2] = {0, 0}, ncs[2] = {0, 0};  // copies issued per buffer
      uint32_t ux[2] = {0, 0}, ucs[2] = {0, 0};  // and waited for
      auto load_xa = [&](const Tile& t, int buf) {
        const uint32_t d = sm + buf * (2 * C::X), f = xF + 8 * buf;
        const int j = t.job, tok = token_of(t);
        mbar_arrive_expect_tx(f, 2 * C::X);
#pragma unroll
        for (int k = 0; k < DK / 64; ++k) {
          tma_load_4d(d + k * kBlkBytes, &m.x[j], 64 * k, t.h * m.xh[j], t.b * m.xb[j], tok, f);
          tma_load_4d(d + C::X + k * kBlkBytes, &m.a[j], 64 * k, t.h * m.ah[j], t.b * m.ab[j], tok, f);
        }
        ++nx[buf];
      };
      auto prefetch_xa = [&](const Tile& t) {
        const int j = t.job, tok = token_of(t);
        if (tok < 0) return;
        for (int k = 0; k < DK / 64; ++k) {
          tma_prefetch_4d(&m.x[j], 64 * k, t.h * m.xh[j], t.b * m.xb[j], tok);
          tma_prefetch_4d(&m.a[j], 64 * k, t.h * m.ah[j], t.b * m.ab[j], tok);
        }
      };
      auto load_cs = [&](const Tile& t, int v, int buf) {
        const uint32_t f = cF + 8 * buf;
        const int j = t.job;
        mbar_arrive_expect_tx(f, kBlkBytes + C::S);
        tma_load_4d(sm + C::c_at(buf), &m.c[j], 64 * v, t.h * m.ch[j], t.b * m.cb[j], token_of(t), f);
        tma_load_2d(sm + C::s_at(buf), &m.s_load, 64 * v, (((j * p.B + t.b) * p.NH + t.h) * nch + t.c) * DK, f);
        ++ncs[buf];
      };
      auto scores = [&](int buf) {
        constexpr uint32_t idesc = idesc_bf16_f32(128, 128, false, false);
        const uint32_t x = sm + buf * (2 * C::X), a = x + C::X;
#pragma unroll
        for (int ks = 0; ks < DK / 16; ++ks) {
          const uint32_t o = (uint32_t)(ks / 4) * kBlkBytes + (ks % 4) * 32;
          umma_bf16(tmem, sdesc_sw128(x + o, 16, 1024), sdesc_sw128(a + o, 16, 1024), idesc, ks != 0);
        }
        umma_commit(sc);
      };
      uint32_t used[2] = {0, 0}, ret[2] = {0, 0};  // sums per TMEM set: issued, waited for
      uint32_t nz = 0;                             // c tiles with rows zeroed
      Tile t, tn, tnn;
      int idx = next_tile(t), nidx = tiles;
      bool ok = true;
      if (idx < tiles) {
        load_xa(t, 0);
        load_cs(t, 0, 0);
        nidx = next_tile(tn);
        if (C::NXA == 2 && nidx < tiles) load_xa(tn, 1);
        ok = wait(xF, 0);
        if (ok) {
          ++ux[0];
          tc_fence_after();
          scores(0);
        }
      }
      for (int k = 0; ok && idx < tiles; ++k) {
        const int buf = C::NXA == 2 ? (k & 1) : 0;
        const uint32_t x = sm + buf * (2 * C::X), a = x + C::X;
        const bool zeroed = ragged(t);
        for (int v = 0; ok && v < vts; ++v) {
          const int cb = C::NCS == 2 ? (v & 1) : 0, o = C::NO == 2 ? (v & 1) : 0;
          if (C::NCS == 2 && v + 1 < vts) {
            // its buffers: read by the MMAs of v - 1; with 256 columns a's upper half (scores done)
            if (v > 0) {
              if (!(ok = wait(oD + 8 * (o ^ 1), ret[o ^ 1] & 1))) break;
              ++ret[o ^ 1];
            } else if (DK == 256) {
              if (!(ok = wait(sc, k & 1))) break;
            }
            load_cs(t, v + 1, cb ^ 1);
          }
          if (!(ok = wait(cF + 8 * cb, ucs[cb] & 1))) break;
          ++ucs[cb];
          if (used[o] > 0 && !(ok = wait(oR + 8 * o, (used[o] - 1) & 1))) break;
          tc_fence_after();
          constexpr uint32_t idesc = idesc_bf16_f32(128, 64, false, true);
          const uint32_t tO = tmem + 128 + o * 128, s = sm + C::s_at(cb), cc = sm + C::c_at(cb);
#pragma unroll
          for (int ks = 0; ks < DK / 16; ++ks)
            umma_bf16(tO + 64, sdesc_sw128(x + (uint32_t)(ks / 4) * kBlkBytes + (ks % 4) * 32, 16, 1024),
                      sdesc_sw128(s + ks * 2048, kBlkBytes, 1024), idesc, ks != 0);
          if (v == 0 && !(ok = wait(pW, k & 1))) break;
          if (zeroed && !(ok = wait(cZ, nz++ & 1))) break;
          tc_fence_after();
#pragma unroll
          for (int ks = 0; ks < kTC / 16; ++ks)
            umma_bf16(tO,
                      sdesc_sw128((ks < 4 ? a : (C::XTRA ? sm + C::sXtra : a + kBlkBytes)) + (ks % 4) * 32, 16, 1024),
                      sdesc_sw128(cc + ks * 2048, kBlkBytes, 1024), idesc, ks != 0);
          umma_commit(oD + 8 * o);
          ++used[o];
          if (C::NCS == 1 && v + 1 < vts) {  // the one buffer, once these MMAs have read it
            if (!(ok = wait(oD, ret[0] & 1))) break;
            ++ret[0];
            load_cs(t, v + 1, 0);
          }
        }
        if (!ok) break;
        if (C::NXA == 2 && nidx < tiles) {  // the next scores, behind these MMAs
          const int nb = buf ^ 1;
          if (!(ok = wait(xF + 8 * nb, ux[nb] & 1))) break;
          ++ux[nb];
          tc_fence_after();
          scores(nb);
        }
        // every buffer of this tile has been read
        for (int o = 0; ok && o < C::NO; ++o)
          while (ok && ret[o] < used[o]) {
            ok = wait(oD + 8 * o, ret[o] & 1);
            ++ret[o];
          }
        if (!ok) break;
        if (nidx < tiles) {
          load_cs(tn, 0, 0);
          const int nn = next_tile(tnn);
          if (C::NXA == 1 && nn < tiles) prefetch_xa(tnn);
          if (C::NXA == 2) {
            if (DK == 64 && !(ok = wait(xR, k & 1))) break;  // outputs in x's place have left
            if (nn < tiles) load_xa(tnn, buf);
          } else {
            load_xa(tn, 0);
            if (!(ok = wait(xF, ux[0] & 1))) break;
            ++ux[0];
            tc_fence_after();
            scores(0);
          }
          t = tn;
          tn = tnn;
          idx = nidx;
          nidx = nn;
        } else {
          idx = tiles;
        }
      }
      if (!ok)
        for (int i = 0; i < 2; ++i) {
          if (nx[i]) drain(xF + 8 * i, (nx[i] - 1) & 1);
          if (ncs[i]) drain(cF + 8 * i, (ncs[i] - 1) & 1);
        }
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------- compute --
    const int q = warp & 3, g = warp >> 2, row = 32 * q + lane;
    const uint32_t lanes = (uint32_t)(q * 32) << 16;
    uint32_t used[2] = {0, 0};
    bool ok = true;
    int k = 0;
    Tile tn = digits(blockIdx.x);
    tn.len = row_len(p, tn.b);
    float dn = p.log_decay[tn.h];
    for (int idx = blockIdx.x; ok && idx < tiles; idx += gridDim.x) {
      const Tile t = tn;
      const float lg = dn * 1.4426950408889634f;
      if (idx + (int)gridDim.x < tiles) {  // its loads are on their way meanwhile
        advance(tn);
        tn.len = row_len(p, tn.b);
        dn = p.log_decay[tn.h];
      }
      const LinAttnPass& ps = p.pass[t.job];
      const int r0 = t.c * kTC, n = t.len - r0 < kTC ? t.len - r0 : kTC;
      const bool rev = ps.reverse != 0;
      __nv_bfloat16* go = static_cast<__nv_bfloat16*>(ps.out) + t.b * ps.os[1] + t.h * ps.os[2] + NC * g;
      // tokens of this chunk that do not count (reversed, the chunk's own rows are others)
      if (row >= n && r0 + row < p.T && (rev || n <= 0)) {
        const uint4 z = make_uint4(0u, 0u, 0u, 0u);
        for (int v = 0; v < vts; ++v)
#pragma unroll
          for (int j = 0; j < NC; j += 8)
            *reinterpret_cast<uint4*>(go + (long long)(r0 + row) * ps.os[0] + 64 * v + j) = z;
      }
      if (n <= 0) continue;
      const int buf = C::NXA == 2 ? (k & 1) : 0;
      const uint32_t sX = sm + buf * (2 * C::X), sP = sX + C::X;
      const float lam = pw(lg, 1);
      const float fr = ps.inter * pw(lg, (rev ? kTC - 1 - row : row) + 1 - ps.shift);
      if (!wait(sc, k & 1)) break;
      tc_fence_after();
      // decay and mask of this thread's row of scores, 32 columns at a time
      for (int blk = g; blk < 4; blk += NG) {
        // columns 0 .. 63 in a's place, the others behind them or in the extra space
        const uint32_t dst = blk < 2 ? sP : (C::XTRA ? sm + C::sXtra : sP + kBlkBytes);
        const int ch = 4 * (blk & 1);
        uint32_t pk[16];
        if (rev ? blk >= q : blk <= q) {
          uint32_t s[32];
          tmem_ld32(tmem + lanes + 32 * blk, s);
          // powers from the column nearest to the diagonal on, each lambda times the one before
          float f = blk == q ? ps.intra : ps.intra * pw(lg, rev ? 32 * blk - row : row - 32 * blk - 31);
          tmem_wait_ld();
          tmem_reg_fence(s);
          const int live = blk == q ? lane : (rev ? 0 : 31);  // last (reversed: first) column that counts
          if (rev) {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const bool on = j >= live;
              s[j] = on ? __float_as_uint(__uint_as_float(s[j]) * f) : 0u;
              f = on ? f * lam : f;
            }
          } else {
#pragma unroll
            for (int j = 31; j >= 0; --j) {
              const bool on = j <= live;
              s[j] = on ? __float_as_uint(__uint_as_float(s[j]) * f) : 0u;
              f = on ? f * lam : f;
            }
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) pk[j] = pack_bf16x2(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1]));
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) pk[j] = 0u;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) sts128(dst + blk_at(row, ch + i), pk + 4 * i);
      }
      fence_async_smem();
      tc_fence_before();
      if (DK == 64 && k > 0) {  // the tile before has left x's place
        if (lane == 0) bulk_wait_read_all();
        warp_arrive(xR);
      }
      warp_arrive(pW);
      const int tok = token_of(t) + 32 * q;  // of this warp's first row
      const bool zero_c = ragged(t);
      for (int v = 0; v < vts; ++v) {
        const int cb = C::NCS == 2 ? (v & 1) : 0, o = C::NO == 2 ? (v & 1) : 0;
        if (zero_c) {
          // the buffer's uses so far: all tiles before this one, and this one's
          const uint32_t uses = C::NCS == 2 ? (uint32_t)k * ((vts + 1 - cb) / 2) + v / 2 : (uint32_t)k * vts + v;
          if (!(ok = wait(cF + 8 * cb, uses & 1))) break;
          const uint32_t z[4] = {0u, 0u, 0u, 0u};
          for (int e = tid; e < kTC * 8; e += 32 * NCW)
            if (e / 8 >= n) sts128(sm + C::c_at(cb) + blk_at(e / 8, e % 8), z);
          fence_async_smem();
          warp_arrive(cZ);
        }
        if (!(ok = wait(oD + 8 * o, used[o] & 1))) break;
        ++used[o];
        tc_fence_after();
        uint32_t pk[NC / 2];
        const bool counts = rev ? row >= kTC - n : row < n;
#pragma unroll
        for (int h = 0; h < NC; h += 16) {
          uint32_t u[16], s[16];
          const uint32_t tO = tmem + 128 + o * 128 + lanes + NC * g + h;
          tmem_ld16(tO, u);
          tmem_ld16(tO + 64, s);
          tmem_wait_ld();
          reg_fence(u);
          reg_fence(s);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            pk[h / 2 + j] =
                counts ? pack_bf16x2(fmaf(fr, __uint_as_float(s[2 * j]), __uint_as_float(u[2 * j])),
                                     fmaf(fr, __uint_as_float(s[2 * j + 1]), __uint_as_float(u[2 * j + 1])))
                       : 0u;
        }
        tc_fence_before();
        warp_arrive(oR + 8 * o);
        // with 64 columns x's place is free behind the last columns' MMAs only
        if (tok >= 0 && (DK != 64 || v == vts - 1)) {
          const uint32_t stg = (DK == 64 ? sX : sm + C::sO) + warp * C::STG;
          if (lane == 0) bulk_wait_read_all();
          __syncwarp();
          // 32 rows of 64 (32) bytes, 64- (32-) byte swizzle
#pragma unroll
          for (int j = 0; j < NC / 8; ++j)
            sts128(stg + lane * (NC * 2) + ((j ^ (NC == 32 ? (lane >> 1) & 3 : (lane >> 2) & 1)) << 4), pk + 4 * j);
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_4d(&m.out[t.job], 64 * v + NC * g, t.h, t.b, tok, stg);
            bulk_commit();
          }
        } else if (tok + lane >= 0 && tok + lane < p.T) {
#pragma unroll
          for (int j = 0; j < NC; j += 8)
            *reinterpret_cast<uint4*>(go + (long long)(tok + lane) * ps.os[0] + 64 * v + j) =
                make_uint4(pk[j / 2], pk[j / 2 + 1], pk[j / 2 + 2], pk[j / 2 + 3]);
        }
      }
      if (!ok) break;
      ++k;
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == NCW) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM);
  }
}

}  // namespace

// ------------------------------------------------------------- host side --
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn();  // tc_gemm.cu

namespace {

bool encode(CUtensorMap* map, const void* ptr, int rank, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swizzle) {
  EncodeTiledFn fn = encode_fn();
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  return fn != nullptr &&
         fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(ptr), dims, strides,
            box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [T, B, NH, D] with strides s (token, row, head; elements): box of 64 (cols) x rows tokens.
// An operand shared by all heads or rows (stride 0) has one in its map; *uh, *ub
// then are 0, the factor of the head's and row's coordinate.
bool encode_operand(CUtensorMap* map, const void* ptr, const long long (&s)[3], const LinAttnParams& p,
                    int D, uint32_t cols, uint32_t rows, CUtensorMapSwizzle swizzle, int* uh, int* ub) {
  const int nh = s[2] == 0 ? 1 : p.NH, nb = s[1] == 0 ? 1 : p.B;
  if (uh) *uh = s[2] != 0, *ub = s[1] != 0;
  if (s[0] == 0 && p.T > 1) return false;
  auto bytes = [&](long long e) { return (cuuint64_t)(e == 0 ? D * 2 : e * 2); };
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)nh, (cuuint64_t)nb, (cuuint64_t)p.T};
  const cuuint64_t strides[3] = {bytes(s[2]), bytes(s[1]), bytes(s[0])};
  const cuuint32_t box[4] = {cols, 1, 1, rows};
  return encode(map, ptr, 4, dims, strides, box, swizzle);
}

template <int DK>
int launch_dk(const LinAttnParams& p, cudaStream_t s) {
  using C = StCfg<DK>;
  using O = OutCfg<DK>;
  static int prep_main[64][5], prep_state[64][5], prep_out[64][5];
  int e = prepare_launch(prep_main, linattn_states_kernel<DK, false>, C::SMEM, C::THREADS, 1);
  if (e != 0) return e;
  e = prepare_launch(prep_out, linattn_outputs_kernel<DK>, O::SMEM, O::THREADS, 1);
  if (e != 0) return e;
  const long long nch = ((long long)p.T + kTC - 1) / kTC;
  const long long base = (long long)p.npass * p.B * p.NH * C::MB * (p.DV / 64);
  const long long outs = (long long)p.npass * p.B * p.NH * nch;
  if (base * p.nseg * (C::TILE / 256) > 0x7fffffffLL || outs * DK > 0x3fffffffLL) return kLinAttnTooWide;
  TcMaps m;
  bool ok = true;
  for (int j = 0; j < p.npass; ++j) {
    const LinAttnPass& ps = p.pass[j];
    const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
    ok = ok && encode_operand(&m.x[j], ps.x, ps.xs, p, DK, 64, kTC, sw, &m.xh[j], &m.xb[j]);
    ok = ok && encode_operand(&m.a[j], ps.a, ps.as, p, DK, 64, kTC, sw, &m.ah[j], &m.ab[j]);
    ok = ok && encode_operand(&m.c[j], ps.c, ps.cs, p, p.DV, 64, kTC, sw, &m.ch[j], &m.cb[j]);
    ok = ok && encode_operand(&m.out[j], ps.out, ps.os, p, p.DV, O::NC, 32,
                              O::NC == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B, nullptr,
                              nullptr);
  }
  const cuuint64_t dims[2] = {(cuuint64_t)p.DV, (cuuint64_t)(outs * DK)};
  const cuuint64_t strides[1] = {(cuuint64_t)p.DV * 2};
  const cuuint32_t in[2] = {64, (cuuint32_t)DK}, out[2] = {(cuuint32_t)C::NC, 32};
  ok = ok && encode(&m.s_load, p.chunk_states, 2, dims, strides, in, CU_TENSOR_MAP_SWIZZLE_128B);
  ok = ok && encode(&m.s_store, p.chunk_states, 2, dims, strides, out,
                    C::NC == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B);
  if (!ok) return kLinAttnTooWide;
  if (cudaMemsetAsync(p.status, 0, sizeof(int), s) != cudaSuccess) return (int)cudaErrorUnknown;
  if (p.nseg > 1) {
    e = prepare_launch(prep_state, linattn_states_kernel<DK, true>, C::SMEM, C::THREADS, 1);
    if (e != 0) return e;
    linattn_states_kernel<DK, true><<<(unsigned)(base * (p.nseg - 1)), C::THREADS, C::SMEM, s>>>(p, m);
    linattn_scan_kernel<TcOrder<DK>>
        <<<(unsigned)(base * (C::TILE / 256)), 256, 0, s>>>(p, p.seg_chunks * kTC);
  }
  linattn_states_kernel<DK, false><<<(unsigned)(base * p.nseg), C::THREADS, C::SMEM, s>>>(p, m);
  const long long cap = (long long)sm_count() * O::OCC;
  linattn_outputs_kernel<DK>
      <<<(unsigned)(outs < cap ? outs : cap), O::THREADS, O::SMEM, s>>>(p, m, (int)outs);
  return (int)cudaGetLastError();
}

}  // namespace

int launch_linattn_tc(const LinAttnParams& p, cudaStream_t s) {
  switch (p.DK) {
    case 64: return launch_dk<64>(p, s);
    case 128: return launch_dk<128>(p, s);
    case 256: return launch_dk<256>(p, s);
    default: return (int)cudaErrorInvalidValue;
  }
}

}  // namespace srnn
