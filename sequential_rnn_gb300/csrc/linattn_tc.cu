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
// In both kernels one warp loads (TMA, one lane), one (outputs: three) issues the MMAs (one lane), and
// the others compute (terms of c, decay and mask of the scores, state and output
// epilogues); mbarriers order them.  Tiles are rows of 64 values (128 bytes, 128-byte
// swizzle): the same tile is a K-major operand (scores) and an MN-major one (state
// update, P c, x S).  Loading through the copy engine matters: with cp.async from all threads
// the copies of a tile took longer to issue (2,000-2,600 cycles) than its MMAs to run.
//
// Measured: 4 x 256, 4 rows of 4096 87 us (states 52, outputs 42 alone); gradient 6 x 128, 4 rows of 2001 54.7
// us (30 and 32).  The states are bound by what a chunk makes the compute warps do one after the other (terms of c, 3 x 128
// columns of sums out of TMEM, the state's stores: issue slots 55%, load and store unit 63%), the outputs by
// the copies (320 KB a tile with 256 columns, half of it from DRAM: inputs, outputs and chunk states are 200 MB
// beside 129 of L2) and the chain from a tile's scores to its stores.
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

// tensor maps: x, a, c, out of each pass [T, B, NH, D]; chunk states as rows of DV
struct TcMaps {
  CUtensorMap x[kLinAttnPasses], a[kLinAttnPasses], c[kLinAttnPasses], out[kLinAttnPasses];
  CUtensorMap s_load;
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
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                             uint32_t src) {
  asm volatile(
      "cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(src)
      : "memory");
}
// 32 bytes to global memory (v8: at a 32-byte boundary, one access)
__device__ __forceinline__ void store32(void* at, const uint32_t* v, bool v8) {
  if (v8)
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(at), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  else
#pragma unroll
    for (int i = 0; i < 8; i += 4)
      reinterpret_cast<uint4*>(at)[i / 4] = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
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
      if (*abort_flag) return false;
      if (mbar_try_wait(bar, parity)) return true;
      if (globaltimer_ns() - t0 > limit_ns) {
        *abort_flag = 1;
        atomicOr(status, kStatusTimeout);
        return false;
      }
    }
  }
};
// After an abort, whoever gave up: what was issued on `bar` (a copy, the MMAs before a commit) ends before the CTA leaves.
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
// Warps: 16 (with 64 state rows 8) that make the terms of c and hold the state, one that
// loads a, one that issues the MMAs.
template <int DK_>
struct StCfg {
  static constexpr int DK = DK_;
  static constexpr int DKB = DK < 128 ? DK : 128;    // state rows (dk) per CTA
  static constexpr int MB = DK / DKB;
  static constexpr bool WIDE = DKB == 128;
  static constexpr int NCW = WIDE ? 16 : 8;
  static constexpr int WLOAD = NCW, WMMA = NCW + 1;
  static constexpr int NC = 64 / (NCW / 4);          // state columns of a thread
  static constexpr int THREADS = 32 * (WMMA + 1);
  static constexpr int OCC = WIDE ? 1 : 2;
  static constexpr uint32_t A = (DKB / 64) * kBlkBytes;
  static constexpr int NA = 3;                       // buffers of a
  // sets of c's three terms.  With two, a chunk's terms are made while the one before is
  // multiplied; with 64 state rows one set, so that two CTAs fit on an SM.
  static constexpr int NT = WIDE ? 2 : 1;
  static constexpr uint32_t sT = NA * A;
  // (with 64 state rows the MMA's other 64 rows read the tile behind a, and are not used)
  static constexpr uint32_t SMEM = sT + NT * 3 * kBlkBytes + 1024;
  // the sums of the three terms, side by side (one MMA of N = 192 reads a once for all three:
  // with three of N = 64 a chunk's MMAs took 2,000 cycles, bound by a's shared-memory reads)
  static constexpr int ND = WIDE ? 2 : 1;            // TMEM buffers
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
  constexpr int DKB = C::DKB, NC = C::NC, NCW = C::NCW, OWN = TcOrder<DK>::OWN, NA = C::NA;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ int abort_flag_s, issued_s;
  __shared__ uint32_t tslot_s;
  __shared__ __align__(8) uint64_t bars_s[13];
  const uint32_t sm = (smem_u32(smem_raw) + 1023u) & ~1023u;
  // copies of a landed; a multiplied; terms ready; MMAs done; sums read; the last MMAs of all done
  const uint32_t bar = smem_u32(bars_s);
  const uint32_t aF = bar, aE = bar + 24, tR = bar + 48, mD = bar + 64, sR = bar + 80, xD = bar + 96;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int vts = p.DV / 64;
  if (STATE_ONLY || p.nseg == 1) {  // the call's first kernel
    depend_wait();
    // (a wait that runs out is told two seconds after its CTA began at the earliest, and this one is the first)
    if (p.clear && blockIdx.x == 0 && tid == 0) *p.status = 0;
  }
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
  // first token of chunk `it`'s rows (reversed: possibly below 0)
  auto token = [&](int it) { return rev ? len - (c0 + it + 1) * kTC : (c0 + it) * kTC; };

  if (tid == 0) {
    for (int i = 0; i < 6; ++i) mbar_init(bar + 8 * i, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(tR + 8 * i, NCW);
      mbar_init(mD + 8 * i, 1);
      mbar_init(sR + 8 * i, NCW);
    }
    mbar_init(xD, 1);
    abort_flag_s = 0;
    issued_s = 0;
    fence_mbar_init();
    fence_async_smem();
  }
  if (warp == C::WMMA) {
    tmem_alloc(smem_u32(&tslot_s), C::TMEM);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tslot_s;
  depend_launch();  // (with its TMEM in hand: the next kernel's CTAs ask for theirs)

  if (warp == C::WLOAD) {
    // ------------------------------------------------------------- loads --
    if (lane == 0) {
      const int hA = w.h * m.ah[w.job], bA = w.b * m.ab[w.job];
      int it = 0;
      for (; it < cnt; ++it) {
        const int s = it % NA;
        if (it >= NA && !wait(aE + 8 * s, ((it - NA) / NA) & 1)) break;
        const uint32_t d = sm + s * C::A, f = aF + 8 * s;
        mbar_arrive_expect_tx(f, C::A);
#pragma unroll
        for (int k = 0; k < DKB / 64; ++k)
          tma_load_4d(d + k * kBlkBytes, &m.a[w.job], mb * DKB + 64 * k, hA, bA, token(it), f);
      }
      issued_s = it;
    }
    __syncwarp();
  } else if (warp == C::WMMA) {
    // -------------------------------------------------------------- MMAs --
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(128, 192, true, true);
      for (int it = 0; it < cnt; ++it) {
        const int s = it % NA, d = it % C::ND, ts = it % C::NT;
        if (!wait(aF + 8 * s, (it / NA) & 1)) break;
        if (!wait(tR + 8 * ts, (it / C::NT) & 1)) break;
        if (it >= C::ND && !wait(sR + 8 * d, ((it - C::ND) / C::ND) & 1)) break;
        tc_fence_after();
        const uint32_t a = sm + s * C::A, t = sm + C::sT + ts * (3 * kBlkBytes);
#pragma unroll
        for (int ks = 0; ks < kTC / 16; ++ks)
          umma_bf16(tmem + d * 192, sdesc_sw128(a + ks * 2048, kBlkBytes, 1024),
                    sdesc_sw128(t + ks * 2048, kBlkBytes, 1024), idesc, ks != 0 ? 1u : 0u);
        umma_commit(aE + 8 * s);
        umma_commit(mD + 8 * (it & 1));
      }
      umma_commit(xD);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------- compute --
    const float lg = p.log_decay[w.h] * 1.4426950408889634f;
    // c comes straight from global memory, two chunks ahead in registers (with 64 state rows, where the state takes more
    // of them, one): rows tid / 8 + .., 16-byte chunk tid % 8
    const __nv_bfloat16* gc = static_cast<const __nv_bfloat16*>(ps.c) + w.b * ps.cs[1] + w.h * ps.cs[2] +
                              vt * 64 + (tid % 8) * 8;
    constexpr int ROWS = 1024 / (32 * NCW), STEP = 4 * NCW;
    uint4 cr[ROWS], cn[ROWS];
    auto fetch = [&](int it, uint4 (&d)[ROWS]) {
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        const int t = token(it) + tid / 8 + STEP * i;
        d[i] = it < cnt && t >= 0 && t < len ? *reinterpret_cast<const uint4*>(gc + (long long)t * ps.cs[0])
                                             : make_uint4(0u, 0u, 0u, 0u);
      }
    };
    fetch(0, cr);
    if (C::WIDE) fetch(1, cn);

    const int q = warp & 3, g = warp >> 2;   // rows dk = 32 q + lane, columns NC g ..
    const bool owner = 32 * q < DKB;
    const int dk = 32 * q + lane, th = g * DKB + dk;
    const int gk = mb * DKB + dk, gv = vt * 64 + NC * g;
    float S[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) S[j] = 0.f;
    if (!STATE_ONLY && owner) {
      if (p.nseg > 1) {
        depend_wait();  // for the scan
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
    float wj[ROWS];
    int wn = -1;
    // c of chunk `it` (in cr), weighted, in three bf16 terms
    auto make_terms = [&](int it) {
      const int n = len - (c0 + it) * kTC < kTC ? len - (c0 + it) * kTC : kTC;
      if (wn != n) {
        wn = n;
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
          const int row = tid / 8 + STEP * i, j = rev ? kTC - 1 - row : row;
          wj[i] = j < n ? ps.upd * pw(lg, n - 1 - j + ps.shift) : 0.f;
        }
      }
      const uint32_t set = sm + C::sT + (it % C::NT) * (3 * kBlkBytes);
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        const uint32_t in[4] = {cr[i].x, cr[i].y, cr[i].z, cr[i].w};
        uint32_t t[3][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float x0 = bf16_lo(in[k]) * wj[i], x1 = bf16_hi(in[k]) * wj[i];
#pragma unroll
          for (int f = 0; f < 3; ++f) {  // the leading 8 bits of the significand, three times
            t[f][k] = __byte_perm(__float_as_uint(x0), __float_as_uint(x1), 0x7632);
            x0 -= __uint_as_float(__float_as_uint(x0) & 0xffff0000u);
            x1 -= __uint_as_float(__float_as_uint(x1) & 0xffff0000u);
          }
        }
#pragma unroll
        for (int f = 0; f < 3; ++f) sts128(set + f * kBlkBytes + blk_at(tid / 8 + STEP * i, tid % 8), t[f]);
        if (C::WIDE) cr[i] = cn[i];
      }
      if (!rev && n < kTC && len < p.T) {
        // a's rows behind the row's last token hold values that do not count: zeros
        wait(aF + 8 * (it % NA), (it / NA) & 1);
        const uint32_t z[4] = {0u, 0u, 0u, 0u};
        for (int k = tid; k < kTC * (DKB / 8); k += 32 * NCW) {
          const int row = k / (DKB / 8), ch = k % (DKB / 8);
          if (row >= n) sts128(sm + (it % NA) * C::A + (ch / 8) * kBlkBytes + blk_at(row, ch % 8), z);
        }
      }
      fence_async_smem();
      if (!(p.withhold && it == 0 && warp == 0)) warp_arrive(tR + 8 * (it % C::NT));
      if (C::WIDE)
        fetch(it + 2, cn);
      else
        fetch(it + 1, cr);
    };
    // the state at the start of chunk `it`, straight to the chunk states (by way of
    // shared memory and TMA stores the fence and barriers took 700 cycles a chunk)
    __nv_bfloat16* cs = static_cast<__nv_bfloat16*>(p.chunk_states) +
                        ((((long long)w.job * p.B * p.NH + w.bh) * nch + c0) * DK + gk) * p.DV + gv;
    auto publish = [&](int it) {
      if (STATE_ONLY || !owner) return;
#pragma unroll
      for (int j = 0; j < NC; j += 16) {
        uint32_t pk[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) pk[k] = pack_bf16x2(S[j + 2 * k], S[j + 2 * k + 1]);
        store32(cs + (long long)it * DK * p.DV + j, pk, true);
      }
    };
    // (after an abort the waits return at once and the loop runs out)
    if (cnt > 0) {
      make_terms(0);
      publish(0);
    }
    for (int it = 0; it < cnt; ++it) {
      if (C::NT == 2 && it + 1 < cnt) make_terms(it + 1);
      const int n = len - (c0 + it) * kTC < kTC ? len - (c0 + it) * kTC : kTC;
      const float wS = pw(lg, n);
      wait(mD + 8 * (it & 1), (it >> 1) & 1);
      tc_fence_after();
      if (owner) {
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
          for (int j = 0; j < 16; ++j) {  // smallest first
            const float hi = __uint_as_float(r0[j]), sum = (__uint_as_float(r2[j]) + __uint_as_float(r1[j])) + hi;
            // an infinite c or a: what it leaves to the lower terms is NaN, or zeros that meet it
            S[h + j] = fmaf(wS, S[h + j], sum == sum ? sum : hi);
          }
        }
      }
      tc_fence_before();
      warp_arrive(sR + 8 * (it % C::ND));
      if (it + 1 < cnt) {
        if (C::NT == 1) make_terms(it + 1);
        publish(it + 1);
      }
    }
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
  if (warp == C::WMMA) {
    if (lane == 0 && abort_flag_s) {
      drain(xD, 0);
      for (int k = issued_s - NA < 0 ? 0 : issued_s - NA; k < issued_s; ++k) drain(aF + 8 * (k % NA), (k / NA) & 1);
    }
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM);
  }
}

// --------------------------------------------------------------- outputs --
// One CTA per SM walks tiles of 128 tokens; two groups of eight compute warps take every
// other tile, so that one tile's scores are masked or its sums stored while the other's MMAs
// run.  The scores stay in TMEM: fp32 in, bf16 out over the same columns, from where
// P c takes them as its A operand.
template <int DK>
struct OutCfg {
  static constexpr int NGW = 8;                          // warps of a group
  static constexpr int WLOAD = 16, WMMA = 17, THREADS = 32 * 20;
  static constexpr uint32_t X = (DK / 64) * kBlkBytes;
  static constexpr int NX = DK == 64 ? 3 : (DK == 128 ? 2 : 1);  // tiles of x and a
  static constexpr uint32_t S = DK * 128;                // DK rows x 64 columns of the state
  static constexpr int NCS = DK == 64 ? 3 : 2;           // c and state tiles of 64 columns
  static constexpr uint32_t CS = kBlkBytes + S;
  // with 256 columns the second of them lies in a's place, free after the scores
  static constexpr uint32_t sCS = NX * 2 * X, sO = sCS + (DK == 256 ? 1 : NCS) * CS;
  static constexpr uint32_t SMEM = sO + 8 * 4096 + 1024;  // outputs on their way: 32 rows x 64 columns for two warps
  static __device__ __forceinline__ uint32_t cs_at(int buf) { return DK == 256 && buf == 1 ? X : sCS + buf * CS; }
};

// D[tmem] (+)= A[tmem, bf16 pairs] * B[smem]^T
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 16 consecutive 32-bit TMEM columns of this warp's lanes
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// a tile as the loading warp tells of it
struct OutTile {
  int job, c, h, b, len;
  float lg;               // log2 of the head's decay
};

// Tiles in the order pass, head, row, chunk (fastest first), the last chunk first: what the states' kernel touched
// last is still in L2.  A step of the grid is added digit by digit, and by the loading warp alone: the
// divisions of a place cost every role 700 cycles a tile, the digits' walk still 1,400 the MMAs' warp.
__device__ __forceinline__ OutTile digits(const LinAttnParams& p, int nch, int idx) {
  OutTile t;
  t.job = idx % p.npass;
  idx /= p.npass;
  t.h = idx % p.NH;
  idx /= p.NH;
  t.b = idx % p.B;
  t.c = nch - 1 - idx / p.B;
  return t;
}
__device__ __forceinline__ void advance(const LinAttnParams& p, int nch, OutTile& t, const OutTile& stride) {
  t.job += stride.job;  // (past the last tile c is below 0)
  t.h += stride.h;
  t.b += stride.b;
  t.c -= nch - 1 - stride.c;
  if (t.job >= p.npass) t.job -= p.npass, ++t.h;
  if (t.h >= p.NH) t.h -= p.NH, ++t.b;
  if (t.b >= p.B) t.b -= p.B, --t.c;
}

// Zero scores stand for a chunk's later tokens, and zero times a c that is not finite is NaN.  Where a P c came out so, the
// warp takes the outputs of its rows (32 q + lane, columns 64 v + 32 g ..) that are not finite again, token by token, each
// with the tokens up to it alone; once its tiles are done, since in their loop the registers for it cost 10-20%.
template <int DK>
__device__ __noinline__ void repair_rows(const LinAttnParams& p, int tiles, int grp, int q, int g) {
  const int nch = (p.T + kTC - 1) / kTC, lane = threadIdx.x & 31;
  const OutTile stride = digits(p, nch, (int)gridDim.x);
  OutTile at = digits(p, nch, blockIdx.x);
  depend_wait();  // (read here straight from memory: the chunk states)
  int k = 0;
  for (int idx = blockIdx.x; idx < tiles; idx += gridDim.x, advance(p, nch, at, stride)) {
    const int len = row_len(p, at.b), first = at.c * kTC;
    if (len <= first || (k++ & 1) != grp) continue;
    const LinAttnPass& ps = p.pass[at.job];
    // i: the row's place in its chunk, in the pass's time
    const int i = ps.reverse ? kTC - 1 - (32 * q + lane) : 32 * q + lane;
    if (first + i >= len) continue;
    auto token = [&](int j) { return (long long)(ps.reverse ? len - 1 - (first + j) : first + j); };
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(ps.x) + token(i) * ps.xs[0] + at.b * ps.xs[1] + at.h * ps.xs[2];
    const __nv_bfloat16* a = static_cast<const __nv_bfloat16*>(ps.a) + at.b * ps.as[1] + at.h * ps.as[2];
    const __nv_bfloat16* c = static_cast<const __nv_bfloat16*>(ps.c) + at.b * ps.cs[1] + at.h * ps.cs[2];
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(ps.out) + token(i) * ps.os[0] + at.b * ps.os[1] + at.h * ps.os[2];
    const __nv_bfloat16* S = static_cast<const __nv_bfloat16*>(p.chunk_states) +
                             ((((long long)at.job * p.B + at.b) * p.NH + at.h) * nch + at.c) * DK * p.DV;
    const float lg = p.log_decay[at.h] * 1.4426950408889634f;
    const float fr = ps.inter * pw(lg, i + 1 - ps.shift);
    auto fma8 = [](float (&o)[8], float f, const __nv_bfloat16* r) {
      const uint4 v = *reinterpret_cast<const uint4*>(r);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        o[2 * e] = fmaf(f, bf16_lo(w[e]), o[2 * e]);
        o[2 * e + 1] = fmaf(f, bf16_hi(w[e]), o[2 * e + 1]);
      }
    };
    // eights of columns: 4 of every 64
    const int eights = p.DV / 16;
    auto col_of = [&](int e) { return 64 * (e >> 2) + 32 * g + 8 * (e & 3); };
    uint32_t need = 0u;
    for (int e = 0; e < eights; ++e) {
      const uint4 v = *reinterpret_cast<const uint4*>(out + col_of(e));
      need |= (seen_finite(seen_finite(seen_finite(seen_finite(0u, v.x), v.y), v.z), v.w) != 0u ? 1u : 0u) << e;
    }
    if (need == 0u) continue;
    float o[16][8];
#pragma unroll 1
    for (int e = 0; e < eights; ++e) {
      if (!(need >> e & 1u)) continue;
      float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
      for (int d = 0; d < DK; ++d) fma8(y, __bfloat162float(x[d]), S + (long long)d * p.DV + col_of(e));
#pragma unroll
      for (int k = 0; k < 8; ++k) o[e][k] = y[k] * fr;
    }
#pragma unroll 1
    for (int j = 0; j <= i; ++j) {
      float s = 0.f;
#pragma unroll 1
      for (int d = 0; d < DK; d += 8) {
        float xf[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, af[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        fma8(xf, 1.f, x + d);
        fma8(af, 1.f, a + token(j) * ps.as[0] + d);
#pragma unroll
        for (int k = 0; k < 8; ++k) s = fmaf(xf[k], af[k], s);
      }
      s = bf16_round(s * (ps.intra * pw(lg, i - j)));
#pragma unroll 1
      for (int e = 0; e < eights; ++e)
        if (need >> e & 1u) fma8(o[e], s, c + token(j) * ps.cs[0] + col_of(e));
    }
#pragma unroll 1
    for (int e = 0; e < eights; ++e)
      if (need >> e & 1u)
        *reinterpret_cast<uint4*>(out + col_of(e)) = make_uint4(pack_bf16x2(o[e][0], o[e][1]), pack_bf16x2(o[e][2], o[e][3]),
                                                                pack_bf16x2(o[e][4], o[e][5]), pack_bf16x2(o[e][6], o[e][7]));
  }
}

template <int DK>
__global__ void __launch_bounds__(OutCfg<DK>::THREADS, 1)
    linattn_outputs_kernel(const __grid_constant__ LinAttnParams p, const __grid_constant__ TcMaps m,
                           int tiles) {
  using C = OutCfg<DK>;
  constexpr int NX = C::NX, NCS = C::NCS;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ int abort_flag_s, issued_s[2];  // copies of x and a, of c and the state
  __shared__ uint32_t tslot_s;
  __shared__ __align__(8) uint64_t bars_s[30];
  __shared__ OutTile info_s[4];  // what the loading warp tells the others of its tiles, the last four
  const uint32_t sm = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t bar = smem_u32(bars_s);
  // x, a landed; c, state landed; MMAs done, by buffer of c and state; scores done; scores in
  // bf16; sums read; c's rows behind the last token zeroed; info_s written; sums done, by group and parity of v; c landed
  // whose rows a group has to zero; scores multiplied; the last MMAs of all done.  A barrier's waiter waits for every one of its phases in turn (of one that it saw only
  // every other time it would take the phase before for the one that it wants: their parity is all it
  // sees), so what a group waits for has a barrier for each group.
  const uint32_t xF = bar, cF = bar + 24, dn = bar + 48, sc = bar + 72, pW = bar + 88, oR = bar + 104, cZ = bar + 120,
                 iF = bar + 136, oD = bar + 168, zF = bar + 200, sF = bar + 216, xD = bar + 232;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nch = (p.T + kTC - 1) / kTC;
  const int vts = p.DV / 64;
  const TcWait wait{p.status, p.timeout_ns, &abort_flag_s};

  int revs = 0;  // passes with reversed time
  for (int j = 0; j < p.npass; ++j) revs |= (p.pass[j].reverse != 0) << j;
  // first token of a tile's rows; whether rows of c have to be zeroed
  auto token_of = [&](const OutTile& t) { return (revs >> t.job) & 1 ? t.len - (t.c + 1) * kTC : t.c * kTC; };
  auto ragged = [&](const OutTile& t) {
    return t.len < p.T && t.len < (t.c + 1) * kTC && !((revs >> t.job) & 1);
  };
  // this CTA's tiles that hold tokens
  int count = ((int)blockIdx.x < tiles ? (tiles - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x : 0);
  if (p.lens != nullptr) {
    const OutTile stride = digits(p, nch, (int)gridDim.x);
    OutTile t = digits(p, nch, blockIdx.x);
    count = 0;
    for (int idx = blockIdx.x; idx < tiles; idx += gridDim.x, advance(p, nch, t, stride))
      count += row_len(p, t.b) > t.c * kTC;
  }

  if (tid == 0) {
    for (int i = 0; i < 11; ++i) mbar_init(bar + 8 * i, 1);
    for (int i = 11; i < 17; ++i) mbar_init(bar + 8 * i, C::NGW);
    for (int i = 17; i < 29; ++i) mbar_init(bar + 8 * i, 1);
    for (int i = 0; i < 3; ++i) mbar_init(dn + 8 * i, 2);  // (P c's and x S's)
    for (int i = 0; i < 4; ++i) mbar_init(oD + 8 * i, 2);
    mbar_init(xD, 3);
    abort_flag_s = issued_s[0] = issued_s[1] = 0;
    fence_mbar_init();
    fence_async_smem();
  }
  if (warp == C::WMMA) {
    tmem_alloc(smem_u32(&tslot_s), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tslot_s;  // two sets of scores (128 columns), then two of sums (P c, x S)

  if (warp == C::WLOAD) {
    // ------------------------------------------------------------- loads --
    if (lane == 0) {
      const OutTile stride = digits(p, nch, (int)gridDim.x);
      OutTile at = digits(p, nch, blockIdx.x);
      int f = 0, done = 0, xa = 0;  // c and state tiles; of these, known to be multiplied; tiles of x and a
      bool ok = true;
      auto multiplied = [&](int upto) {  // one after the other: no barrier is left two phases behind
        for (; ok && done < upto; ++done) ok = wait(dn + 8 * (done % NCS), (done / NCS) & 1);
        return ok;
      };
      auto next = [&]() {  // the next tile that holds tokens (there is one)
        for (;; advance(p, nch, at, stride)) {
          at.len = row_len(p, at.b);
          if (at.len > at.c * kTC) break;
        }
        OutTile t = at;
        t.lg = p.log_decay[t.h] * 1.4426950408889634f;
        advance(p, nch, at, stride);
        return t;
      };
      auto load_xa = [&](const OutTile& t, int k) {
        const int j = t.job, tok = token_of(t), s = k % NX;
        // (the roles have read the description of a tile before its last MMAs are issued)
        if (!multiplied((k - NX + 1) * vts)) return;
        info_s[k & 3] = t;
        mbar_arrive(iF + 8 * (k & 3));
        const uint32_t d = sm + s * (2 * C::X);
        mbar_arrive_expect_tx(xF + 8 * s, 2 * C::X);
#pragma unroll
        for (int i = 0; i < DK / 64; ++i) {
          tma_load_4d(d + i * kBlkBytes, &m.x[j], 64 * i, t.h * m.xh[j], t.b * m.xb[j], tok, xF + 8 * s);
          tma_load_4d(d + C::X + i * kBlkBytes, &m.a[j], 64 * i, t.h * m.ah[j], t.b * m.ab[j], tok, xF + 8 * s);
        }
        xa = k + 1;
      };
      // in the order in which the MMAs take them (the next tile's scores follow this one's first product
      // with the state): a copy whose buffer a later MMA has to free must not stand before one that this MMA needs
      OutTile t, tn;
      if (count > 0) {
        t = next();
        load_xa(t, 0);
      }
      depend_wait();  // for the chunk states (without a tile, too: a kernel that ends stands for those before it)
      for (int k = 0; ok && k < count; ++k) {
        const int j = t.job, tok = token_of(t), srow = (((j * p.B + t.b) * p.NH + t.h) * nch + t.c) * DK;
        for (int v = 0; ok && v < vts; ++v, ++f) {
          const int cb = f % NCS;
          if (!multiplied(f - NCS + 1)) break;
          if (DK == 256 && cb == 1) {  // in a's place: its scores are done
            if (!(ok = wait(sc + 8 * (k & 1), (k >> 1) & 1))) break;
          }
          mbar_arrive_expect_tx(cF + 8 * cb, C::CS);
          tma_load_2d(sm + C::cs_at(cb), &m.s_load, 64 * v, srow, cF + 8 * cb);
          tma_load_4d(sm + C::cs_at(cb) + C::S, &m.c[j], 64 * v, t.h * m.ch[j], t.b * m.cb[j], tok, cF + 8 * cb);
          if (v == 0 && k + 1 < count) {
            tn = next();
            if (NX > 1) load_xa(tn, k + 1);
          }
        }
        if (NX == 1 && ok && k + 1 < count) load_xa(tn, k + 1);
        t = tn;
      }
      issued_s[0] = xa, issued_s[1] = f;
    }
    __syncwarp();
  } else if (warp >= C::WMMA) {
    // -------------------------------------------------------------- MMAs --
    // Three warps issue, a product each, as soon as its own operands are there: one that issued all three held this
    // tile's P c back until the next tile's x and a had landed, 4,500 cycles of a tile's 7,000, and stood still
    // for the waits (100 cycles even when a phase is over) and commits (120).
    if (lane == 0 && warp == C::WMMA) {  // scores
      constexpr uint32_t idesc = idesc_bf16_f32(128, 128, false, false);
      for (int k = 0; k < count; ++k) {
        const uint32_t x = sm + (k % NX) * (2 * C::X), a = x + C::X;
        if (!wait(xF + 8 * (k % NX), (k / NX) & 1)) break;
        if (k >= 2 && !wait(sF + 8 * (k & 1), ((k - 2) >> 1) & 1)) break;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < DK / 16; ++ks) {
          const uint32_t o = (uint32_t)(ks / 4) * kBlkBytes + (ks % 4) * 32;
          umma_bf16(tmem + (k & 1) * 128, sdesc_sw128(x + o, 16, 1024), sdesc_sw128(a + o, 16, 1024), idesc,
                    ks != 0);
        }
        umma_commit(sc + 8 * (k & 1));
      }
      umma_commit(xD);
    } else if (lane == 0 && warp == C::WMMA + 1) {  // P c
      constexpr uint32_t idesc = idesc_bf16_f32(128, 64, false, true);
      uint32_t nz[2] = {0, 0};  // c tiles with rows zeroed, by group
      bool ok = true;
      int f = 0;
      for (int k = 0; ok && k < count; ++k) {
        if (!(ok = wait(pW + 8 * (k & 1), (k >> 1) & 1))) break;
        const bool zeroed = ragged(info_s[k & 3]);
        for (int v = 0; v < vts; ++v, ++f) {
          const int cb = f % NCS, o = f & 1;
          if (!(ok = wait(cF + 8 * cb, (f / NCS) & 1))) break;
          if (zeroed) {
            mbar_arrive(zF + 8 * (k & 1));
            if (!(ok = wait(cZ + 8 * (k & 1), nz[k & 1]++ & 1))) break;
          }
          if (f >= 2 && !(ok = wait(oR + 8 * o, ((f - 2) >> 1) & 1))) break;
          tc_fence_after();
          const uint32_t cc = sm + C::cs_at(cb) + C::S;
#pragma unroll
          for (int ks = 0; ks < kTC / 16; ++ks)
            umma_bf16_ts(tmem + 256 + o * 128, tmem + (k & 1) * 128 + ks * 8,
                         sdesc_sw128(cc + ks * 2048, kBlkBytes, 1024), idesc, ks != 0);
          umma_commit(oD + 8 * (2 * (k & 1) + (v & 1)));
          umma_commit(dn + 8 * cb);
        }
        if (ok) umma_commit(sF + 8 * (k & 1));
      }
      umma_commit(xD);
    } else if (lane == 0) {  // x S
      constexpr uint32_t idesc = idesc_bf16_f32(128, 64, false, true);
      bool ok = true;
      int f = 0;
      for (int k = 0; ok && k < count; ++k) {
        if (!(ok = wait(xF + 8 * (k % NX), (k / NX) & 1))) break;
        const uint32_t x = sm + (k % NX) * (2 * C::X);
        for (int v = 0; v < vts; ++v, ++f) {
          const int cb = f % NCS, o = f & 1;
          if (!(ok = wait(cF + 8 * cb, (f / NCS) & 1))) break;
          if (f >= 2 && !(ok = wait(oR + 8 * o, ((f - 2) >> 1) & 1))) break;
          tc_fence_after();
          const uint32_t st = sm + C::cs_at(cb);
#pragma unroll
          for (int ks = 0; ks < DK / 16; ++ks)
            umma_bf16(tmem + 256 + o * 128 + 64,
                      sdesc_sw128(x + (uint32_t)(ks / 4) * kBlkBytes + (ks % 4) * 32, 16, 1024),
                      sdesc_sw128(st + ks * 2048, kBlkBytes, 1024), idesc, ks != 0);
          umma_commit(oD + 8 * (2 * (k & 1) + (v & 1)));
          umma_commit(dn + 8 * cb);
        }
      }
      umma_commit(xD);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------- compute --
    const int grp = warp >> 3, q = warp & 3, g = (warp >> 2) & 1;
    const int row = 32 * q + lane, gt = tid & 255;  // thread of the group
    const uint32_t lanes = (uint32_t)(q * 32) << 16;
    const int id = 1 + grp * 4 + q;  // named barrier of the two warps of these rows
    const uint32_t tS = tmem + lanes + grp * 128;
    const uint32_t stg = sm + C::sO + (grp * 4 + q) * 4096;
    uint32_t nz = 0;  // c tiles with rows zeroed
    if (p.lens != nullptr) {
      // Zeros for tokens that do not count, of tiles without tokens and of reversed ones (whose rows
      // are other tokens): row r0 + row, 64 v + 32 g ..
      const OutTile stride = digits(p, nch, (int)gridDim.x);
      OutTile t = digits(p, nch, blockIdx.x);
      for (int idx = blockIdx.x; idx < tiles; idx += gridDim.x, advance(p, nch, t, stride)) {
        t.len = row_len(p, t.b);
        const int r = t.c * kTC + row;
        if (grp != 0 || r < t.len || r >= p.T || (t.len > t.c * kTC && !((revs >> t.job) & 1))) continue;
        const LinAttnPass& ps = p.pass[t.job];
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(ps.out) + (long long)r * ps.os[0] + t.b * ps.os[1] +
                           t.h * ps.os[2] + 32 * g;
        for (int v = 0; v < vts; ++v)
#pragma unroll
          for (int j = 0; j < 32; j += 8) *reinterpret_cast<uint4*>(o + 64 * v + j) = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    bool spoilt = false;  // a row of P c that is not finite
    for (int k = grp; k < count; k += 2) {
      // After an abort the waits of a tile return at once, and the two warps of a named barrier leave
      // the loop together.
      const bool told = wait(iF + 8 * (k & 3), (k >> 2) & 1);
      if (bar_red_or(id, 64, !told)) break;
      const OutTile t = info_s[k & 3];
      const int n = t.len - t.c * kTC < kTC ? t.len - t.c * kTC : kTC;
      const LinAttnPass& ps = p.pass[t.job];
      const bool rev = (revs >> t.job) & 1;
      const float lg = t.lg, lam = pw(lg, 1);
      const float fr = ps.inter * pw(lg, (rev ? kTC - 1 - row : row) + 1 - ps.shift);
      // blocks of 32 columns g and g + 2; powers from the column nearest to the diagonal on, each lambda
      // times the one before
      float f0[2];
      int live[2];  // last (reversed: first) column that counts; 32 (-1): none
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int blk = g + 2 * i, d = rev ? 32 * (blk - q) - lane : lane + 32 * (q - blk) - 31;
        f0[i] = ps.intra * (blk == q ? 1.f : pw(lg, d > 0 ? d : 0));
        live[i] = blk == q ? lane : ((rev ? blk > q : blk < q) ? (rev ? 0 : 31) : (rev ? 32 : -1));
      }
      wait(sc + 8 * grp, (k >> 1) & 1);
      tc_fence_after();
      uint32_t pk[2][16];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int blk = g + 2 * i;
        if (rev ? blk >= q : blk <= q) {
          uint32_t s[32];
          tmem_ld32(tS + 32 * blk, s);
          tmem_wait_ld();
          tmem_reg_fence(s);
          float fac = f0[i];
          if (rev) {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const bool on = j >= live[i];
              s[j] = on ? __float_as_uint(__uint_as_float(s[j]) * fac) : 0u;
              fac = on ? fac * lam : fac;
            }
          } else {
#pragma unroll
            for (int j = 31; j >= 0; --j) {
              const bool on = j <= live[i];
              s[j] = on ? __float_as_uint(__uint_as_float(s[j]) * fac) : 0u;
              fac = on ? fac * lam : fac;
            }
          }
#pragma unroll
          for (int j = 0; j < 16; ++j)
            pk[i][j] = pack_bf16x2(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1]));
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) pk[i][j] = 0u;
        }
      }
      bar_sync(id, 64);  // both warps of these rows have read their scores
      tmem_st16(tS + 16 * g, pk[0]);
      tmem_st16(tS + 16 * (g + 2), pk[1]);
      tmem_wait_st();
      tc_fence_before();
      if (!(p.withhold && k == 0 && warp == 0)) warp_arrive(pW + 8 * grp);
      const int tok0 = token_of(t) + 32 * q;  // of this warp's first row (reversed: possibly below 0)
      const bool zero_c = ragged(t), counts = rev ? row >= kTC - n : row < n;
      for (int v = 0; v < vts; ++v) {
        const int f = k * vts + v, o = f & 1;
        if (zero_c) {
          const int cb = f % NCS;
          wait(zF + 8 * grp, nz++ & 1);
          const uint32_t z[4] = {0u, 0u, 0u, 0u};
          for (int e = gt; e < kTC * 8; e += 256)
            if (e / 8 >= n) sts128(sm + C::cs_at(cb) + C::S + blk_at(e / 8, e % 8), z);
          fence_async_smem();
          warp_arrive(cZ + 8 * grp);
        }
        const int vp = v & 1;  // (k >> 1) tiles of this group before, (vts + 1 - vp) / 2 sums of v's parity in each
        wait(oD + 8 * (2 * grp + vp), ((k >> 1) * ((vts + 1 - vp) / 2) + (v >> 1)) & 1);
        tc_fence_after();
        uint32_t w[16];
        float top = 0.f;  // of P c
        const uint32_t tO = tmem + 256 + o * 128 + lanes + 32 * g;
#pragma unroll
        for (int h = 0; h < 32; h += 16) {
          uint32_t u[16], s[16];
          tmem_ld16(tO + h, u);
          tmem_ld16(tO + 64 + h, s);
          tmem_wait_ld();
          reg_fence(u);
          reg_fence(s);
#pragma unroll
          for (int j = 0; j < 16; j += 2) top = max_abs3(top, __uint_as_float(u[j]), __uint_as_float(u[j + 1]));
#pragma unroll
          for (int j = 0; j < 8; ++j)
            w[h / 2 + j] =
                counts ? pack_bf16x2(fmaf(fr, __uint_as_float(s[2 * j]), __uint_as_float(u[2 * j])),
                                     fmaf(fr, __uint_as_float(s[2 * j + 1]), __uint_as_float(u[2 * j + 1])))
                       : 0u;
        }
        spoilt |= counts && !(top < INFINITY);
        tc_fence_before();
        warp_arrive(oR + 8 * o);
        if (tok0 >= 0) {
          if (g == 0 && lane == 0) bulk_wait_read_all();
          bar_sync(id, 64);
#pragma unroll
          for (int j = 0; j < 4; ++j) sts128(stg + blk_at(lane, 4 * g + j), w + 4 * j);
          fence_async_smem();
          bar_sync(id, 64);
          if (g == 0 && lane == 0) {
            tma_store_4d(&m.out[t.job], 64 * v, t.h, t.b, tok0, stg);
            bulk_commit();
          }
        } else if (tok0 + lane >= 0) {  // a store may not begin before token 0
          __nv_bfloat16* go = static_cast<__nv_bfloat16*>(ps.out) + (long long)(tok0 + lane) * ps.os[0] +
                              t.b * ps.os[1] + t.h * ps.os[2] + 64 * v + 32 * g;
          store32(go, w, false);
          store32(go + 16, w + 8, false);
        }
      }
    }
    if (g == 0 && lane == 0) bulk_wait_all();
    __syncwarp();
    if (bar_red_or(id, 64, spoilt)) repair_rows<DK>(p, tiles, grp, q, g);  // (behind the stores of both warps' columns)
  }
  tc_fence_before();
  __syncthreads();
  if (warp == C::WMMA) {
    if (lane == 0 && abort_flag_s) {
      drain(xD, 0);
      for (int k = issued_s[0] - NX < 0 ? 0 : issued_s[0] - NX; k < issued_s[0]; ++k) drain(xF + 8 * (k % NX), (k / NX) & 1);
      for (int k = issued_s[1] - NCS < 0 ? 0 : issued_s[1] - NCS; k < issued_s[1]; ++k)
        drain(cF + 8 * (k % NCS), (k / NCS) & 1);
    }
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
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
  *uh = s[2] != 0;
  *ub = s[1] != 0;
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
  int one;
  for (int j = 0; j < p.npass; ++j) {
    const LinAttnPass& ps = p.pass[j];
    const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
    ok = ok && encode_operand(&m.x[j], ps.x, ps.xs, p, DK, 64, kTC, sw, &m.xh[j], &m.xb[j]);
    ok = ok && encode_operand(&m.a[j], ps.a, ps.as, p, DK, 64, kTC, sw, &m.ah[j], &m.ab[j]);
    ok = ok && encode_operand(&m.c[j], ps.c, ps.cs, p, p.DV, 64, kTC, sw, &m.ch[j], &m.cb[j]);
    ok = ok && encode_operand(&m.out[j], ps.out, ps.os, p, p.DV, 64, 32, sw, &one, &one);
  }
  const cuuint64_t dims[2] = {(cuuint64_t)p.DV, (cuuint64_t)(outs * DK)};
  const cuuint64_t strides[1] = {(cuuint64_t)p.DV * 2};
  const cuuint32_t in[2] = {64, (cuuint32_t)DK};
  ok = ok && encode(&m.s_load, p.chunk_states, 2, dims, strides, in, CU_TENSOR_MAP_SWIZZLE_128B);
  if (!ok) return kLinAttnTooWide;
  if (p.nseg > 1) {
    e = prepare_launch(prep_state, linattn_states_kernel<DK, true>, C::SMEM, C::THREADS, 1);
    if (e != 0) return e;
    e = launch_dependent(linattn_states_kernel<DK, true>, (unsigned)(base * (p.nseg - 1)), C::THREADS, C::SMEM, s, p, m);
    if (e != 0) return e;
    e = launch_dependent(linattn_scan_kernel<TcOrder<DK>>, (unsigned)(base * (C::TILE / 256)), 256, 0, s, p,
                         p.seg_chunks * kTC);
    if (e != 0) return e;
    e = launch_dependent(linattn_states_kernel<DK, false>, (unsigned)(base * p.nseg), C::THREADS, C::SMEM, s, p, m);
  } else {
    e = launch_dependent(linattn_states_kernel<DK, false>, (unsigned)base, C::THREADS, C::SMEM, s, p, m);
  }
  if (e != 0) return e;
  const long long cap = sm_count();
  e = launch_dependent(linattn_outputs_kernel<DK>, (unsigned)(outs < cap ? outs : cap), O::THREADS, O::SMEM, s, p,
                       m, (int)outs);
  return e;
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
