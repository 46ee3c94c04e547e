// Which kernels a linear-attention call takes, and how it cuts the token axis.
#include "kernels.h"
#include "lm.h"

namespace srnn {

LinAttnPlan linattn_plan(bool bf16, int npass, int T, int B, int NH, int DK, int DV) {
  LinAttnPlan pl{};
  // tcgen05 where it is the faster (us, mma.sync / tcgen05, T x rows x heads x Dk x Dv unless said).  Both sizes 128
  // or more: from 256 tokens on (256x8x6x128x128 20.6 / 16.7, its gradient 39 / 25; 256x8x4x256x256 27.8 / 25.1; the
  // same at 128 tokens 17.2 / 20.9).  Dk = 64, whose products with a are small, against wider values: the gradient from
  // 256 tokens on (256x8x8x64x128 32.4 / 31.2, 1024x16 187 / 115), the forward pass with enough work (1024x16x8 52.9 /
  // 46.1, 16384x1x8 70.9 / 62.7; 512x16x8 28.7 / 29.0, 2048x1x8 20.1 / 25.2).  64 x 64: the gradient's passes on long rows
  // (4096x4x12 147 / 124; 2048x8x12 100 / 109), the forward pass with many long rows (2048x8x12 66.4 / 55.3,
  // 1024x16x12 53.2 / 48.4; 4096x4x12 64.5 / 66.9, 16384x1x12 54.8 / 61.2).
  const long long heads = (long long)B * NH;
  bool tc = DK % 64 == 0 && DV % 64 == 0;
  if (DK > 64)
    tc = tc && T >= 256;
  else if (DV > 64)
    tc = tc && (npass > 1 ? T >= 256 : T >= 1024 && T * heads >= 65536);
  else
    tc = tc && (npass > 1 ? T >= 4096 : T >= 1024 && heads >= 96);
  pl.path = !bf16 ? kLinAttnF32 : (tc ? kLinAttnTc : kLinAttnMma);
  int chunk, tiles, occ;  // tokens per chunk, state tiles per head, CTAs per SM
  if (pl.path == kLinAttnTc) {
    chunk = 128;
    tiles = (DK > 128 ? DK / 128 : 1) * (DV / 64);
    occ = DK == 64 ? 2 : 1;
  } else if (pl.path == kLinAttnMma) {
    chunk = 64;
    tiles = DV % 64 == 0 ? DV / 64 : DV / 32;
    occ = DK <= 64 ? 3 : (DK == 128 ? 2 : 1);
  } else {
    chunk = 32;
    tiles = DV % 64 == 0 ? DV / 64 : DV / 32;
    occ = DK <= 64 ? 4 : (DK == 128 ? 2 : 1);
  }
  const long long nch = ((long long)T + chunk - 1) / chunk;
  const long long base = (long long)npass * B * NH * tiles;
  const long long cap = (long long)sm_count() * occ;
  // Chunks one after the other on the busiest SM: all of them, or with segments twice
  // a segment's (its contribution, then the states or outputs) and what the extra
  // launches and the scan cost, about eight chunks' time.
  long long nseg = 1, best = ((base + cap - 1) / cap) * nch;
  for (long long n = 2; base > 0 && n <= nch / 2 && base * (n - 1) < cap; ++n) {
    const long long per = (nch + n - 1) / n, waves = (base * n + cap - 1) / cap;
    // (fp32: the contributions are a product of three, at most)
    const long long cost = pl.path == kLinAttnF32 ? waves * per + (per + 1) / 2 + 4 : (waves + 1) * per + 8;
    if (cost < best) best = cost, nseg = n;
  }
  const long long per = nch > 0 ? (nch + nseg - 1) / nseg : 1;
  pl.seg_chunks = (int)per;
  pl.nseg = nch > 0 ? (int)((nch + per - 1) / per) : 1;
  const size_t state = (size_t)npass * B * NH * DK * DV;
  pl.seg_bytes = pl.nseg > 1 ? pl.nseg * state * sizeof(float) : 0;
  pl.chunk_bytes = pl.path == kLinAttnTc ? (size_t)nch * state * 2 : 0;
  return pl;
}

}  // namespace srnn
