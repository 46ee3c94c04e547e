// Which kernels a linear-attention call takes, and how it cuts the token axis.
#include "kernels.h"
#include "lm.h"

namespace srnn {

LinAttnPlan linattn_plan(bool bf16, int npass, int T, int B, int NH, int DK, int DV) {
  LinAttnPlan pl{};
  // tcgen05 where it is the faster (us, mma.sync / tcgen05, T x rows x heads x Dk x Dv).  Dk of 128 or more: from 128
  // tokens on (128x8x6x128x128 12.7 / 10.1, its gradient 24.1 / 17.3; 128x8x4x256x256 16.8 / 17.4, 45.7 / 32.9; 64 tokens
  // 8.3 / 9.9 and 15.7 / 17.0; few heads: 128x1x1x128x128 9.0 / 9.9, 9.0 / 12.0, 256x1x2x128x128 14.4 / 10.9, 14.4 / 12.1,
  // 128x1x1x256x256 12.4 / 11.8, 12.3 / 12.7; 128x1x2x256x64 12.3 / 9.8).  Dk = 64, whose products with a are small, against
  // wider values: the gradient from 192 tokens on (200x16x8x64x128 59 / 40; 128x2x8 15.6 / 18.1), the forward pass from 512
  // (512x2x8 16.0 / 14.1, 1024x16x8 53 / 43; 256x8x8 12.6 / 13.9).  64 x 64: the gradient's passes on long rows (4096x4x12
  // 150 / 119; 1024x16x12 101 / 105, 2048x8x12 101.7 / 101.8), the forward pass with enough long rows (1024x4x12 28.4 /
  // 23.6, 2048x8x12 67.5 / 52.0; 16384x1x12 55.7 / 58.1, 512x16x12 25.8 / 26.5).
  const long long heads = (long long)B * NH;
  bool tc = DK % 64 == 0 && DV % 64 == 0;
  if (DK > 64)
    tc = tc && T >= 128;
  else if (DV > 64)
    tc = tc && T >= (npass > 1 ? 192 : 512);
  else
    tc = tc && (npass > 1 ? T >= 4096 : T >= 1024 && heads >= 48);
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
