// Which kernels a linear-attention call takes, and how it cuts the token axis.
#include "kernels.h"
#include "lm.h"

namespace srnn {

LinAttnPlan linattn_plan(bool bf16, int npass, int T, int B, int NH, int DK, int DV) {
  LinAttnPlan pl{};
  // tcgen05 where it is the faster (us, mma.sync / tcgen05, T x rows x heads x Dk x Dv).  Dk of 128 or more: from 128
  // tokens on (128x8x6x128x128 12.1 / 9.5, its gradient 23.0 / 16.4; 128x8x4x256x256 16.8 / 16.7, 44.8 / 32.2; 64 tokens
  // 8.2 / 9.3 and 11.4 / 16.5).  Dk = 64, whose products with a are small, against wider values: the gradient from 192
  // tokens on (200x16x8x64x128 58 / 40; 128x2x8 14.4 / 16.5), the forward pass from 512 (512x2x8 15.4 / 13.3, 1024x16x8 69 /
  // 42; 256x8x8 12.8 / 13.5).  64 x 64: the gradient's passes on long rows (4096x4x12 148 / 119; 1024x16x12 101 / 108,
  // 2048x8x12 100 / 105), the forward pass with enough long rows (1024x4x12 27.8 / 22.6, 2048x8x12 66.9 / 51.1;
  // 16384x1x12 55.3 / 57.1, 512x16x12 25.3 / 26.3).
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
