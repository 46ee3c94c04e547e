// Which kernels a linear-attention call takes, and how it cuts the token axis.
#include "kernels.h"
#include "lm.h"

namespace srnn {

LinAttnPlan linattn_plan(bool bf16, int npass, int T, int B, int NH, int DK, int DV) {
  LinAttnPlan pl{};
  // tcgen05 from the lengths on where it is the faster (us, 8 rows unless said; mma.sync / tcgen05): 6 x 128,
  // T = 128 13.5 / 17.0, T = 256 21.5 / 18.8, 16 rows of 1024 108 / 63; 4 x 256, T = 256 29.9 / 29.3, 4 rows of 4096 370 /
  // 98.  With 64 columns of x and a, whose products are small, the gradient's passes gain on long rows only
  // (16 rows of 1024 104 / 113, 4 rows of 4096 154 / 123), the forward's does not (1 row of 4096 24.8 / 34.1).
  const bool tc = DK % 64 == 0 && DV % 64 == 0 && (DK == 64 ? npass > 1 && T >= 2048 : T >= 256);
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
    tiles = DV / 32;
    occ = DK <= 64 ? 4 : (DK == 128 ? 3 : 2);
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
    const long long cost = (waves + 1) * per + 8;
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
