// C ABI of the language-model operators (declared in include/rnn.h): argument
// checks, workspace layouts, launches on the caller's stream.
#include <cuda_runtime.h>

#include <cstdint>

#include "api.h"
#include "lm.h"

using namespace srnn;
using namespace srnn::api;

namespace {

bool valid_dtype(int32_t d) { return d == RNN_F32 || d == RNN_BF16; }
// the widest row: the kernels count its columns, rounded up to tiles or strided over by a grid's share, in 32 bits
constexpr int32_t kMaxCols = INT32_MAX - 4095;
size_t dtype_bytes(int32_t d) { return d == RNN_F32 ? 4 : 2; }
bool head_dim_ok(int32_t d) { return d == 32 || d == 64 || d == 128 || d == 256; }

int check_linattn(const rnn_linattn_desc_t* d) {
  if (d == nullptr || !valid_dtype(d->dtype)) return RNN_ERR_INVALID_ARG;
  if (d->T < 0 || d->B < 0 || d->NH < 0 || d->Dk <= 0 || d->Dv <= 0 ||
      (d->flags & ~RNN_FLAG_TEST_TIMEOUT) != 0)
    return RNN_ERR_INVALID_ARG;
  if (!head_dim_ok(d->Dk) || !head_dim_ok(d->Dv) || d->T > (1 << 30)) return RNN_ERR_UNSUPPORTED;
  // one CTA per row, head, column tile and segment: the largest grid
  if ((long long)d->B * d->NH > (1 << 20)) return RNN_ERR_UNSUPPORTED;
  return RNN_OK;
}

// strides of a [T, B, NH, D] operand: the caller's, or contiguous
struct St {
  long long s[3];
};
St strides_or(const int64_t* given, const rnn_linattn_desc_t* d, int D) {
  St r;
  if (given != nullptr) {
    for (int i = 0; i < 3; ++i) r.s[i] = given[i];
  } else {
    r.s[2] = D;
    r.s[1] = (long long)d->NH * D;
    r.s[0] = (long long)d->B * d->NH * D;
  }
  return r;
}
bool strides_aligned(const St& s, size_t esize, int first = 0) {  // (1: without the token's)
  for (int i = first; i < 3; ++i)
    if (s.s[i] < 0 || s.s[i] % (long long)(16 / esize) != 0) return false;
  return true;
}
void set3(long long (&dst)[3], const St& s) {
  for (int i = 0; i < 3; ++i) dst[i] = s.s[i];
}

size_t plan_bytes(const LinAttnPlan& pl) {
  return align_up(pl.seg_bytes, 256) + align_up(pl.chunk_bytes, 256);
}
// workspace of the gradient: the passes of dq and dk contract over Dv, dv's over Dk;
// with equal sizes the three run as one launch
size_t linattn_ws(const rnn_linattn_desc_t* d, int pass) {
  const bool bf16 = d->dtype == RNN_BF16;
  if (pass == 0) return plan_bytes(linattn_plan(bf16, 1, d->T, d->B, d->NH, d->Dk, d->Dv));
  if (d->Dk == d->Dv) return plan_bytes(linattn_plan(bf16, 3, d->T, d->B, d->NH, d->Dk, d->Dv));
  const size_t a = plan_bytes(linattn_plan(bf16, 2, d->T, d->B, d->NH, d->Dv, d->Dk));
  const size_t b = plan_bytes(linattn_plan(bf16, 1, d->T, d->B, d->NH, d->Dk, d->Dv));
  return a > b ? a : b;  // the two launches follow one another on the stream
}

// RNN_FLAG_TEST_TIMEOUT is for the kernels that wait on the device
bool waits(const rnn_linattn_desc_t* d, int pass) {
  const bool bf16 = d->dtype == RNN_BF16;
  auto tc = [&](int npass, int DK, int DV) {
    return linattn_plan(bf16, npass, d->T, d->B, d->NH, DK, DV).path == kLinAttnTc;
  };
  if (pass == 0) return tc(1, d->Dk, d->Dv);
  return d->Dk == d->Dv ? tc(3, d->Dk, d->Dv) : tc(2, d->Dv, d->Dk) && tc(1, d->Dk, d->Dv);
}

int run_passes(LinAttnParams& p, bool bf16, int DK, int DV, void* workspace, cudaStream_t s) {
  p.DK = DK;
  p.DV = DV;
  const LinAttnPlan pl = linattn_plan(bf16, p.npass, p.T, p.B, p.NH, DK, DV);
  p.nseg = pl.nseg;
  p.seg_chunks = pl.seg_chunks;
  char* ws = static_cast<char*>(workspace) + kStatusBytes;
  p.ws = reinterpret_cast<float*>(ws);
  p.chunk_states = ws + align_up(pl.seg_bytes, 256);
  p.status = static_cast<int*>(workspace);
  p.timeout_ns = p.withhold ? kTestTimeoutNs : kTimeoutNs;
  if (pl.path == kLinAttnTc) {
    const int e = launch_linattn_tc(p, s);
    if (e != kLinAttnTooWide) return e;
    p.nseg = 1;  // the other kernels, with the token axis in one piece: no workspace
    p.seg_chunks = p.T / 64 + 1;
    return launch_linattn_mma(p, s);
  }
  return pl.path == kLinAttnMma ? launch_linattn_mma(p, s) : launch_linattn_f32(p, s);
}

}  // namespace

extern "C" {

int rnn_rms_norm(int32_t dtype, int32_t rows, int32_t N, float eps, const void* x,
                 const void* residual, const float* weight, void* h, void* y, float* scale,
                 float* rstd, void* stream) {
  if (!valid_dtype(dtype) || rows < 0 || N <= 0 || !(eps >= 0.f)) return RNN_ERR_INVALID_ARG;
  if (N > kMaxCols) return RNN_ERR_UNSUPPORTED;
  if (rows == 0) return RNN_OK;
  if (x == nullptr || weight == nullptr || y == nullptr) return RNN_ERR_INVALID_ARG;
  const size_t es = dtype_bytes(dtype);
  if (!aligned(x, es) || !aligned(residual, es) || !aligned(h, es) || !aligned(weight, 4) ||
      !aligned(scale, 4) || !aligned(rstd, 4) || (scale == nullptr && !aligned(y, es)))
    return RNN_ERR_MISALIGNED;
  NormParams p{x, residual, weight, h, y, scale, rstd, rows, N, eps};
  return map_launch_error(launch_rms_norm(p, dtype == RNN_BF16, static_cast<cudaStream_t>(stream)));
}

size_t rnn_rms_norm_bwd_workspace_size(int32_t rows, int32_t N) {
  if (rows < 0 || N <= 0) return 0;
  return kStatusBytes + align_up((size_t)norm_bwd_parts(rows, N) * N * sizeof(float), 256);
}

int rnn_rms_norm_bwd(int32_t dtype, int32_t rows, int32_t N, const void* dy, const void* h,
                     const float* weight, const float* rstd, const void* dh, void* dx, float* dw,
                     void* workspace, size_t workspace_bytes, void* stream) {
  if (!valid_dtype(dtype) || rows < 0 || N <= 0) return RNN_ERR_INVALID_ARG;
  if (N > kMaxCols) return RNN_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    if (dw == nullptr) return RNN_OK;
    if (!aligned(dw, 4)) return RNN_ERR_MISALIGNED;
    return cudaMemsetAsync(dw, 0, (size_t)N * sizeof(float), s) == cudaSuccess ? RNN_OK
                                                                                : RNN_ERR_LAUNCH;
  }
  if (dy == nullptr || h == nullptr || weight == nullptr || rstd == nullptr || dx == nullptr)
    return RNN_ERR_INVALID_ARG;
  if (dw != nullptr && (workspace == nullptr || workspace_bytes < rnn_rms_norm_bwd_workspace_size(rows, N)))
    return RNN_ERR_INVALID_ARG;
  const size_t es = dtype_bytes(dtype);
  if (!aligned(dy, es) || !aligned(h, es) || !aligned(dh, es) || !aligned(dx, es) ||
      !aligned(weight, 4) || !aligned(rstd, 4) || !aligned(dw, 4) || !aligned(workspace, 256))
    return RNN_ERR_MISALIGNED;
  NormBwdParams p{dy, h, weight, rstd, dh, dx, dw, nullptr, rows, N};
  if (dw != nullptr)
    p.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + kStatusBytes);
  return map_launch_error(launch_rms_norm_bwd(p, dtype == RNN_BF16, s));
}

int rnn_quantize_weight(int32_t dtype, int32_t N, int32_t K, const void* W, void* Wq, float* Ws,
                        void* stream) {
  if (!valid_dtype(dtype) || N <= 0 || K <= 0) return RNN_ERR_INVALID_ARG;
  if (N > 65535 * 128 || K > kMaxCols) return RNN_ERR_UNSUPPORTED;
  if (W == nullptr || Wq == nullptr || Ws == nullptr) return RNN_ERR_INVALID_ARG;
  if (!aligned(W, dtype_bytes(dtype)) || !aligned(Ws, 4)) return RNN_ERR_MISALIGNED;
  return map_launch_error(
      launch_quantize_weight(W, dtype == RNN_BF16, N, K, Wq, Ws, static_cast<cudaStream_t>(stream)));
}

int rnn_input_proj_fp8(int32_t M, int32_t N, int32_t K, const void* xq, const float* xs,
                       const void* Wq, const float* Ws, const float* bias, void* y,
                       void* workspace, size_t workspace_bytes, void* stream) {
  if (M < 0 || N <= 0 || K <= 0) return RNN_ERR_INVALID_ARG;
  if (workspace == nullptr || workspace_bytes < kStatusBytes) return RNN_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return RNN_ERR_MISALIGNED;
  if (K % 16 != 0 || N % 8 != 0 || M > 65535 * 128 || N > kMaxCols || K > kMaxCols)
    return RNN_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 0) return clear_status(workspace, workspace_bytes, s);
  if (xq == nullptr || xs == nullptr || Wq == nullptr || Ws == nullptr || y == nullptr)
    return RNN_ERR_INVALID_ARG;
  if (!aligned(xq, 16) || !aligned(Wq, 16) || !aligned(y, 16) || !aligned(xs, 4) ||
      !aligned(Ws, 4) || !aligned(bias, 4))
    return RNN_ERR_MISALIGNED;
  ProjFp8Params p{xq, xs, Wq, Ws, bias, y, M, N, K, static_cast<int*>(workspace), kTimeoutNs};
  return map_launch_error(launch_proj_fp8(p, s));
}

size_t rnn_linattn_workspace_size(const rnn_linattn_desc_t* d, int pass) {
  if (check_linattn(d) != RNN_OK || (pass != 0 && pass != 1)) return 0;
  return kStatusBytes + linattn_ws(d, pass);
}

int rnn_linattn_fwd(const rnn_linattn_desc_t* d, const rnn_linattn_strides_t* st, const void* q,
                    const void* k, const void* v, const float* log_decay, const int32_t* lens,
                    const float* state0, void* o, float* stateT, void* workspace,
                    size_t workspace_bytes, void* stream) {
  int e = check_linattn(d);
  if (e != RNN_OK) return e;
  if (workspace == nullptr || workspace_bytes < rnn_linattn_workspace_size(d, 0))
    return RNN_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return RNN_ERR_MISALIGNED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d->B == 0 || d->NH == 0) return clear_status(workspace, workspace_bytes, s);
  if (d->flags != 0 && !waits(d, 0)) return RNN_ERR_UNSUPPORTED;
  if (log_decay == nullptr) return RNN_ERR_INVALID_ARG;
  if (d->T > 0 && (q == nullptr || k == nullptr || v == nullptr || o == nullptr))
    return RNN_ERR_INVALID_ARG;
  const size_t es = dtype_bytes(d->dtype);
  const St sq = strides_or(st ? st->q : nullptr, d, d->Dk), sk = strides_or(st ? st->k : nullptr, d, d->Dk);
  const St sv = strides_or(st ? st->v : nullptr, d, d->Dv), so = strides_or(st ? st->o : nullptr, d, d->Dv);
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) ||
      !aligned(state0, 16) || !aligned(stateT, 16) || !aligned(log_decay, 4) || !aligned(lens, 4) ||
      !strides_aligned(sq, es) || !strides_aligned(sk, es) || !strides_aligned(sv, es) ||
      !strides_aligned(so, es))
    return RNN_ERR_MISALIGNED;
  LinAttnParams p{};
  p.npass = 1;
  p.clear = 1;
  p.withhold = d->flags != 0;
  p.log_decay = log_decay;
  p.lens = lens;
  p.T = d->T;
  p.B = d->B;
  p.NH = d->NH;
  LinAttnPass& a = p.pass[0];
  a.x = q;
  a.a = k;
  a.c = v;
  a.out = o;
  a.init = state0;
  a.fin = stateT;
  set3(a.xs, sq);
  set3(a.as, sk);
  set3(a.cs, sv);
  set3(a.os, so);
  a.intra = a.inter = d->scale;
  a.upd = 1.f;
  return map_launch_error(run_passes(p, d->dtype == RNN_BF16, d->Dk, d->Dv, workspace, s));
}

int rnn_linattn_bwd(const rnn_linattn_desc_t* d, const rnn_linattn_strides_t* st, const void* q,
                    const void* k, const void* v, const float* log_decay, const int32_t* lens,
                    const float* state0, const void* dout, const float* dstateT, void* dq, void* dk,
                    void* dv, float* dstate0, void* workspace, size_t workspace_bytes,
                    void* stream) {
  int e = check_linattn(d);
  if (e != RNN_OK) return e;
  if (workspace == nullptr || workspace_bytes < rnn_linattn_workspace_size(d, 1))
    return RNN_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return RNN_ERR_MISALIGNED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d->B == 0 || d->NH == 0) return clear_status(workspace, workspace_bytes, s);
  if (d->flags != 0 && !waits(d, 1)) return RNN_ERR_UNSUPPORTED;
  if (log_decay == nullptr) return RNN_ERR_INVALID_ARG;
  if (d->T > 0 && (q == nullptr || k == nullptr || v == nullptr || dout == nullptr ||
                   dq == nullptr || dk == nullptr || dv == nullptr))
    return RNN_ERR_INVALID_ARG;
  // the passes run at once: some read state0 and dstateT while another writes dstate0
  if (dstate0 != nullptr && (dstateT == dstate0 || state0 == dstate0)) return RNN_ERR_INVALID_ARG;
  const size_t es = dtype_bytes(d->dtype);
  const St sq = strides_or(st ? st->q : nullptr, d, d->Dk), sk = strides_or(st ? st->k : nullptr, d, d->Dk);
  const St sv = strides_or(st ? st->v : nullptr, d, d->Dv), so = strides_or(st ? st->o : nullptr, d, d->Dv);
  const St gk = strides_or(nullptr, d, d->Dk), gv = strides_or(nullptr, d, d->Dv);
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(dout, 16) ||
      !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16) || !aligned(state0, 16) ||
      !aligned(dstateT, 16) || !aligned(dstate0, 16) || !aligned(log_decay, 4) ||
      !aligned(lens, 4) || !strides_aligned(sq, es) || !strides_aligned(sk, es) ||
      !strides_aligned(sv, es) || !strides_aligned(so, es))
    return RNN_ERR_MISALIGNED;
  LinAttnParams p{};
  p.clear = 1;
  p.withhold = d->flags != 0;
  p.log_decay = log_decay;
  p.lens = lens;
  p.T = d->T;
  p.B = d->B;
  p.NH = d->NH;
  LinAttnPass gq{}, gkp{}, gvp{};
  // dq_t = scale S_t do_t: forward in time on (do, v, k), the state transposed
  gq.x = dout, gq.a = v, gq.c = k, gq.out = dq;
  set3(gq.xs, so), set3(gq.as, sv), set3(gq.cs, sk), set3(gq.os, gk);
  gq.init = state0;
  gq.init_t = 1;
  gq.intra = gq.inter = d->scale;
  gq.upd = 1.f;
  // dk_t = dS_t v_t: reversed, on (v, do, q), the state transposed
  gkp.x = v, gkp.a = dout, gkp.c = q, gkp.out = dk;
  set3(gkp.xs, sv), set3(gkp.as, so), set3(gkp.cs, sq), set3(gkp.os, gk);
  gkp.init = dstateT;
  gkp.init_t = 1;
  gkp.reverse = 1;
  gkp.shift = 1;
  gkp.intra = gkp.upd = d->scale;
  gkp.inter = 1.f;
  // dv_t = dS_t^T k_t: reversed, on (k, q, do); its final state is dS_0
  gvp.x = k, gvp.a = q, gvp.c = dout, gvp.out = dv;
  set3(gvp.xs, sk), set3(gvp.as, sq), set3(gvp.cs, so), set3(gvp.os, gv);
  gvp.init = dstateT;
  gvp.fin = dstate0;
  gvp.reverse = 1;
  gvp.shift = 1;
  gvp.intra = gvp.upd = d->scale;
  gvp.inter = 1.f;
  const bool bf16 = d->dtype == RNN_BF16;
  p.pass[0] = gq;
  p.pass[1] = gkp;
  if (d->Dk == d->Dv) {
    p.pass[2] = gvp;
    p.npass = 3;
    return map_launch_error(run_passes(p, bf16, d->Dk, d->Dv, workspace, s));
  }
  p.npass = 2;
  e = run_passes(p, bf16, d->Dv, d->Dk, workspace, s);
  if (e != 0) return map_launch_error(e);
  p.pass[0] = gvp;
  p.npass = 1;
  p.clear = 0;  // what the first two passes reported stays
  return map_launch_error(run_passes(p, bf16, d->Dk, d->Dv, workspace, s));
}

int rnn_linattn_step(const rnn_linattn_desc_t* d, const rnn_linattn_strides_t* st, const void* q,
                     const void* k, const void* v, const float* log_decay, const int32_t* slots,
                     int32_t n_slots, float* state, void* o, void* stream) {
  int e = check_linattn(d);
  if (e != RNN_OK) return e;
  if (n_slots < 0 || d->T != 1 || d->flags != 0) return RNN_ERR_INVALID_ARG;
  if (d->B == 0 || d->NH == 0) return RNN_OK;
  if (slots == nullptr && n_slots < d->B) return RNN_ERR_INVALID_ARG;
  if (q == nullptr || k == nullptr || v == nullptr || log_decay == nullptr || o == nullptr ||
      (state == nullptr && n_slots > 0))
    return RNN_ERR_INVALID_ARG;
  const size_t es = dtype_bytes(d->dtype);
  const St sq = strides_or(st ? st->q : nullptr, d, d->Dk), sk = strides_or(st ? st->k : nullptr, d, d->Dk);
  const St sv = strides_or(st ? st->v : nullptr, d, d->Dv);
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) ||
      !aligned(state, 16) || !aligned(log_decay, 4) || !aligned(slots, 4) ||
      !strides_aligned(sq, es, 1) || !strides_aligned(sk, es, 1) || !strides_aligned(sv, es, 1))
    return RNN_ERR_MISALIGNED;
  LinAttnStepParams p{};
  p.q = q, p.k = k, p.v = v, p.o = o;
  p.state = state;
  p.log_decay = log_decay;
  p.slots = slots;
  for (int i = 0; i < 2; ++i) p.qs[i] = sq.s[i + 1], p.ks[i] = sk.s[i + 1], p.vs[i] = sv.s[i + 1];
  p.B = d->B, p.NH = d->NH, p.DK = d->Dk, p.DV = d->Dv;
  p.nslots = n_slots;
  p.scale = d->scale;
  return map_launch_error(
      launch_linattn_step(p, d->dtype == RNN_BF16, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
