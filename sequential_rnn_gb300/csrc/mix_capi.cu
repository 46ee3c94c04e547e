// C ABI of the gated linear recurrence, the norm and rotation of heads and the clipping of gradients (declared in
// include/rnn.h): argument checks, launches on the caller's stream.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>

#include "api.h"
#include "lm.h"

using namespace srnn;
using namespace srnn::api;

namespace {

bool valid_dtype(int32_t d) { return d == RNN_F32 || d == RNN_BF16; }
size_t dtype_bytes(int32_t d) { return d == RNN_F32 ? 4 : 2; }

int check_gated(const rnn_gated_desc_t* d) {
  if (d == nullptr || !valid_dtype(d->dtype)) return RNN_ERR_INVALID_ARG;
  if (d->T < 0 || d->B < 0 || d->NH < 0 || d->D <= 0) return RNN_ERR_INVALID_ARG;
  if (d->gates < RNN_GATES_FZ || d->gates > RNN_GATES_IFZO || (d->flags & ~RNN_FLAG_TEST_TIMEOUT) != 0)
    return RNN_ERR_INVALID_ARG;
  // tokens and channels are counted in 32 bits, up to a cluster's share past the end; a CTA for 32 channels
  const long long n = (long long)d->NH * d->D;
  if (d->T > (1 << 30) || n > (1 << 30) || (n + 31) / 32 * d->B > (1 << 27)) return RNN_ERR_UNSUPPORTED;
  return RNN_OK;
}
size_t stash_bytes(const rnn_gated_desc_t* d) {
  return (size_t)((d->T + kGatedRun - 1) / kGatedRun) * d->B * d->NH * d->D * sizeof(float);
}
int gated_status(int e) { return e == kGatedNoTile ? RNN_ERR_UNSUPPORTED : map_launch_error(e); }
GatedParams gated_params(const rnn_gated_desc_t* d, const void* Wx, const int32_t* lens, void* workspace) {
  GatedParams p{};
  p.status = static_cast<int*>(workspace);
  p.withhold = d->flags != 0;
  p.timeout_ns = d->flags != 0 ? kTestTimeoutNs : kTimeoutNs;
  p.wx = Wx;
  p.lens = lens;
  p.T = d->T, p.B = d->B, p.N = d->NH * d->D, p.D = d->D;
  return p;
}

int check_rotary(const rnn_rotary_desc_t* d) {
  if (d == nullptr || !valid_dtype(d->dtype)) return RNN_ERR_INVALID_ARG;
  if (d->T < 0 || d->B < 0 || d->NQ < 0 || d->NK < 0 || d->D <= 0 || d->rot < 0 || d->rot > d->D || !(d->eps >= 0.f) ||
      (d->flags & ~(RNN_ROTARY_INTERLEAVED | RNN_ROTARY_PER_TOKEN)) != 0)
    return RNN_ERR_INVALID_ARG;
  if (d->D % 2 != 0 || d->rot % 2 != 0 || d->D > 4096) return RNN_ERR_UNSUPPORTED;
  if ((long long)d->T * d->B > INT32_MAX || (long long)d->NQ + d->NK > (1 << 20)) return RNN_ERR_UNSUPPORTED;
  return RNN_OK;
}
bool set_strides(long long (&dst)[3], const int64_t* given, const rnn_rotary_desc_t* d, int heads) {
  if (given == nullptr) {
    dst[2] = d->D;
    dst[1] = (long long)heads * d->D;
    dst[0] = (long long)d->B * heads * d->D;
    return true;
  }
  for (int i = 0; i < 3; ++i) dst[i] = given[i];
  return dst[0] >= 0 && dst[1] >= 0 && dst[2] >= 0;
}
// what both directions check and set
int rotary_params(RotaryParams& p, const rnn_rotary_desc_t* d, const rnn_rotary_strides_t* st, const void* q,
                  const void* k, const float* qw, const float* kw, const double* freqs, const int32_t* positions,
                  void* qo, void* ko) {
  const bool any = d->T > 0 && d->B > 0;
  if (any && ((d->NQ > 0 && (q == nullptr || qo == nullptr)) || (d->NK > 0 && (k == nullptr || ko == nullptr))))
    return RNN_ERR_INVALID_ARG;
  if ((qw == nullptr) != (kw == nullptr) || (d->rot > 0 && freqs == nullptr)) return RNN_ERR_INVALID_ARG;
  if (positions == nullptr && (d->flags & RNN_ROTARY_PER_TOKEN) != 0) return RNN_ERR_INVALID_ARG;
  if (!set_strides(p.qs, st ? st->q : nullptr, d, d->NQ) || !set_strides(p.ks, st ? st->k : nullptr, d, d->NK))
    return RNN_ERR_INVALID_ARG;
  const size_t es = dtype_bytes(d->dtype);
  if (!aligned(q, es) || !aligned(k, es) || !aligned(qo, es) || !aligned(ko, es) || !aligned(qw, 4) || !aligned(kw, 4) ||
      !aligned(freqs, 8) || !aligned(positions, 4))
    return RNN_ERR_MISALIGNED;
  p.q = q, p.k = k, p.qw = qw, p.kw = kw, p.freqs = freqs, p.positions = positions;
  p.qo = qo, p.ko = ko;
  p.T = d->T, p.B = d->B, p.NQ = d->NQ, p.NK = d->NK, p.D = d->D, p.rot = d->rot;
  p.interleaved = (d->flags & RNN_ROTARY_INTERLEAVED) != 0;
  p.per_token = (d->flags & RNN_ROTARY_PER_TOKEN) != 0;
  p.eps = d->eps;
  return RNN_OK;
}

struct Span {
  uintptr_t at, end;
};

}  // namespace

extern "C" {

size_t rnn_gated_stash_size(const rnn_gated_desc_t* d) { return check_gated(d) == RNN_OK ? stash_bytes(d) : 0; }

int rnn_gated_fwd(const rnn_gated_desc_t* d, const void* Wx, const int32_t* lens, const float* state0, void* y,
                  float* stateT, float* stash, void* workspace, size_t workspace_bytes, void* stream) {
  const int e = check_gated(d);
  if (e != RNN_OK) return e;
  if (workspace == nullptr || workspace_bytes < kStatusBytes) return RNN_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return RNN_ERR_MISALIGNED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d->B == 0 || d->NH == 0) return clear_status(workspace, workspace_bytes, s);
  if (d->T > 0 && (Wx == nullptr || y == nullptr)) return RNN_ERR_INVALID_ARG;
  const size_t es = dtype_bytes(d->dtype);
  if (!aligned(Wx, es) || !aligned(y, es) || !aligned(lens, 4) || !aligned(state0, 4) || !aligned(stateT, 4) ||
      !aligned(stash, 4))
    return RNN_ERR_MISALIGNED;
  GatedParams p = gated_params(d, Wx, lens, workspace);
  if (d->flags != 0 && !gated_takes_tiles(p, d->dtype == RNN_BF16)) return RNN_ERR_UNSUPPORTED;
  p.state0 = state0, p.y = y, p.stateT = stateT, p.stash = stash;
  return gated_status(launch_gated(p, d->gates, d->dtype == RNN_BF16, false, s));
}

int rnn_gated_bwd(const rnn_gated_desc_t* d, const void* Wx, const int32_t* lens, const float* stash, const void* dy,
                  const float* dstateT, void* dWx, float* dstate0, void* workspace, size_t workspace_bytes,
                  void* stream) {
  const int e = check_gated(d);
  if (e != RNN_OK) return e;
  if (workspace == nullptr || workspace_bytes < kStatusBytes) return RNN_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return RNN_ERR_MISALIGNED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d->B == 0 || d->NH == 0) return clear_status(workspace, workspace_bytes, s);
  if (d->T > 0 && (Wx == nullptr || stash == nullptr || dy == nullptr || dWx == nullptr)) return RNN_ERR_INVALID_ARG;
  const size_t es = dtype_bytes(d->dtype);
  if (!aligned(Wx, es) || !aligned(dy, es) || !aligned(dWx, es) || !aligned(lens, 4) || !aligned(stash, 4) ||
      !aligned(dstateT, 4) || !aligned(dstate0, 4))
    return RNN_ERR_MISALIGNED;
  GatedParams p = gated_params(d, Wx, lens, workspace);
  if (d->flags != 0 && !gated_takes_tiles(p, d->dtype == RNN_BF16)) return RNN_ERR_UNSUPPORTED;
  p.stash = const_cast<float*>(stash), p.dy = dy, p.dstateT = dstateT, p.dwx = dWx, p.dstate0 = dstate0;
  return gated_status(launch_gated(p, d->gates, d->dtype == RNN_BF16, true, s));
}

int rnn_gated_config(const rnn_gated_desc_t* d, int32_t gradient, int32_t* out7) {
  const int e = check_gated(d);
  if (e != RNN_OK) return e;
  if (out7 == nullptr) return RNN_ERR_INVALID_ARG;
  for (int i = 0; i < 7; ++i) out7[i] = 0;
  if (d->B == 0 || d->NH == 0) return RNN_OK;
  GatedInfo info{};
  const GatedParams p = gated_params(d, nullptr, nullptr, nullptr);
  const int err = launch_gated(p, d->gates, d->dtype == RNN_BF16, gradient != 0, nullptr, &info);
  if (err != 0) return map_launch_error(err);
  const int32_t out[7] = {info.grid, info.threads, info.cluster, info.tile, info.ahead, info.smem, info.held};
  std::copy(out, out + 7, out7);
  return RNN_OK;
}

int rnn_gated_step(const rnn_gated_desc_t* d, const void* Wx, const int32_t* slots, int32_t n_slots, float* state,
                   void* y, void* stream) {
  const int e = check_gated(d);
  if (e != RNN_OK) return e;
  if (n_slots < 0 || d->T != 1 || d->flags != 0) return RNN_ERR_INVALID_ARG;
  if (d->B == 0 || d->NH == 0) return RNN_OK;
  if (slots == nullptr && n_slots < d->B) return RNN_ERR_INVALID_ARG;
  if (Wx == nullptr || y == nullptr || (state == nullptr && n_slots > 0)) return RNN_ERR_INVALID_ARG;
  const size_t es = dtype_bytes(d->dtype);
  if (!aligned(Wx, es) || !aligned(y, es) || !aligned(state, 4) || !aligned(slots, 4)) return RNN_ERR_MISALIGNED;
  const GatedStepParams p{Wx, slots, state, y, d->B, d->NH * d->D, d->D, n_slots};
  return map_launch_error(launch_gated_step(p, d->gates, d->dtype == RNN_BF16, static_cast<cudaStream_t>(stream)));
}

int rnn_head_norm_rotary(const rnn_rotary_desc_t* d, const rnn_rotary_strides_t* st, const void* q, const void* k,
                         const float* q_weight, const float* k_weight, const double* freqs, const int32_t* positions,
                         void* q_out, void* k_out, void* stream) {
  int e = check_rotary(d);
  if (e != RNN_OK) return e;
  RotaryParams p{};
  if ((e = rotary_params(p, d, st, q, k, q_weight, k_weight, freqs, positions, q_out, k_out)) != RNN_OK) return e;
  if (d->T == 0 || d->B == 0 || d->NQ + d->NK == 0) return RNN_OK;
  return map_launch_error(launch_rotary(p, d->dtype == RNN_BF16, false, static_cast<cudaStream_t>(stream)));
}

size_t rnn_head_norm_rotary_bwd_workspace_size(const rnn_rotary_desc_t* d) {
  return check_rotary(d) == RNN_OK ? align_up((size_t)kRotaryParts * 2 * d->D * sizeof(float), 256) : 0;
}

int rnn_head_norm_rotary_bwd(const rnn_rotary_desc_t* d, const rnn_rotary_strides_t* st, const void* q,
                             const void* k, const float* q_weight, const float* k_weight, const double* freqs,
                             const int32_t* positions, const void* dq_out, const void* dk_out, void* dq, void* dk,
                             float* dq_weight, float* dk_weight, void* workspace, size_t workspace_bytes,
                             void* stream) {
  int e = check_rotary(d);
  if (e != RNN_OK) return e;
  RotaryParams p{};
  if ((e = rotary_params(p, d, st, q, k, q_weight, k_weight, freqs, positions, dq, dk)) != RNN_OK) return e;
  const bool any = d->T > 0 && d->B > 0;
  if (any && ((d->NQ > 0 && dq_out == nullptr) || (d->NK > 0 && dk_out == nullptr))) return RNN_ERR_INVALID_ARG;
  if (!set_strides(p.dqs, st ? st->dq : nullptr, d, d->NQ) || !set_strides(p.dks, st ? st->dk : nullptr, d, d->NK))
    return RNN_ERR_INVALID_ARG;
  if (q_weight != nullptr && (dq_weight == nullptr || dk_weight == nullptr || workspace == nullptr ||
                              workspace_bytes < rnn_head_norm_rotary_bwd_workspace_size(d)))
    return RNN_ERR_INVALID_ARG;
  const size_t es = dtype_bytes(d->dtype);
  if (!aligned(dq_out, es) || !aligned(dk_out, es) || !aligned(dq_weight, 4) || !aligned(dk_weight, 4) ||
      !aligned(workspace, 256))
    return RNN_ERR_MISALIGNED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!any || d->NQ + d->NK == 0) {
    if (q_weight == nullptr) return RNN_OK;
    const size_t n = (size_t)d->D * sizeof(float);
    return cudaMemsetAsync(dq_weight, 0, n, s) == cudaSuccess && cudaMemsetAsync(dk_weight, 0, n, s) == cudaSuccess
               ? RNN_OK
               : RNN_ERR_LAUNCH;
  }
  p.dq = dq_out, p.dk = dk_out, p.dqw = dq_weight, p.dkw = dk_weight;
  p.part = static_cast<float*>(workspace);
  return map_launch_error(launch_rotary(p, d->dtype == RNN_BF16, true, s));
}

size_t rnn_clip_grad_norm_workspace_size(int32_t n) {
  return n < 0 || n > kClipMost ? 0 : align_up((size_t)clip_parts(n) * sizeof(double), 256);
}

int rnn_clip_grad_norm(int32_t n, const int32_t* dtypes, const int64_t* sizes, void* const* tensors, float max_norm,
                       float* norm, void* workspace, size_t workspace_bytes, void* stream) {
  if (n < 0 || !(max_norm >= 0.f)) return RNN_ERR_INVALID_ARG;
  if (n > kClipMost) return RNN_ERR_UNSUPPORTED;
  if (n > 0 && (dtypes == nullptr || sizes == nullptr || tensors == nullptr)) return RNN_ERR_INVALID_ARG;
  bool rising = true;
  uintptr_t end = 0;
  int64_t units = 0;
  for (int32_t i = 0; i < n; ++i) {
    if (!valid_dtype(dtypes[i]) || sizes[i] < 0) return RNN_ERR_INVALID_ARG;
    if (sizes[i] > (int64_t)1 << 40) return RNN_ERR_UNSUPPORTED;
    if (sizes[i] == 0) continue;
    // (the same tensor may come more than once, so that the device's memory is no bound)
    units += clip_units(sizes[i], dtypes[i]);
    if (units > INT32_MAX) return RNN_ERR_UNSUPPORTED;
    if (tensors[i] == nullptr) return RNN_ERR_INVALID_ARG;
    if (!aligned(tensors[i], dtype_bytes(dtypes[i]))) return RNN_ERR_MISALIGNED;
    const uintptr_t at = reinterpret_cast<uintptr_t>(tensors[i]);
    rising = rising && at >= end;
    end = at + (uintptr_t)sizes[i] * dtype_bytes(dtypes[i]);
  }
  if (workspace == nullptr || workspace_bytes < rnn_clip_grad_norm_workspace_size(n)) return RNN_ERR_INVALID_ARG;
  if (!aligned(workspace, 256) || !aligned(norm, 4)) return RNN_ERR_MISALIGNED;
  if (!rising && std::isfinite(max_norm)) {  // not in the order of their addresses: sorted to see that none overlap
    Span* spans = new (std::nothrow) Span[n];
    if (spans == nullptr) return RNN_ERR_LAUNCH;
    int m = 0;
    for (int32_t i = 0; i < n; ++i) {
      const uintptr_t at = reinterpret_cast<uintptr_t>(tensors[i]);
      if (sizes[i] > 0) spans[m++] = Span{at, at + (uintptr_t)sizes[i] * dtype_bytes(dtypes[i])};
    }
    std::sort(spans, spans + m, [](const Span& a, const Span& b) { return a.at < b.at; });
    bool apart = true;
    for (int i = 1; i < m; ++i) apart = apart && spans[i].at >= spans[i - 1].end;
    delete[] spans;
    if (!apart) return RNN_ERR_INVALID_ARG;
  }
  const ClipParams p{tensors, sizes, dtypes, n, max_norm, norm, static_cast<double*>(workspace)};
  return map_launch_error(launch_clip(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
