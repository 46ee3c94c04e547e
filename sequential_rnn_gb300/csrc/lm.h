// Internal interface of the language-model operators: the root-mean-square
// norm, the 8-bit projection and the linear attention with a decay per head
// (entry points and argument checks in lm_capi.cu); the gated linear recurrence, the
// norm and rotation of heads and the clipping of gradients (mix_capi.cu).
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace srnn {

// Launch of a kernel that may begin while the one in front of it on the stream still runs (its start-up then
// overlaps that one's end) and that waits for the whole of it at depend_wait().  Two uses:
// - inside a call, before it touches what the call's kernel in front writes; that one says depend_launch() once
//   everything before the call has ended (where it was itself launched so, after its own depend_wait());
// - as a call's first kernel, whatever is in front: every one of its CTAs waits before its first access, so that
//   "the kernel in front has ended" goes on meaning that everything before that one has.
// No non-coherent load (__ldg, const __restrict__) in such a kernel: its inputs may be written after it began.
template <class... P, class... A>
int launch_dependent(void (*kern)(P...), unsigned grid, unsigned threads, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return (int)cudaLaunchKernelEx(&cfg, kern, args...);
}
#ifdef __CUDACC__
__device__ __forceinline__ void depend_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void depend_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
#endif

// ------------------------------------------------------------------ norm --
struct NormParams {
  const void* x;
  const void* residual;  // or null
  const float* weight;
  void* h;               // x + residual, or null
  void* y;               // input type, or e4m3 when scale is set
  float* scale;          // [rows, ceil(N / 128)] or null
  float* rstd;           // [rows] or null
  long long rows;
  int N;
  float eps;
};
struct NormBwdParams {
  const void* dy;
  const void* h;
  const float* weight;
  const float* rstd;
  const void* dh;  // or null
  void* dx;
  float* dw;       // or null
  float* part;     // [norm_bwd_ctas, N] partial sums of dw (workspace)
  long long rows;
  int N;
};
// each returns a cudaError_t value
int launch_rms_norm(const NormParams& p, bool bf16, cudaStream_t s);
int launch_rms_norm_bwd(const NormBwdParams& p, bool bf16, cudaStream_t s);
// partial rows of dw launch_rms_norm_bwd may write (an upper bound that depends on the sizes alone)
int norm_bwd_parts(long long rows, int N);
int launch_quantize_weight(const void* W, bool bf16, int N, int K, void* Wq, float* Ws,
                           cudaStream_t s);

// ------------------------------------------------------------ projection --
struct ProjFp8Params {
  const void* xq;
  const float* xs;
  const void* Wq;
  const float* Ws;
  const float* bias;  // or null
  void* y;
  int M, N, K;
  int* status;
  unsigned long long timeout_ns;
};
int launch_proj_fp8(const ProjFp8Params& p, cudaStream_t s);

// ------------------------------------------------------ linear attention --
// One pass of the chunked recurrence over tokens r = 0, 1, .. of each row,
//   S_r = lambda S_{r-1} + upd a_r c_r^T,
//   out_r = intra sum_{j<=r} lambda^(r-j) (x_r . a_j) c_j
//           + inter lambda^(r+1-shift) x_r S_init ...,
// with x, a [.., DK], c, out [.., DV].  The forward takes (x, a, c) = (q, k, v);
// the gradients are three more passes of it (see linattn.cu).
struct LinAttnPass {
  const void* x;
  const void* a;
  const void* c;
  void* out;
  const float* init;  // [B, NH, DK, DV] (or its transpose), or null (zero)
  float* fin;         // the same, or null
  long long xs[3], as[3], cs[3], os[3];  // strides in elements: token, row, head
  int init_t;         // init is stored [DV, DK]
  int reverse;        // r = 0 is the row's last token
  float intra, inter, upd;
  int shift;          // 0 forward in time, 1 reversed (see above)
};
constexpr int kLinAttnPasses = 3;
struct LinAttnParams {
  LinAttnPass pass[kLinAttnPasses];
  int npass;
  const float* log_decay;  // [NH]
  const int* lens;         // [B] or null
  int T, B, NH, DK, DV;
  float* ws;               // segment states
  int nseg, seg_chunks;    // segments of the token axis, chunks in each
  void* chunk_states;      // bf16 [pass][head of a row][chunk][DK][DV] (kLinAttnTc)
  int* status;
  int clear;               // clear the status word (the first launch of a call)
  int withhold;            // test: an arrival of each kernel's first wait for compute warps is left out (kLinAttnTc)
  unsigned long long timeout_ns;
};
enum : int { kLinAttnF32 = 0, kLinAttnMma = 1, kLinAttnTc = 2 };
struct LinAttnPlan {
  int path;
  int nseg, seg_chunks;
  size_t seg_bytes;    // segment states
  size_t chunk_bytes;  // chunk states (kLinAttnTc)
};
LinAttnPlan linattn_plan(bool bf16, int npass, int T, int B, int NH, int DK, int DV);
int launch_linattn_mma(const LinAttnParams& p, cudaStream_t s);
// kLinAttnTooWide: the operands' strides or the sizes have no tensor map
constexpr int kLinAttnTooWide = -2;
int launch_linattn_tc(const LinAttnParams& p, cudaStream_t s);
int launch_linattn_f32(const LinAttnParams& p, cudaStream_t s);

struct LinAttnStepParams {
  const void* q;
  const void* k;
  const void* v;
  void* o;
  float* state;            // [slots, NH, DK, DV]
  const float* log_decay;
  const int* slots;        // [B] or null
  long long qs[2], ks[2], vs[2];  // strides in elements: row, head
  int B, NH, DK, DV, nslots;
  float scale;
};
int launch_linattn_step(const LinAttnStepParams& p, bool bf16, cudaStream_t s);

// ------------------------------------------- gated linear recurrence --
constexpr int kGatedRun = 8;  // tokens that share a state of the stash
struct GatedParams {
  const void* wx;       // [T, B, NH, gates D]
  const int* lens;      // [B] or null
  const float* state0;  // [B, N] or null
  void* y;              // [T, B, N]
  float* stateT;        // or null
  float* stash;         // [ceil(T / kGatedRun), B, N] states before every run of tokens (forward: or null)
  const void* dy;       // gradient alone: [T, B, N]
  const float* dstateT; // or null
  void* dwx;
  float* dstate0;       // or null
  int T, B, N, D;       // N = NH D
  int tiles, cs;        // (launch) channel tiles of a row, CTAs of a cluster along time
  int* status;
  int withhold;         // test: no tile is brought (tile kernels)
  unsigned long long timeout_ns;
};
struct GatedInfo {  // of a launch
  int grid, threads, cluster;
  int tile;  // channels of a tile that TMA brings; 0: the kernels without
  int ahead; // maps are made a round ahead
  int smem;
  int held;   // clusters (cluster 1: CTAs) of it that the device holds at once
};
// info: filled in the place of a launch (addresses are taken as aligned); a cudaError_t value, or kGatedNoTile where no tile can
// be withheld
int launch_gated(GatedParams p, int gates, bool bf16, bool bwd, cudaStream_t s, GatedInfo* info = nullptr);
// the kernels on tiles: whether the sizes suit them; kGatedNoTile: addresses or strides have no tensor map
constexpr int kGatedTileTokens = 65;
constexpr int kGatedNoTile = -2;
bool gated_takes_tiles(const GatedParams& p, bool bf16);
int launch_gated_tile(const GatedParams& p, int gates, bool bf16, bool bwd, cudaStream_t s, GatedInfo* info);
struct GatedStepParams {
  const void* wx;    // [B, NH, gates D]
  const int* slots;  // [B] or null
  float* state;      // [nslots, N]
  void* y;           // [B, N]
  int B, N, D, nslots;
};
int launch_gated_step(const GatedStepParams& p, int gates, bool bf16, cudaStream_t s);

// ------------------------------------------ norm and rotation of heads --
constexpr int kRotaryParts = 608;  // partial sums of the weights' gradients: 4 x 152 SMs
struct RotaryParams {
  const void* q;
  const void* k;
  const float* qw;       // [D]; null (both): no norm
  const float* kw;
  const double* freqs;   // [rot / 2]
  const int* positions;  // [B] (of the first token) or, per_token, [T, B]; null: 0
  void* qo;              // [T, B, NQ, D] (gradient: of q)
  void* ko;
  const void* dq;        // gradient alone: of the outputs
  const void* dk;
  float* dqw;
  float* dkw;
  float* part;           // [kRotaryParts, 2, D]
  long long qs[3], ks[3], dqs[3], dks[3];  // strides in elements: token, row, head
  int T, B, NQ, NK, D, rot, interleaved, per_token, split, ctas_q;
  float eps;
};
int launch_rotary(RotaryParams p, bool bf16, bool bwd, cudaStream_t s);

// ------------------------------------------------------------ clipping --
constexpr int kClipTensors = 256;  // of a launch: their table is a kernel parameter
constexpr int kClipUnit = 16384;   // bytes
constexpr int kClipMost = 1 << 28; // tensors of a call: its partial sums are counted in 32 bits
inline int64_t clip_units(int64_t size, int dtype) {  // of a tensor; dtype 1: bf16
  const int64_t per = kClipUnit / (dtype == 1 ? 2 : 4);
  return (size + per - 1) / per;
}
struct ClipParams {
  void* const* at;
  const int64_t* sizes;
  const int32_t* dtypes;  // 1: bf16
  int n;
  float limit;   // infinite: the norm alone
  float* norm;   // or null
  double* part;  // clip_parts(n) partial sums: of every launch's CTAs
};
int clip_parts(int n);
int launch_clip(const ClipParams& p, cudaStream_t s);

}  // namespace srnn
