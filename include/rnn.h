/*
 * sequential_rnn_gb300 -- C ABI of the head-wise RNN recurrence on GB300 (sm_103a).
 *
 * What is computed (FlashRNN pages: "FlashRNN: I/O-Aware Optimization of
 * Traditional RNNs on modern hardware", abstract -- LSTM, GRU and sLSTM
 * processed as many small heads; blog page "re-examining RNNs from a GPU
 * programming perspective", register-caching and head-wise paragraphs -- the
 * recurrent matrix R stays on chip across the time loop, heads form a
 * block-diagonal R and map to separate thread blocks):
 *
 *   for each head h, batch row b, step t = 0..T-1:
 *     pre_t = Wx[t,b,h,:] + h_{t-1}[b,h,:] @ R[h] + bias[h]        (row vectors)
 *     cell update (below) -> h_t, c_t (, n_t, m_t)
 *
 *   LSTM  gates (i,f,z,o): i,f,o = sigmoid, z = tanh; c = f*c + i*z; h = o*tanh(c)
 *   GRU   gates (r,z,n):   rec = h_{t-1}@R + bias; r = sigm(Wx_r+rec_r);
 *                          z = sigm(Wx_z+rec_z); n = tanh(Wx_n + r*rec_n);
 *                          h = (1-z)*n + z*h_{t-1}
 *   sLSTM gates (i,f,z,o): m_t = max(f~+m, i~); i = exp(i~-m_t); f = exp(f~+m-m_t);
 *                          c = f*c + i*tanh(z~); n = f*n + i; h = sigm(o~)*c/n
 *
 * Layouts (all row-major, contiguous; G = 4 for LSTM/sLSTM, 3 for GRU):
 *   Wx     [T, B, NH, G*Dh]  input dtype     gate-major: column g*Dh + j = gate g, unit j
 *   R      [NH, Dh, G*Dh]    input dtype
 *   bias   [NH, G*Dh]        fp32            (NULL = zeros)
 *   h0,c0,n0,m0 [B, NH, Dh]  fp32            (NULL = zeros; c0 unused by GRU, n0/m0 sLSTM only)
 *   h_seq  [T, B, NH, Dh]    input dtype     h_t for every step (bf16: rounded to nearest even)
 *   hT,cT,nT,mT [B, NH, Dh]  fp32            final states (NULL = not written)
 *
 * Numerics: RNN_F32 computes in fp32 throughout (fp32 FMA contraction,
 * accurate exp/tanh).  RNN_BF16 feeds bf16(h_{t-1}) and bf16 R to the tensor
 * cores with fp32 accumulation; gate math and all states are fp32 (LSTM/GRU
 * gates on the hardware tanh).  For the sLSTM, whose exponential gating
 * amplifies per-step rounding of h by ~10^3 over 4096 steps, h_{t-1} enters
 * the tensor cores as a bf16 pair hi + lo (hi = bf16(h), lo = bf16(h - hi),
 * both products accumulated in fp32; with B <= 4 the two halves share one
 * MMA tile) and tanh(z~) is evaluated as 1 - 2/(e^{2z~}+1) on the
 * 2-ulp exponential instead of the ~2^-11 hardware tanh, for Dh <= 256
 * (Dh = 768 runs the plain bf16 operand: the pair does not fit on chip beside
 * R); RNN_FLAG_H_BF16 turns this off.  With the plain operand the deviation
 * from the exact recurrence grows about linearly with T (~1.5e-5 per step on
 * R ~ U(+-1/sqrt(768)) inputs, fp64 emulation), so an sLSTM with Dh = 768 and
 * T > 768 is rejected with RNN_ERR_UNSUPPORTED unless RNN_FLAG_H_BF16 is set
 * (the caller accepts the plain operand's drift).
 *
 * Ownership: the caller allocates and owns every buffer (device memory),
 * including the workspace and the training stash.  Nothing is allocated by
 * the library.  All calls are asynchronous on `stream` (a cudaStream_t,
 * NULL = legacy default stream).  Host-side checks fail fast with a status
 * and launch nothing.  Device-side failures (a bounded wait that ran out) are
 * recorded in the status word at the start of the workspace; read it with
 * rnn_read_status().  Every call that returns RNN_OK with a workspace leaves
 * its own status there -- 0 also for a call that launches nothing (B, NH or
 * T zero) -- so the workspace needs no clearing by the caller.
 */
#ifndef SEQUENTIAL_RNN_GB300_RNN_H
#define SEQUENTIAL_RNN_GB300_RNN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { RNN_LSTM = 0, RNN_GRU = 1, RNN_SLSTM = 2 } rnn_cell_t;
typedef enum { RNN_F32 = 0, RNN_BF16 = 1 } rnn_dtype_t;

/* desc.flags */
enum {
  RNN_FLAG_TRAIN = 1,              /* forward also writes the stash rnn_bwd needs */
  RNN_FLAG_H_BF16 = 2,             /* sLSTM: plain bf16 h operand and fast gate math
                                      (default for sLSTM is the hi+lo split, see Numerics) */
  RNN_FLAG_TEST_TIMEOUT = 1 << 30  /* test only: the kernel waits on a barrier that nothing
                                      completes, gives up after ~50 ms and reports
                                      RNN_ERR_TIMEOUT in the status word */
};

typedef struct {
  int32_t cell;    /* rnn_cell_t */
  int32_t dtype;   /* rnn_dtype_t: type of Wx, R, h_seq, dh_seq, dWx */
  int32_t T, B, NH, Dh;
  int32_t flags;   /* RNN_FLAG_* */
  int32_t cluster; /* 0 = automatic; else CTAs per head for bf16 (1,2,4,8,16) */
} rnn_desc_t;

typedef enum {
  RNN_OK = 0,
  RNN_ERR_INVALID_ARG = 1, /* null pointer, negative size, bad enum, small workspace */
  RNN_ERR_UNSUPPORTED = 2, /* shape/dtype/cell combination without a kernel */
  RNN_ERR_MISALIGNED = 3,  /* a pointer violates the alignment stated below */
  RNN_ERR_LAUNCH = 4,      /* the CUDA launch itself failed */
  RNN_ERR_TIMEOUT = 5,     /* device status: a bounded wait ran out, outputs invalid */
  RNN_ERR_NO_CLUSTER = 6,  /* the device cannot co-schedule the needed thread-block cluster */
  RNN_ERR_SCRATCH_LIMIT = 7, /* rnn_fwd_noalloc: the call needs more scratch than its array holds */
  RNN_ERR_BOUNDS = 8         /* device status, bounds-check builds only (libsrnn_bc.so, compiled with
                                -DRNN_BOUNDS_CHECK): a kernel index fell outside its buffer; the
                                access was skipped, outputs invalid */
} rnn_status_t;

/* Bytes of device workspace rnn_fwd (pass 0) / rnn_bwd (pass 1) need.
 * Always >= 256 (the status word lives at offset 0).  0 on invalid desc. */
size_t rnn_workspace_size(const rnn_desc_t* desc, int pass);

/* Bytes of the training stash rnn_fwd writes with RNN_FLAG_TRAIN (bf16 only):
 * four gate values fp32 [T,B,NH,4*Dh], then one state fp32 [T,B,NH,Dh] (LSTM c_t,
 * GRU h_t), then for the sLSTM n_t [T,B,NH,Dh].  Opaque to the caller; pass the
 * same buffer to rnn_bwd. */
size_t rnn_stash_size(const rnn_desc_t* desc);

/* Forward recurrence.  Alignment: Wx, R, h_seq, stash 16 bytes; fp32
 * pointers 4 bytes.  Supported: RNN_F32 with Dh in {16,32,64};
 * RNN_BF16 with Dh in {32,64,128,256,768} (Dh > 128 runs as a thread-block
 * cluster per head).  T == 0 copies the initial states to the final ones;
 * B == 0 or NH == 0 is a no-op.  Returns rnn_status_t. */
int rnn_fwd(const rnn_desc_t* desc, const void* Wx, const void* R, const float* bias,
            const float* h0, const float* c0, const float* n0, const float* m0, void* h_seq,
            float* hT, float* cT, float* nT, float* mT, void* stash, void* workspace,
            size_t workspace_bytes, void* stream);

/* Backward through time (RNN_BF16; LSTM, GRU or sLSTM; Dh in {32,64,128,256,768}),
 * from the stash of a RNN_FLAG_TRAIN forward with the same desc, inputs and
 * h_seq.  Gradients of L = sum(h_seq*dh_seq) + sum(hT*dhT) + sum(cT*dcT) + sum(nT*dnT):
 *   dWx [T,B,NH,G*Dh] input dtype,
 *   dR [NH,Dh,G*Dh] fp32 = sum_t h_{t-1}^T dG_t (h_{-1} = h0 as bf16; dG the
 *      gradient of the recurrent preactivation h@R+b, = dWx except the GRU n block),
 *   db [NH,G*Dh] fp32 = sum_t dG_t, dh0, dc0, dn0 [B,NH,Dh] fp32
 *   (dc0: LSTM/sLSTM, dn0: sLSTM; each of dR/db/dh0/dc0/dn0 may be NULL).
 * h0, c0, n0: the forward's initial states (NULL = zeros).  dhT, dcT, dnT: upstream
 * gradients of the final states (NULL = zero).  The sLSTM stabiliser m is held at
 * its forward values and carries no gradient: exact for any loss of h (h does not
 * depend on m); the dcT, dnT terms are differentiated with m_T held fixed, so
 * that the backward of consecutive time chunks, each fed the next chunk's
 * dh0/dc0/dn0 as dhT/dcT/dnT, composes to the whole sequence's.  dh_seq: input dtype.  Alignment:
 * R, h_seq, dh_seq, dWx, stash 16 bytes; fp32 pointers 8 bytes; workspace 256.
 * The reverse recurrence runs as one thread-block cluster per head slice (as the
 * forward), then the dR contraction (tcgen05 tensor cores) and the db reduction. */
int rnn_bwd(const rnn_desc_t* desc, const void* R, const float* h0, const float* c0,
            const float* n0, const void* h_seq, const void* stash, const void* dh_seq,
            const float* dhT, const float* dcT, const float* dnT, void* dWx, float* dR, float* db,
            float* dh0, float* dc0, float* dn0, void* workspace, size_t workspace_bytes,
            void* stream);

/* rnn_fwd for a sequence in (pinned) host memory: Wx_host [T, B, NH, G*Dh] is
 * read from and h_seq_host [T, B, NH, Dh] written to host memory while the
 * recurrence runs.  Time is cut into chunks of `chunk` steps (0 = automatic:
 * T/8, at least 64 -- or, for bf16 runs that consume Wx at under ~64 GB/s by
 * the plan's step time and pinned, mapped host buffers, the RNN_HOST_DIRECT
 * mode below); chunk c's Wx is copied in on a copy stream while chunk
 * c-1 runs, and chunk c-1's h_seq is copied out on another, so only the first
 * chunk's upload and the last chunk's download are not hidden behind the
 * recurrence.  Each chunk continues from the previous chunk's final state,
 * which gives results identical to one rnn_fwd over all T steps.  R, bias,
 * the initial and final states and the workspace are device memory (as for
 * rnn_fwd); no RNN_FLAG_TRAIN.  The copy streams and events are created on a
 * device's first call and kept (host resources); the enqueue is serialised
 * across host threads; `stream` waits for all of it.  Alignment: R 16 bytes,
 * fp32 pointers 4, workspace 256 and >= rnn_fwd_host_workspace_size() bytes
 * (status word at offset 0, then two Wx chunks, two h_seq chunks and the
 * carried states).  Host memory that is not pinned still works, without the
 * overlap.
 *
 * chunk = RNN_HOST_DIRECT: no staging copies; one rnn_fwd whose kernel reads
 * Wx_host and writes h_seq_host through their device mapping (page-locked host
 * memory on a unified-addressing system, reached over the CPU-GPU link; on
 * Grace-Blackwell NVLink-C2C).  Both buffers must be page-locked and mapped
 * (cudaHostAlloc / cudaMallocHost, or cudaHostRegister with mapping), else
 * RNN_ERR_INVALID_ARG; alignment as for rnn_fwd (16 bytes); workspace as for
 * rnn_fwd. */
#define RNN_HOST_DIRECT (-1)
size_t rnn_fwd_host_workspace_size(const rnn_desc_t* desc, int32_t chunk);
int rnn_fwd_host(const rnn_desc_t* desc, int32_t chunk, const void* Wx_host, const void* R,
                 const float* bias, const float* h0, const float* c0, const float* n0,
                 const float* m0, void* h_seq_host, float* hT, float* cT, float* nT, float* mT,
                 void* workspace, size_t workspace_bytes, void* stream);

/* Input projection, the dense step in front of the recurrence (FlashRNN blog
 * page, register-caching paragraph: only the recurrent weight R has to stay on
 * chip through the sequential time loop; the input weight is applied to all
 * steps at once):
 *   Wx[m, n] = sum_k x[m, k] * W[n, k] + bias[n]
 * x [M, K] bf16 (M = T*B rows of the input sequence), W [N, K] bf16 (rows are
 * output features, as in a linear layer's weight), bias [N] fp32 (NULL = none),
 * Wx [M, N] bf16 (fp32 sum rounded to nearest even once).  With N = NH*G*Dh,
 * Wx is rnn_fwd's input.  fp32 accumulation on the tensor cores (tcgen05, TMA).
 * Requires K % 8 == 0, N % 16 == 0, M <= 8388480.  Alignment: x, W, Wx 16 bytes,
 * bias 4 bytes, workspace 256 bytes and >= 256 bytes (status word at offset 0).
 * M == 0 is a no-op.  Returns rnn_status_t. */
int rnn_input_proj(int32_t M, int32_t N, int32_t K, const void* x, const void* W,
                   const float* bias, void* Wx, void* workspace, size_t workspace_bytes,
                   void* stream);

/* Stacked layers run as a wavefront (FlashRNN blog page, paragraph on cuDNN
 * and layer-level parallelism: layer l+1 can work on step t once layer l has
 * produced h_t).  L layers of one cell and head shape (desc: RNN_BF16, no
 * RNN_FLAG_TRAIN); layer 0 reads x, layer l > 0 reads layer l-1's h_seq; per
 * layer Wx = in W^T + b_ih (as rnn_input_proj) feeds the recurrence.  Time is
 * cut into chunks of `chunk` steps: layer l runs chunk c (its input projection,
 * then the recurrence continuing from chunk c-1's final state) once layer l-1
 * has finished chunk c, each layer on its own stream, so up to L layers run at
 * once.  The result equals running the layers one after the other.
 * Layouts (d = NH*Dh; the G*d projection rows are ordered [NH, G*Dh] like Wx):
 *   x [T, B, Din] bf16;  W_ih0 [G*d, Din] bf16;  W_ih [L-1, G*d, d] bf16 (NULL if
 *   L == 1);  b_ih [L, G*d] fp32 (NULL = 0);  R [L, NH, Dh, G*Dh] bf16;
 *   bias [L, NH, G*Dh] fp32 (NULL = 0);  h0, c0, n0, m0 [L, B, NH, Dh] fp32
 *   (NULL = 0);  h_seq [T, B, NH, Dh] bf16 (last layer);  hT, cT, nT, mT
 *   [L, B, NH, Dh] fp32 (NULL = not written).
 * chunk 0 = chosen by the plan search (rnn_plan), as are the CTAs per head when
 * desc->cluster is 0 (so that the layers' recurrences fit the SMs together).
 * Requires 1 <= L <= 8, chunk >= 0, Din % 8 == 0.  Alignment: bf16 arrays 16
 * bytes, fp32 arrays 4, workspace 256 bytes and >= rnn_stack_workspace_size()
 * (status word at offset 0, then the layers' intermediate h_seq, Wx chunks and
 * carried states).  The per-layer streams and events are created on a device's
 * first call and kept (host resources, no device memory); the enqueue is
 * serialised across host threads.  `stream` waits for all of the work. */
size_t rnn_stack_workspace_size(const rnn_desc_t* desc, int32_t L, int32_t chunk);
int rnn_stack_fwd(const rnn_desc_t* desc, int32_t L, int32_t Din, int32_t chunk, const void* x,
                  const void* W_ih0, const void* W_ih, const float* b_ih, const void* R,
                  const float* bias, const float* h0, const float* c0, const float* n0,
                  const float* m0, void* h_seq, float* hT, float* cT, float* nT, float* mT,
                  void* workspace, size_t workspace_bytes, void* stream);

/* The launch plan the library picks when desc->cluster is 0: an integer search
 * over CTAs per head (1, 2, 4, 8, 16) -- and for L > 1 stacked layers the time
 * chunk -- in the spirit of the FlashRNN card's ConstrINT (hardware limits as
 * integer constraints with divisibility).  A candidate must split the head into
 * whole unit groups of a warp, fit the compiled variant's register budget and
 * shared memory, and (clusters) at most 16 CTAs; the cost is the per-step time
 * (measured on GB300 per cell, Dh and CTAs per head; a latency model where not
 * measured) times the waves the CTAs need over `sms` SMs, and for L > 1 the
 * wavefront's stages given how many layers fit on the SMs at once.
 * sms <= 0: the current device's SM count.  out5[0..4] = CTAs per head, time
 * chunk (T for one layer), CTAs per layer, waves, predicted microseconds.
 * RNN_BF16 only.  Host computation (no launch). */
int rnn_plan(const rnn_desc_t* desc, int32_t L, int32_t sms, int32_t* out5);

/* Synchronises `stream`, reads the device status word of `workspace` into
 * *device_status (RNN_OK, RNN_ERR_TIMEOUT, or in bounds-check builds
 * RNN_ERR_BOUNDS; a timeout is reported first).  Returns RNN_OK if the read
 * itself worked, else RNN_ERR_LAUNCH. */
int rnn_read_status(const void* workspace, void* stream, int* device_status);

/* Measurement aid: runs `iters` iterations of only the per-step
 * synchronisation of the rnn_fwd launch `desc` selects (same grid, cluster
 * shape and barrier kind, no loads and no math).  Its time / iters is the
 * sync floor of one step. */
int rnn_sync_floor(const rnn_desc_t* desc, int iters, void* workspace, size_t workspace_bytes,
                   void* stream);

/* Launch geometry rnn_fwd would use: out[0..5] = grid CTAs, threads per CTA,
 * cluster size, batch rows per CTA, dynamic smem bytes, kernel id. */
int rnn_fwd_config(const rnn_desc_t* desc, int32_t* out6);

const char* rnn_status_str(int status);

/* rnn_fwd for callers that cannot allocate device memory.  The FlashRNN pages
 * have no counterpart; this exists for callers such as a serving process that
 * reserved its whole device-memory budget up front, or a latency-critical loop
 * that must not risk an allocation's implicit device synchronisation.  Same
 * arguments and behaviour as rnn_fwd minus the workspace: its scratch (the
 * device status word) lives in a 4096-byte file-scope __device__ array of the
 * library, held by every GPU that loads the library until the process exits.
 * Calls needing more scratch than that return RNN_ERR_SCRATCH_LIMIT.  The first
 * call on a device looks up the array's device address (cudaGetSymbolAddress)
 * and keeps it for the life of the process, so make that first call before any
 * stream capture, and do not call cudaDeviceReset on that device afterwards (the
 * kept address would then be stale).  Every call shares the array and clears
 * the status word it uses.  Because the caller cannot read the array, the
 * call's device status is delivered through `device_status`: NULL (not
 * reported), or an int the caller owns in device memory or page-locked host
 * memory, which receives the status word by a copy ordered on `stream` after
 * the recurrence -- 0 when every bounded wait completed, nonzero when one ran
 * out (RNN_ERR_TIMEOUT: outputs invalid).  Calls that overlap on the GPU race on
 * the array, so a status delivered to one of them may belong to the other.
 * Allocates nothing (no cudaMalloc / cudaFree, no allocating library call). */
int rnn_fwd_noalloc(const rnn_desc_t* desc, const void* Wx, const void* R, const float* bias,
                    const float* h0, const float* c0, const float* n0, const float* m0,
                    void* h_seq, float* hT, float* cT, float* nT, float* mT, void* stash,
                    int* device_status, void* stream);

/* ---- Operators of language models around and beside the recurrences ------
 *
 * Root-mean-square norm with the residual's addition, over rows of N values:
 *   h = x + residual (rounded to dtype),  r = 1 / sqrt(mean_n h^2 + eps),  y = h r weight
 * dtype (RNN_F32 / RNN_BF16): type of x, residual, h and y [rows, N]; weight [N]
 * fp32.  residual NULL = none; h NULL = not written (h may be x or residual).  The
 * norm is taken of h as stored.  rstd [rows] fp32 (NULL = not written) is r, for the
 * gradient.  scale NULL: y has dtype.  Otherwise y is 8-bit floating point (e4m3)
 * and scale [rows, ceil(N/128)] fp32 holds, for each row and block of 128
 * columns, max|y| / 448 (1 where that is zero); y holds the exact quotient y / scale,
 * rounded to fp32 and then to e4m3 (to nearest even).  A y that is not a number has a
 * NaN code and does not count towards its block's scale; an infinite one has a NaN code
 * and makes the scale infinite.  Squares are summed in fp32: a row with values past 2^63
 * can have r = 0.  N == 0 is refused, rows == 0 a no-op.  Any N up to 2^31 - 4096; widths
 * that are a multiple of 16 bytes (of 8 values for e4m3) with 16-byte aligned pointers
 * run the vector kernels.  Alignment: the element's.  No workspace, no device status. */
int rnn_rms_norm(int32_t dtype, int32_t rows, int32_t N, float eps, const void* x,
                 const void* residual, const float* weight, void* h, void* y, float* scale,
                 float* rstd, void* stream);

/* Its gradient from the stored h and rstd (an 8-bit output's rounding counts as the
 * identity): with xh = h rstd,
 *   dx = rstd (weight dy - xh mean_n(weight dy xh)) + dh,   dw = sum over rows of dy xh
 * dx is the gradient of x and of residual alike; dh (NULL = 0) what reaches h from
 * elsewhere.  dy, h, dh, dx [rows, N] in dtype (dx may be dh), dw [N] fp32 (NULL = not
 * computed, then the workspace may be NULL).  Sums in fp32, in a fixed order.
 * rows == 0 sets dw to zero.  Workspace: 256-byte aligned, size below. */
size_t rnn_rms_norm_bwd_workspace_size(int32_t rows, int32_t N);
int rnn_rms_norm_bwd(int32_t dtype, int32_t rows, int32_t N, const void* dy, const void* h,
                     const float* weight, const float* rstd, const void* dh, void* dx, float* dw,
                     void* workspace, size_t workspace_bytes, void* stream);

/* A weight W [N, K] (dtype) in 8 bits: Wq [N, K] e4m3, Ws [ceil(N/128), ceil(K/128)]
 * fp32, one scale (max|W| / 448, 1 where that is zero) for each 128 x 128 block;
 * values that are not finite as above.  N at most 8388480, K at most 2^31 - 4096. */
int rnn_quantize_weight(int32_t dtype, int32_t N, int32_t K, const void* W, void* Wq, float* Ws,
                        void* stream);

/* rnn_input_proj in 8-bit floating point with a scale for each block of 128:
 *   y[m, n] = sum_b xs[m, b] Ws[n/128, b] (sum_{k in block b} xq[m, k] Wq[n, k]) + bias[n]
 * xq [M, K], Wq [N, K] e4m3; xs [M, ceil(K/128)] and Ws [ceil(N/128), ceil(K/128)] fp32
 * (rnn_rms_norm's and rnn_quantize_weight's outputs); bias [N] fp32 (NULL =
 * none); y [M, N] bf16, rounded once from the fp32 sum.  Requires K % 16 == 0,
 * N % 8 == 0, M <= 8388480, N and K at most 2^31 - 4096.  Alignment: xq, Wq, y 16
 * bytes, fp32 pointers 4, workspace 256 bytes and >= 256 bytes (status word at offset 0).  M == 0 is a no-op. */
int rnn_input_proj_fp8(int32_t M, int32_t N, int32_t K, const void* xq, const float* xs,
                       const void* Wq, const float* Ws, const float* bias, void* y,
                       void* workspace, size_t workspace_bytes, void* stream);

/* Linear attention with a decay for each head, lambda_h = exp(log_decay[h]):
 *   S_t = lambda S_{t-1} + k_t v_t^T,   o_t = scale q_t S_t      (S [Dk, Dv] fp32 per head)
 * q, k [T, B, NH, Dk], v, o [T, B, NH, Dv] in dtype; Dk, Dv in {32, 64, 128, 256};
 * log_decay [NH] fp32, <= 0 (a constant of the layer: no gradient; -inf forgets all);
 * state0, stateT [B, NH, Dk, Dv] fp32 (NULL = zero / not written; stateT may be state0).
 * lens [B] int32 (NULL = T for every row): tokens of a row that count, taken as at
 * least 0 and at most T; what the others hold does not matter, their outputs are zero, and
 * stateT is the state after the last one that counts.
 * Operands may be strided views (of one fused projection, say): strides in elements
 * for (token, row, head), the innermost dimension contiguous; st NULL = contiguous.
 * RNN_BF16: tokens are taken in chunks of 64 or 128 on the tensor cores, scores and the
 * state as an operand rounded to bf16 once, all sums and the state fp32.  RNN_F32: fp32 throughout.
 * A value that is not finite reaches the outputs of its own and later tokens of its row and head and the
 * state, as the recurrence has it (in the gradient: the tokens before it, too); never an
 * output that does not depend on it.
 * Alignment: 16 bytes for tensors and strides, 4 for log_decay and lens, workspace 256
 * and >= rnn_linattn_workspace_size(desc, 0) bytes (status word at offset 0). */
typedef struct {
  int32_t dtype; /* rnn_dtype_t of q, k, v, o */
  int32_t T, B, NH, Dk, Dv;
  float scale;
  int32_t flags; /* 0, or RNN_FLAG_TEST_TIMEOUT: rnn_linattn_fwd and _bwd at sizes whose kernels wait on the device
                    (tcgen05), else RNN_ERR_UNSUPPORTED */
} rnn_linattn_desc_t;

typedef struct {
  int64_t q[3], k[3], v[3], o[3]; /* (token, row, head), elements */
} rnn_linattn_strides_t;

/* Bytes of device workspace of rnn_linattn_fwd (pass 0) / rnn_linattn_bwd (pass 1);
 * 0 on an invalid desc. */
size_t rnn_linattn_workspace_size(const rnn_linattn_desc_t* desc, int pass);

int rnn_linattn_fwd(const rnn_linattn_desc_t* desc, const rnn_linattn_strides_t* st, const void* q,
                    const void* k, const void* v, const float* log_decay, const int32_t* lens,
                    const float* state0, void* o, float* stateT, void* workspace,
                    size_t workspace_bytes, void* stream);

/* Gradients of L = sum(o * dout) + sum(stateT * dstateT) from the forward's inputs (nothing
 * is stashed): dq, dk [T, B, NH, Dk], dv [T, B, NH, Dv] contiguous in dtype, zero for
 * tokens that do not count; dstate0 [B, NH, Dk, Dv] fp32 (NULL = not written; must be neither
 * state0 nor dstateT).  dout has the strides st->o; dstateT NULL = zero.  Workspace as above (pass 1). */
int rnn_linattn_bwd(const rnn_linattn_desc_t* desc, const rnn_linattn_strides_t* st, const void* q,
                    const void* k, const void* v, const float* log_decay, const int32_t* lens,
                    const float* state0, const void* dout, const float* dstateT, void* dq, void* dk,
                    void* dv, float* dstate0, void* workspace, size_t workspace_bytes,
                    void* stream);

/* One token (desc->T == 1) for each of B rows out of a cache of n_slots states
 * [n_slots, NH, Dk, Dv] fp32, updated in place: row b uses state slots[b] (slots NULL: state
 * b).  A row whose slot is not in [0, n_slots) has no state: its o is zero.  Two rows must
 * not name the same slot.  o [B, NH, Dv] contiguous in dtype; token strides and st->o are
 * not used.  Alignment as above.  No workspace, no device status. */
int rnn_linattn_step(const rnn_linattn_desc_t* desc, const rnn_linattn_strides_t* st, const void* q,
                     const void* k, const void* v, const float* log_decay, const int32_t* slots,
                     int32_t n_slots, float* state, void* o, void* stream);

/* Gated linear recurrence: the cells without a recurrent matrix, so that a sequence is a scan.  For
 * each row, head and channel, with the gates of Wx [T, B, NH, G*D] (gate-major, as for rnn_fwd):
 *   RNN_GATES_FZ    c_t = sigm(f) c_{t-1} + sigm(-f) z           y_t = c_t
 *   RNN_GATES_FZO   the same                                     y_t = sigm(o) c_t
 *   RNN_GATES_IFZO  c_t = sigm(f) c_{t-1} + sigm(i) z            y_t = sigm(o) c_t
 * y [T, B, NH, D] in dtype; state0, stateT [B, NH, D] fp32 (NULL = zero / not written; stateT may be
 * state0).  lens [B] int32 (NULL = T for every row): tokens of a row that count, taken as at least
 * 0 and at most T; what the others hold does not matter, their y is zero, and stateT is the state
 * after the last one that counts.  stash (NULL = not written): what rnn_gated_bwd needs,
 * rnn_gated_stash_size bytes.  Gates, states and sums are fp32, y is rounded once.  A value that is not
 * finite reaches its own and later tokens of its row and channel (in the gradient: earlier ones, too) and
 * nothing else; where a product of forget gates underflows, an infinity before it may turn to NaN.
 * Wx, y contiguous; aligned as their element is.  From 65 tokens on, heads of a multiple of 16 bytes at addresses that
 * are run on tiles that the kernels wait for.  workspace: 256-byte aligned, >= 256 bytes (status word at offset 0). */
typedef enum { RNN_GATES_FZ = 2, RNN_GATES_FZO = 3, RNN_GATES_IFZO = 4 } rnn_gates_t;

typedef struct {
  int32_t dtype; /* rnn_dtype_t of Wx, y, dy, dWx */
  int32_t T, B, NH, D;
  int32_t gates; /* rnn_gates_t: the gates' number G */
  int32_t flags; /* 0, or RNN_FLAG_TEST_TIMEOUT: rnn_gated_fwd and _bwd at sizes and addresses that run on tiles,
                    else RNN_ERR_UNSUPPORTED */
} rnn_gated_desc_t;

/* Bytes of the stash: the fp32 state before every eighth token, [ceil(T/8), B, NH, D].  0 on an invalid desc. */
size_t rnn_gated_stash_size(const rnn_gated_desc_t* desc);

int rnn_gated_fwd(const rnn_gated_desc_t* desc, const void* Wx, const int32_t* lens, const float* state0, void* y,
                  float* stateT, float* stash, void* workspace, size_t workspace_bytes, void* stream);

/* Gradients of L = sum(y * dy) + sum(stateT * dstateT) from the forward's Wx, lens and stash: dWx like Wx (zero for
 * tokens that do not count), dstate0 [B, NH, D] fp32 (NULL = not written; may be dstateT).  dstateT NULL = zero. */
int rnn_gated_bwd(const rnn_gated_desc_t* desc, const void* Wx, const int32_t* lens, const float* stash, const void* dy,
                  const float* dstateT, void* dWx, float* dstate0, void* workspace, size_t workspace_bytes,
                  void* stream);

/* Launch geometry that rnn_gated_fwd (gradient != 0: rnn_gated_bwd) would use for tensors at aligned addresses:
 * out[0..6] = grid CTAs, threads per CTA, cluster size, channels of a tile, whether maps are made a round ahead, dynamic
 * smem bytes, clusters (cluster size 1: CTAs) that the device holds at once; the last four are 0 for the kernels without
 * tiles, all where nothing is launched. */
int rnn_gated_config(const rnn_gated_desc_t* desc, int32_t gradient, int32_t* out7);

/* One token (desc->T == 1, Wx [B, NH, G*D]) for each of B rows out of a cache of n_slots states [n_slots, NH, D] fp32,
 * updated in place: row b uses state slots[b] (slots NULL: state b).  A row whose slot is not in [0, n_slots) has no
 * state: its y is zero.  Two rows must not name the same slot.  No workspace, no device status. */
int rnn_gated_step(const rnn_gated_desc_t* desc, const void* Wx, const int32_t* slots, int32_t n_slots, float* state,
                   void* y, void* stream);

/* Norm of each query's and key's head with the rotation by its token's position, in one pass: for x = a head [D] of q
 * or k at position pos, w its weight,
 *   y = x w / sqrt(mean x^2 + eps);  for j < rot/2 the pair (y1, y2) becomes
 *   (y1 cos - y2 sin, y2 cos + y1 sin) of the angle pos freqs[j]
 * with the pair's columns j and j + rot/2, or 2j and 2j + 1 with RNN_ROTARY_INTERLEAVED; columns from rot on are not
 * turned (y alone, whatever their neighbours hold).  q [T, B, NQ, D], k [T, B, NK, D] in dtype (strided views as for the
 * attention: strides of q and k for (token, row, head), st NULL = contiguous), outputs contiguous in dtype, rounded once.
 * q_weight, k_weight [D] fp32; both NULL = no norm.  freqs [rot/2] fp64, below 2^54, radians a position (NULL with
 * rot == 0: no rotation).  positions int32: [B], where each row's first token stands, the following ones after it;
 * [T, B] with RNN_ROTARY_PER_TOKEN; NULL = 0 for every row.  Any position: angles are formed modulo a turn in 64 bits of
 * fraction.  Squares are summed in fp32: a head with values past 2^63 comes out as zero; with eps = 0 one whose values
 * are all below 2^-63 loses bits, below 2^-75 all of them (infinities, or NaN for zeros).
 * D and rot even, rot <= D <= 4096, T*B at most 2^31 - 1.  Alignment: the element's.  D that is a multiple of 8 up to
 * 256 (and, unless interleaved, rot too) with strides and addresses that are multiples of four values runs the vector
 * kernels. */
enum { RNN_ROTARY_INTERLEAVED = 1, RNN_ROTARY_PER_TOKEN = 2 };

typedef struct {
  int32_t dtype; /* rnn_dtype_t of q, k and what comes of them */
  int32_t T, B, NQ, NK, D, rot;
  float eps;
  int32_t flags; /* RNN_ROTARY_* */
} rnn_rotary_desc_t;

typedef struct {
  int64_t q[3], k[3], dq[3], dk[3]; /* (token, row, head), elements; dq, dk: the gradient's inputs */
} rnn_rotary_strides_t;

int rnn_head_norm_rotary(const rnn_rotary_desc_t* desc, const rnn_rotary_strides_t* st, const void* q, const void* k,
                         const float* q_weight, const float* k_weight, const double* freqs, const int32_t* positions,
                         void* q_out, void* k_out, void* stream);

/* Its gradient from q and k as the forward took them and dq_out, dk_out (strides st->dq, st->dk), the gradients of its
 * outputs: dq, dk contiguous in dtype, dq_weight, dk_weight [D] fp32 (both needed where the weights are given), summed in
 * fp32 in a fixed order.  Workspace: 256-byte aligned, size below (none without weights). */
size_t rnn_head_norm_rotary_bwd_workspace_size(const rnn_rotary_desc_t* desc);
int rnn_head_norm_rotary_bwd(const rnn_rotary_desc_t* desc, const rnn_rotary_strides_t* st, const void* q,
                             const void* k, const float* q_weight, const float* k_weight, const double* freqs,
                             const int32_t* positions, const void* dq_out, const void* dk_out, void* dq, void* dk,
                             float* dq_weight, float* dk_weight, void* workspace, size_t workspace_bytes,
                             void* stream);

/* The common norm of n tensors, sqrt(sum of all x^2), to *norm (fp32, NULL = not written), and their scaling to it: where
 * it is finite and above max_norm every value becomes x (max_norm / norm) in place, rounded once; else nothing is written to
 * them.  max_norm >= 0; INFINITY = the norm alone.  dtypes (rnn_dtype_t), sizes (elements; 0 is allowed) and
 * tensors (device memory, aligned as the element is) are host arrays, read before the call returns.  Unless max_norm is
 * INFINITY no two tensors may overlap (RNN_ERR_INVALID_ARG).  Sums are taken in fixed order: fp32 over 64 bytes, fp32 with
 * the rounding errors carried along over what a warp takes, fp64 above; no square overflows (a norm that fp32 cannot hold
 * is told as infinity, and clipped to max_norm all the same).  A tensor's size is at most 2^40, at most 2^28 tensors,
 * 2^31 - 1 pieces of 16 KB in all of them.  Workspace: 256-byte aligned, size below. */
size_t rnn_clip_grad_norm_workspace_size(int32_t n);
int rnn_clip_grad_norm(int32_t n, const int32_t* dtypes, const int64_t* sizes, void* const* tensors, float max_norm,
                       float* norm, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* SEQUENTIAL_RNN_GB300_RNN_H */
