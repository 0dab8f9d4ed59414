/*
 * kda.h - C ABI of libkda.so: Kimi Delta Attention (KDA) chunked prefill and
 * decode step on one GB300 (sm_103a), the gated linear recurrence, the norms
 * around a block, and the softmax attention over a paged cache of the layers
 * that stand between recurrent ones.
 *
 * Cited page: "Kimi K3：从 3T 稀疏预训练到百万 Token Agent 的端到端扩展"
 * (liuzhao09.github.io/papers/kimi-k3), [K3-notes] below.
 *
 * The operation ([K3-notes §2.2, KDA state recurrence]), per sequence n and
 * head h, over that sequence's tokens t in order:
 *     S_t = (I - beta_t k_t k_t^T) Diag(alpha_t) S_{t-1} + beta_t k_t v_t^T
 *     o_t = S_t^T q_t,            alpha_t = exp(log_alpha_t)  (per channel)
 * with S in R^{dk x dv}.  The library does not scale or normalise q or k.
 *
 * Conventions shared by every call
 * --------------------------------
 *  - All tensor pointers are DEVICE pointers owned by the caller; the library
 *    keeps no pointer after the call returns.  Alignment (KDA_ERR_ALIGN
 *    otherwise): kda_chunk_fwd needs q, k, v, log_alpha and out 16-byte
 *    aligned and the other pointers 4-byte aligned; kda_decode_step needs
 *    state_inout 16-byte aligned and the other pointers aligned to their
 *    element size.  Tensors are dense and row-major in the shapes written
 *    below (last index contiguous).
 *  - Work is enqueued on `stream` (a cudaStream_t; NULL = legacy default
 *    stream) and the call returns without waiting, except in validate mode.
 *  - Argument errors are reported synchronously, before anything is launched,
 *    as a negative kda_status.  A launch failure returns KDA_ERR_CUDA.
 *    Asynchronous device faults surface at the caller's next synchronisation.
 *  - Preconditions on values ([K3-notes §2.2, Eq. 5] bounds the log-decay
 *    below by g_min = -5): log_alpha in [-5, 0], beta in [0, 1], cu_seqlens
 *    non-decreasing from 0 to T.  The kernels rely on the log-decay floor for
 *    their range guard.  They are checked only in validate mode (desc.validate
 *    = 1), which runs a check kernel first, synchronises the stream and
 *    returns KDA_ERR_RANGE without computing anything if a value is outside.
 *  - Results are deterministic: the same inputs give bitwise the same outputs.
 */
#ifndef KDA_H_
#define KDA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st;
typedef struct CUstream_st *kda_stream_t; /* the same type as cudaStream_t */

typedef enum { KDA_F32 = 0, KDA_BF16 = 1 } kda_dtype;

typedef enum {
  KDA_OK = 0,
  KDA_ERR_NULL = -1,        /* a required pointer (or the descriptor) is NULL      */
  KDA_ERR_SHAPE = -2,       /* a size is out of the supported set                  */
  KDA_ERR_DTYPE = -3,       /* unsupported dtype combination                       */
  KDA_ERR_ALIGN = -4,       /* a pointer is not 16-byte aligned                    */
  KDA_ERR_RANGE = -5,       /* validate mode found a value outside its range       */
  KDA_ERR_CUDA = -6,        /* a CUDA call or kernel launch failed                 */
  KDA_ERR_UNSUPPORTED = -7, /* a kernel choice that does not cover these arguments */
  KDA_ERR_ALIAS = -8,       /* forbidden aliasing between arguments                */
  KDA_ERR_SCRATCH_LIMIT = -9 /* kda_chunk_fwd_noalloc: the call needs more scratch
                                than KDA_STATIC_WORKSPACE_BYTES                      */
} kda_status;

/* Which prefill kernel runs.  AUTO picks the tensor-core kernel when it covers
 * the arguments (bf16 q/k/v, bf16 out, dk = dv = 128, chunk = 64) and the
 * CUDA-core kernel otherwise.  Asking for TC on arguments it does not cover
 * returns KDA_ERR_UNSUPPORTED. */
typedef enum { KDA_KERNEL_AUTO = 0, KDA_KERNEL_SIMT = 1, KDA_KERNEL_TC = 2 } kda_kernel;

typedef struct {
  int B;          /* batch; must be 1 when cu_seqlens is given                */
  int T;          /* tokens per sequence, or total tokens when varlen          */
  int H;          /* heads                                                    */
  int dk, dv;     /* key and value head dims: each one of 16, 32, 64, 128      */
  int chunk;      /* chunk length C: 16, 32 or 64 (outputs do not depend on it
                     beyond rounding)                                          */
  int num_seqs;   /* varlen: number of sequences N (cu_seqlens has N+1 entries);
                     0 when cu_seqlens is NULL                                 */
  kda_dtype qkv_dtype;  /* q, k, v                                             */
  kda_dtype out_dtype;  /* out                                                 */
  kda_dtype gate_dtype; /* log_alpha and beta                                  */
  int validate;   /* 1: range-check inputs first (synchronises the stream)     */
  kda_kernel kernel;
  int segments;   /* long sequences: split each sequence into this many
                     segments that run in parallel and are joined through
                     their affine pairs; 0 = choose automatically, 1 = never  */
} kda_chunk_desc;

/*
 * kda_chunk_fwd - chunked prefill ([K3-notes §2.2, chunkwise form];
 * initial/final state for prefix-cache resume, [K3-notes §2.5, Fig. 12]).
 *
 *   q, k        [B*T, H, dk]  qkv_dtype   (token-major; B sequences of T
 *                                          tokens, or N packed sequences)
 *   v           [B*T, H, dv]  qkv_dtype
 *   log_alpha   [B*T, H, dk]  gate_dtype  (g = ln alpha, per channel)
 *   beta        [B*T, H]      gate_dtype
 *   initial_state [Nseq, H, dk, dv] fp32, or NULL for zeros
 *   cu_seqlens  [N+1] int32 (varlen: sequence n is tokens
 *               [cu_seqlens[n], cu_seqlens[n+1]) ), or NULL for B x T
 *   out         [B*T, H, dv]  out_dtype   (written)
 *   final_state [Nseq, H, dk, dv] fp32, or NULL (written)
 * Nseq = num_seqs when varlen, else B.  An empty sequence leaves its
 * final state equal to its initial state.  initial_state may equal
 * final_state (in-place resume); out may not alias any input.
 * When the planner splits long sequences into segments it allocates a
 * stream-ordered workspace (cudaMallocAsync/cudaFreeAsync on `stream`); use
 * kda_chunk_fwd_ex to pass one instead.
 */
kda_status kda_chunk_fwd(const kda_chunk_desc *desc, const void *q, const void *k, const void *v,
                         const void *log_alpha, const void *beta, const float *initial_state,
                         const int32_t *cu_seqlens, void *out, float *final_state,
                         kda_stream_t stream);

/* Bytes of device workspace kda_chunk_fwd_ex needs for these arguments (0 when
 * no sequence is split).  Host-only; launches nothing. */
kda_status kda_chunk_fwd_workspace_size(const kda_chunk_desc *desc, size_t *bytes);

/* kda_chunk_fwd with a caller-owned device workspace of at least
 * kda_chunk_fwd_workspace_size bytes (16-byte aligned; NULL allowed when that
 * size is 0).  The workspace must not be in use by another call in flight. */
kda_status kda_chunk_fwd_ex(const kda_chunk_desc *desc, const void *q, const void *k,
                            const void *v, const void *log_alpha, const void *beta,
                            const float *initial_state, const int32_t *cu_seqlens, void *out,
                            float *final_state, void *workspace, size_t workspace_bytes,
                            kda_stream_t stream);

/*
 * kda_chunk_fwd_ckpt - kda_chunk_fwd that also stores the state at fixed
 * intervals along each sequence, for prefix-cache reuse ([K3-notes §2.5,
 * Fig. 12]: a request that shares a cached prefix resumes from the state at
 * the prefix's end; a cache that keeps a state every `every` tokens can
 * resume at any multiple of it).
 *
 *   every     checkpoint interval in tokens, a positive multiple of
 *             desc->chunk (KDA_ERR_SHAPE otherwise)
 *   cu_ckpt   [N+1] int32 device, required with cu_seqlens: sequence n's
 *             checkpoints go to slots cu_ckpt[n] .. cu_ckpt[n+1]-1, and
 *             cu_ckpt[n+1] - cu_ckpt[n] must be floor(len_n / every)
 *             (checked in validate mode); NULL for a B x T batch, whose
 *             sequence n uses slots n*floor(T/every) .. (n+1)*floor(T/every)-1
 *   ckpt      [slots, H, dk, dv] fp32 device, written: the j-th slot of a
 *             sequence (j = 1, 2, ...) holds its state after its first
 *             j*every tokens, exactly what kda_chunk_fwd on that prefix
 *             alone would return as final_state (up to rounding)
 *   workspace as in kda_chunk_fwd_ex; NULL makes a split plan allocate its
 *             workspace stream-ordered, as kda_chunk_fwd does
 * Other arguments and conventions as kda_chunk_fwd.  ckpt may alias no other
 * argument (KDA_ERR_ALIAS; for packed sequences only its first slot's extent
 * is known on the host and checked).
 */
kda_status kda_chunk_fwd_ckpt(const kda_chunk_desc *desc, const void *q, const void *k,
                              const void *v, const void *log_alpha, const void *beta,
                              const float *initial_state, const int32_t *cu_seqlens, void *out,
                              float *final_state, int every, const int32_t *cu_ckpt, float *ckpt,
                              void *workspace, size_t workspace_bytes, kda_stream_t stream);

typedef struct {
  int N;          /* independent sequences, one token each                    */
  int H;          /* heads                                                    */
  int dk, dv;     /* each one of 16, 32, 64, 128                              */
  kda_dtype qkv_dtype, out_dtype, gate_dtype;
  int validate;   /* 1: range-check inputs first (synchronises the stream)     */
} kda_decode_desc;

/*
 * kda_decode_step - one token of the recurrence for N sequences, updating
 * their states in place ([K3-notes §2.2, KDA state recurrence]; the decode
 * regime of [K3-notes §2.5]).
 *
 *   q, k        [N, H, dk]  qkv_dtype
 *   v           [N, H, dv]  qkv_dtype
 *   log_alpha   [N, H, dk]  gate_dtype
 *   beta        [N, H]      gate_dtype
 *   state_inout [N, H, dk, dv] fp32, read and overwritten
 *   out         [N, H, dv]  out_dtype, written
 * state_inout may not alias out or any input.
 */
kda_status kda_decode_step(const kda_decode_desc *desc, const void *q, const void *k,
                           const void *v, const void *log_alpha, const void *beta,
                           float *state_inout, void *out, kda_stream_t stream);

/*
 * The KDA layer's gates around the recurrence ([K3-notes §2.2]):
 *   decay gate (Eq. 5):  log_alpha = g_min * Sigmoid(exp(A_h) * z)
 *       z the decay logits [tokens, H, dk] (from the layer's low-rank decay
 *       projection), A_h a per-head log scale, Sigmoid(x) = 1 / (1 + e^-x);
 *   output (the KDA output equation, before W_o):
 *       y = Sigmoid(out_gate) * RMSNorm(o),   per token and head over dv,
 *       RMSNorm(o)_j = o_j * norm_weight_j / sqrt(mean_j o_j^2 + norm_eps),
 *       out_gate = W_g x [tokens, H, dv].
 * The page names the RMSNorm without its weight or epsilon; here the weight
 * is one learned value per channel, shared by the heads, and eps is given.
 * The projections W_g x, W_o y and the one that makes z are plain GEMMs
 * outside these calls.
 */
typedef struct {
  const float *A_log;       /* [H] fp32 device, required                         */
  float g_min;              /* log-decay floor, in [-5, 0) (-5 on the page: the
                               kernels' range guard needs g_min >= -5)           */
  const void *out_gate;     /* [tokens, H, dv] qkv_dtype device, or NULL: out is
                               o itself (no norm, no gate)                       */
  const float *norm_weight; /* [dv] fp32 device, or NULL for ones               */
  float norm_eps;           /* >= 0 (used only with out_gate)                   */
} kda_layer_gates;

/*
 * kda_layer_fwd - kda_chunk_fwd_ex with the layer's gates: the log-decay is
 * computed in the kernels from z (so log_alpha is never materialised) and,
 * when gates->out_gate is given, each output row is normalised and gated
 * before it is stored.
 *
 *   z         [B*T, H, dk] qkv_dtype (takes log_alpha's place; desc->gate_dtype
 *             now describes beta alone)
 *   out       [B*T, H, dv] out_dtype: y, or o when out_gate is NULL
 * Other arguments and conventions as kda_chunk_fwd_ex (workspace NULL: a
 * split plan allocates its workspace stream-ordered).  z, out_gate and out are
 * 16-byte aligned, A_log and norm_weight 4-byte aligned.  Validate mode checks
 * that z has no NaN, A_log is finite and beta is in [0, 1]; g_min outside
 * [-5, 0) or a negative (or NaN) norm_eps is KDA_ERR_RANGE without validate.
 * On the tensor-core kernel the norm reads the bf16-rounded o, the value an
 * unfused norm would read from out.
 */
kda_status kda_layer_fwd(const kda_chunk_desc *desc, const kda_layer_gates *gates, const void *q,
                         const void *k, const void *v, const void *z, const void *beta,
                         const float *initial_state, const int32_t *cu_seqlens, void *out,
                         float *final_state, void *workspace, size_t workspace_bytes,
                         kda_stream_t stream);

/*
 * kda_layer_decode_step - kda_decode_step with the layer's gates:
 *   z        [N, H, dk] qkv_dtype (in log_alpha's place)
 *   out      [N, H, dv] out_dtype: y, or o when gates->out_gate is NULL
 *   gates->out_gate, when given, [N, H, dv] qkv_dtype
 * Other arguments as kda_decode_step; alignment as kda_decode_step for z and
 * out_gate, 4 bytes for A_log and norm_weight.
 */
kda_status kda_layer_decode_step(const kda_decode_desc *desc, const kda_layer_gates *gates,
                                 const void *q, const void *k, const void *v, const void *z,
                                 const void *beta, float *state_inout, void *out,
                                 kda_stream_t stream);

/*
 * Context parallelism across GPUs ([K3-notes §2.5, context-parallel affine
 * pair]): a segment of a sequence maps any entry state to
 *     S_out = S~ + M S_in,
 * S~ its final state from S_in = 0 and M (dk x dk) the product of its
 * per-token transitions (I - beta k k^T) Diag(alpha); the pairs compose.  A
 * sequence split over R GPUs runs on each rank r: kda_chunk_affine_pair on
 * its segment, an all-gather of the R pairs (fixed size, independent of the
 * segment length), kda_affine_compose for the entry states, and
 * kda_chunk_fwd on its segment from entry state r.
 *
 * kda_chunk_affine_pair - the pair of each sequence of the call (each whole
 * sequence is one segment).  Arguments as kda_chunk_fwd (no states, no out);
 *   pairs  [2][Nseq][H][dk][dv] fp32 device, written: [0] = S~, [1] = M.
 * Tensor-core arguments only (bf16 q/k/v, fp32 gates, dk = dv = 128, chunk
 * 64); KDA_ERR_UNSUPPORTED otherwise or with desc->kernel = KDA_KERNEL_SIMT.
 */
kda_status kda_chunk_affine_pair(const kda_chunk_desc *desc, const void *q, const void *k, const void *v,
                                 const void *log_alpha, const void *beta, const int32_t *cu_seqlens,
                                 float *pairs, kda_stream_t stream);

/*
 * kda_affine_compose - entry states of P consecutive segments:
 *   E_0 = initial_state (NULL: zero),  E_{p+1} = S~_p + M_p E_p   (fp32)
 *   pairs         [2][N][P-1][H][dk][dv] fp32 device (S~ block, then M block;
 *                 may be NULL when P = 1)
 *   entry_states  [N][P][H][dk][dv] fp32 device, written
 * dk = dv = 128; pointers 16-byte aligned; entry_states may alias nothing.
 */
kda_status kda_affine_compose(int N, int H, int dk, int dv, int P, const float *initial_state, const float *pairs,
                              float *entry_states, kda_stream_t stream);

/*
 * kda_chunk_bwd - gradients of kda_chunk_fwd, for training (the chunkwise form
 * of [K3-notes §2.2] is the training form; the page prints no backward, and
 * this one is the exact derivative of the forward's mathematics).  For the
 * scalar L = sum_t <d_out_t, o_t> + sum_n <d_final_state_n, S_T(n)> it writes
 *
 *   dq, dk       [B*T, H, dk] fp32    dL/dq, dL/dk
 *   dv           [B*T, H, dv] fp32    dL/dv
 *   dlog_alpha   [B*T, H, dk] fp32    dL/dlog_alpha
 *   dbeta        [B*T, H]     fp32    dL/dbeta
 *   d_initial_state [Nseq, H, dk, dv] fp32, or NULL   dL/dinitial_state
 *
 * from the forward's inputs (same arguments and conventions as kda_chunk_fwd;
 * initial_state NULL = zeros) and
 *   d_out          [B*T, H, dv] out_dtype   (gradient of out)
 *   d_final_state  [Nseq, H, dk, dv] fp32, or NULL for zero.
 * The forward is recomputed inside; nothing of it needs to be kept.  The
 * gradients do not depend on desc->chunk (the backward works on 16-token
 * chunks, the tile within which the decay floor keeps every factor in fp32
 * range); desc->segments is ignored and desc->kernel = KDA_KERNEL_TC returns
 * KDA_ERR_UNSUPPORTED (the backward runs on CUDA cores, in fp32).
 *
 *   workspace  device buffer of kda_chunk_bwd_workspace_size bytes, 16-byte
 *              aligned, or NULL: then the call allocates it stream-ordered
 *              (cudaMallocAsync / cudaFreeAsync on `stream`).  It holds, per
 *              16-token chunk and head, the state before the chunk and the
 *              state gradient after it (2 dk dv floats) and 3 C dk + 2 C^2 + dk
 *              floats of chunk matrices: about 130 KB per 16 tokens per head at
 *              dk = dv = 128.
 * Gradients may alias no input and no other gradient (KDA_ERR_ALIAS); all
 * pointers 4-byte aligned except q, k, v, log_alpha, d_out (16 bytes, as the
 * forward's q/k/v/log_alpha/out).
 */
kda_status kda_chunk_bwd_workspace_size(const kda_chunk_desc *desc, size_t *bytes);
kda_status kda_chunk_bwd(const kda_chunk_desc *desc, const void *q, const void *k, const void *v,
                         const void *log_alpha, const void *beta, const float *initial_state,
                         const int32_t *cu_seqlens, const void *d_out, const float *d_final_state,
                         float *dq, float *dk, float *dv, float *dlog_alpha, float *dbeta,
                         float *d_initial_state, void *workspace, size_t workspace_bytes,
                         kda_stream_t stream);

/*
 * Gated linear recurrence.  The recurrence without its key: every channel of
 * every head is a chain of its own,
 *     h_t = alpha_t h_{t-1} + w_t x_t,     out_t = h_t,     alpha_t = exp(g_t)
 *     w_t = 1              (KDA_WRITE_ONE)
 *     w_t = 1 - alpha_t    (KDA_WRITE_COMPLEMENT: h is a running mean of x)
 * with the log-decay g given, or formed from decay logits z by the layer's
 * decay gate (see kda_layer_gates), g = g_min Sigmoid(exp(A_h) z).
 *
 * Conventions shared by kda_scan_fwd, kda_scan_bwd and kda_scan_step
 *  - [tokens, H, d] tensors are token-major and dense, as kda_chunk_fwd's;
 *    H and d are any positive sizes with H * d < 2^27; tokens are below 2^31 - 65536.
 *  - x, out and their gradients have dtype `dtype`.  `decay` is log_alpha in
 *    `gate_dtype` when A_log is NULL, and z in `dtype` otherwise (g_min is then
 *    in [-5, 0), KDA_ERR_RANGE otherwise).
 *  - Pointers need their element's alignment; tensors that are all 16-byte
 *    aligned, with rows of H * d elements that are multiples of 16 bytes, run
 *    vectorised, others elementwise, with the same results up to rounding.
 *  - Arithmetic is fp32, states and state gradients are fp32; out, dx and
 *    d_decay are rounded once.  An alpha below 2^-126 is 0.  What is left of a state
 *    (or of a gradient) after some tokens is off by at most 9 half steps of fp32
 *    (2^-24) for each 16 tokens begun and 18 |g_t| for each one; dA_log is summed
 *    with compensation.  Results are deterministic.
 *  - log_alpha is any value <= 0; -inf is alpha = 0 and forgets the state.  z is
 *    any value; at +-inf its gradient is 0.  A non-finite x, state or gradient
 *    makes what follows of its own chain non-finite, and no other chain.
 *    Validate mode returns KDA_ERR_RANGE for a log_alpha above 0 or NaN, a NaN
 *    z, a non-finite A_log, or cu_seqlens that do not start at 0 or that
 *    decrease or pass the token count.  (Without it such cu_seqlens are clamped
 *    to the tensors, so no call reads or writes outside them, and a NaN reaches
 *    its own chain, one in A_log its own head.)
 *  - cu_seqlens may end before the last token: rows behind the last sequence
 *    are neither read nor written.
 */
typedef enum { KDA_WRITE_ONE = 0, KDA_WRITE_COMPLEMENT = 1 } kda_scan_write;

/* Tokens between two of the states kda_scan_fwd keeps for kda_scan_bwd. */
#define KDA_SCAN_TILE 16

typedef struct {
  int B;          /* batch; must be 1 when cu_seqlens is given                */
  int T;          /* tokens per sequence, or total tokens when varlen          */
  int H, d;       /* heads, channels per head                                  */
  int num_seqs;   /* varlen: number of sequences N; 0 when cu_seqlens is NULL  */
  kda_dtype dtype;      /* x, out, d_out, dx; z and its gradient               */
  kda_dtype gate_dtype; /* log_alpha and its gradient (ignored with A_log)     */
  kda_scan_write write;
  int validate;   /* 1: range-check inputs first (synchronises the stream)     */
} kda_scan_desc;

/* Bytes of the `states` buffer of kda_scan_fwd and kda_scan_bwd. */
kda_status kda_scan_states_size(const kda_scan_desc *desc, size_t *bytes);

/*
 * kda_scan_fwd
 *   x             [tokens, H, d] dtype
 *   decay         [tokens, H, d] log_alpha or z
 *   A_log         [H] fp32 device, or NULL
 *   initial_state [Nseq, H, d] fp32, or NULL for zeros
 *   cu_seqlens    [N+1] int32, or NULL for B x T
 *   out           [tokens, H, d] dtype, written
 *   final_state   [Nseq, H, d] fp32, or NULL (written); may equal initial_state
 *   states        kda_scan_states_size bytes, or NULL (written): the state
 *                 before every KDA_SCAN_TILE-th token of each sequence, in the
 *                 library's own order, for kda_scan_bwd on the same arguments
 * An empty sequence leaves its final state equal to its initial state.  Outputs
 * may alias nothing else (KDA_ERR_ALIAS).
 */
kda_status kda_scan_fwd(const kda_scan_desc *desc, const void *x, const void *decay, const float *A_log,
                        float g_min, const float *initial_state, const int32_t *cu_seqlens, void *out,
                        float *final_state, float *states, kda_stream_t stream);

/*
 * kda_scan_bwd - gradients of kda_scan_fwd for
 * L = sum_t <d_out_t, out_t> + sum_n <d_final_state_n, h_T(n)>:
 *     D_t = d_out_t + alpha_{t+1} D_{t+1}   (D_T also gets d_final_state)
 *     dx_t = w_t D_t,    dg_t = alpha_t D_t (h_{t-1} - [x_t with COMPLEMENT])
 *     d_initial_state = alpha_1 D_1
 *     dz = dg g (1 - g / g_min) exp(A_h),    dA_log_h = sum z dz
 *   states          what kda_scan_fwd stored, or NULL: then a forward pass
 *                   inside the call rebuilds them
 *   d_out           [tokens, H, d] dtype
 *   d_final_state   [Nseq, H, d] fp32, or NULL for zero
 *   dx              [tokens, H, d] dtype, written
 *   d_decay         [tokens, H, d] decay's dtype, written: dlog_alpha or dz
 *   dA_log          [H] fp32, written; required with A_log and NULL without
 *   d_initial_state [Nseq, H, d] fp32, or NULL
 *   workspace       kda_scan_bwd_workspace_size bytes (16-byte aligned; with
 *                   `states` given the size is smaller), or NULL: then a call
 *                   that needs some allocates it stream-ordered
 * Rows behind the last sequence get no gradient and add nothing to dA_log.
 */
kda_status kda_scan_bwd_workspace_size(const kda_scan_desc *desc, int logits, int have_states, size_t *bytes);
kda_status kda_scan_bwd(const kda_scan_desc *desc, const void *x, const void *decay, const float *A_log,
                        float g_min, const float *initial_state, const int32_t *cu_seqlens,
                        const float *states, const void *d_out, const float *d_final_state, void *dx,
                        void *d_decay, float *dA_log, float *d_initial_state, void *workspace,
                        size_t workspace_bytes, kda_stream_t stream);

/*
 * kda_scan_step - one token for B sequences (desc: T = 1, num_seqs = 0).
 *   x, decay, out [B, H, d];  state_in, state_out [B, H, d] fp32, state_out
 *   written; state_out may equal state_in (update in place).
 */
kda_status kda_scan_step(const kda_scan_desc *desc, const void *x, const void *decay, const float *A_log,
                         float g_min, const float *state_in, float *state_out, void *out, kda_stream_t stream);

/*
 * Norms before and after a block, fused with its gate and residual scale.  Per
 * row of `width` channels (a token; or a token's head, then width = dv and the
 * result is the KDA output equation, see kda_layer_gates):
 *     u      = RMSNorm(y; post_weight, post_eps)        (post_norm; else y)
 *     b      = Sigmoid(gate) o u                        (gate given; else u)
 *     out    = residual + scale o b                     (missing parts: 0, 1)
 *     normed = RMSNorm(out; pre_weight, pre_eps)        (the next block's input)
 *     RMSNorm(a; w, e)_j = a_j w_j / sqrt(mean_j a_j^2 + e)
 * Conventions
 *  - y, gate and normed (and their gradients) have dtype `dtype`; residual and
 *    out (and theirs) `res_dtype`, which equals dtype when residual is NULL.
 *    Weights, scale and their gradients are fp32 [width].
 *  - 0 <= rows, 1 <= width <= KDA_NORM_MAX_WIDTH.  Rows are dense.  Pointers need
 *    their element's alignment; 16-byte aligned tensors of a width that is a
 *    multiple of 8 run vectorised.
 *  - Arithmetic is fp32 (mean squares too: a row's squares must not overflow)
 *    and each output is rounded once; normed is formed from the unrounded out.
 *    A row of zeros gives zeros when eps > 0.  Non-finite values reach their own
 *    row and the weights' gradients alone (those are fp32 sums over the rows).
 *    Results are deterministic.
 */
#define KDA_NORM_MAX_WIDTH 8192

typedef struct {
  int64_t rows;
  int width;
  kda_dtype dtype, res_dtype;
  int post_norm;  /* 1: RMSNorm of y                                           */
  float post_eps; /* >= 0, used with post_norm                                 */
  float pre_eps;  /* >= 0, used with normed / d_normed                         */
} kda_norm_desc;

/*
 * kda_block_norm_fwd
 *   y           [rows, width] dtype
 *   residual    [rows, width] res_dtype, or NULL
 *   gate        [rows, width] dtype (logits), or NULL
 *   post_weight [width] fp32, or NULL for ones (must be NULL without post_norm)
 *   scale       [width] fp32, or NULL for ones
 *   pre_weight  [width] fp32, or NULL for ones (must be NULL without normed)
 *   out         [rows, width] res_dtype, or NULL when not wanted; may equal
 *               residual (update in place)
 *   normed      [rows, width] dtype, or NULL when not wanted (one of the two
 *               outputs is required)
 * Outputs may alias nothing else (KDA_ERR_ALIAS).
 */
kda_status kda_block_norm_fwd(const kda_norm_desc *desc, const void *y, const void *residual, const void *gate,
                              const float *post_weight, const float *scale, const float *pre_weight, void *out,
                              void *normed, kda_stream_t stream);

/*
 * kda_block_norm_bwd - gradients of L = <d_out, out> + <d_normed, normed>, from
 * the forward's inputs (the forward is recomputed).
 *   d_out       [rows, width] res_dtype, or NULL for zero
 *   d_normed    [rows, width] dtype, or NULL for zero (one of them is required);
 *               pre_weight is not read without it
 *   d_y         [rows, width] dtype, written
 *   d_residual  [rows, width] res_dtype, or NULL; may equal d_out
 *   d_gate      [rows, width] dtype; given exactly when gate is
 *   d_post_weight, d_scale, d_pre_weight  [width] fp32, each or NULL; sums over
 *               the rows (zeros when rows = 0).  d_post_weight needs post_norm,
 *               d_pre_weight needs d_normed (KDA_ERR_NULL otherwise); the
 *               gradient of an absent (all ones) weight or scale may be asked for
 *   workspace   kda_block_norm_bwd_workspace_size bytes, 16-byte aligned (used
 *               for the weights' gradients only), or NULL: then a call that needs
 *               some allocates it stream-ordered
 */
kda_status kda_block_norm_bwd_workspace_size(const kda_norm_desc *desc, size_t *bytes);
kda_status kda_block_norm_bwd(const kda_norm_desc *desc, const void *y, const void *residual, const void *gate,
                              const float *post_weight, const float *scale, const float *pre_weight,
                              const void *d_out, const void *d_normed, void *d_y, void *d_residual, void *d_gate,
                              float *d_post_weight, float *d_scale, float *d_pre_weight, void *workspace,
                              size_t workspace_bytes, kda_stream_t stream);

/*
 * Norm and position rotation of queries and keys.  Per token and head, a row x
 * of d channels becomes
 *     u   = x o w / sqrt(mean x^2 + eps)              (norm; else u = x)
 *     y_a = rot_scale (u_a cos f - u_b sin f)
 *     y_b = rot_scale (u_b cos f + u_a sin f),  f = position * inv_freq[i]
 * for the rot / 2 pairs (a, b) of its first rot channels: (i, i + rot / 2) with
 * KDA_ROPE_HALF, (2i, 2i + 1) with KDA_ROPE_INTERLEAVED; the others stay, y = u.
 * Frequencies scaled for long contexts are the caller's: inv_freq holds them as
 * they are, and rot_scale is the factor on the rotated channels that goes with
 * some scalings (1 otherwise).  With rot = 0, norm and a weight of d^-1/2
 * everywhere a row is divided by its L2 norm, as the delta rule wants its q and k.
 *
 * Conventions
 *  - d is 16, 32, 64 or 128; rot a multiple of 8 from 0 to d.
 *  - q and k (outputs and gradients likewise) are [tokens, heads, d] of `dtype`
 *    with dense heads; a token's row starts `stride` elements after the one
 *    before (0: dense), so they may be parts of one projection's output.
 *    Pointers and strides are multiples of 16 bytes; a stride is at least
 *    heads * d.  Hk may be 0, without any k then.
 *  - positions are any int32 (negative ones turn backwards), inv_freq is fp32
 *    and below 2^16 in magnitude.  position * inv_freq is reduced to a part of a
 *    turn in 64-bit fixed point, to 2^-30 of a turn at any position; whole quarters
 *    of a turn are taken out before the rest is rounded to fp32, and the sine and
 *    cosine are off by 1.5 x 2^-24 at most.  Arithmetic is fp32 and each output is
 *    rounded once.
 *  - A non-finite value reaches its own row and, in the backward, the weight's
 *    gradient.  Results are deterministic.
 */
typedef enum { KDA_ROPE_HALF = 0, KDA_ROPE_INTERLEAVED = 1 } kda_rope_layout;

typedef struct {
  int tokens;
  int Hq, Hk, d;  /* heads of q (>= 1) and of k (>= 0), channels per head         */
  kda_dtype dtype;
  int rot;
  kda_rope_layout layout;
  float rot_scale;       /* finite                                                */
  int norm;              /* 1: RMSNorm of each row                                */
  float eps;             /* >= 0, used with norm                                  */
  int64_t q_stride, k_stride;         /* of q, k                                  */
  int64_t q_out_stride, k_out_stride; /* of q_out, k_out; d_q_out, d_k_out        */
  int64_t dq_stride, dk_stride;       /* of dq, dk (backward)                     */
} kda_rope_desc;

/*
 * kda_qk_rope_fwd
 *   q, k          [tokens, Hq, d], [tokens, Hk, d]
 *   positions     [tokens] int32, or NULL with rot = 0
 *   inv_freq      [rot / 2] fp32, or NULL with rot = 0
 *   q_weight, k_weight  [d] fp32, each or NULL for ones (must be NULL without norm)
 *   q_out, k_out  as q and k, written; each may be its input with the same stride
 * Outputs may overlap nothing else (KDA_ERR_ALIAS); rows of one stride that lie
 * beside each other, as the parts of one projection do, do not overlap.
 */
kda_status kda_qk_rope_fwd(const kda_rope_desc *desc, const void *q, const void *k, const int32_t *positions,
                           const float *inv_freq, const float *q_weight, const float *k_weight, void *q_out,
                           void *k_out, kda_stream_t stream);

/*
 * kda_qk_rope_bwd - gradients of L = <d_q_out, q_out> + <d_k_out, k_out>, from the
 * forward's inputs.  With g the gradient of u, r = (mean x^2 + eps)^-1/2:
 *     dx = r (g o w - x r^2 mean(g o w o x)),   dw = sum g o x r   (norm; else dx = g)
 *   dq, dk      as q and k, written; each may be d_q_out / d_k_out with the same stride
 *   dq_weight, dk_weight  [d] fp32, each or NULL: sums over tokens and heads (of
 *               absent weights too); NULL without norm
 *   workspace   kda_qk_rope_bwd_workspace_size bytes, 16-byte aligned (used for
 *               the weights' gradients only), or NULL: then a call that needs
 *               some allocates it stream-ordered
 * Without norm, q and k are not read (and may be NULL).
 */
kda_status kda_qk_rope_bwd_workspace_size(const kda_rope_desc *desc, size_t *bytes);
kda_status kda_qk_rope_bwd(const kda_rope_desc *desc, const void *q, const void *k, const int32_t *positions,
                           const float *inv_freq, const float *q_weight, const float *k_weight,
                           const void *d_q_out, const void *d_k_out, void *dq, void *dk, float *dq_weight,
                           float *dk_weight, void *workspace, size_t workspace_bytes, kda_stream_t stream);

/*
 * Softmax attention over a paged cache.  Keys and values live in pages of
 * page_size tokens; page_table[n] lists sequence n's pages in order, and
 * lens[n] is its length in tokens, the call's own new tokens included (they are
 * appended first).  New token i of the L_n that sequence n brings stands at
 * position lens[n] - L_n + i.
 *
 * Conventions shared by kda_kv_append and kda_paged_attn
 *  - k_cache, v_cache  [num_pages, Hk, page_size, d] dtype; each page is dense and
 *    starts cache_stride elements after the one before (0: dense), so that the
 *    two may be halves of one buffer.  Hq is a multiple of Hk; heads h * Hq / Hk
 *    to (h + 1) * Hq / Hk - 1 of the queries share head h of the cache.
 *  - Token tensors are as kda_qk_rope_fwd's: dense heads of 16, 32, 64 or 128
 *    channels, a stride from token to token, 16-byte aligned.
 *  - page_table [N, max_pages], lens [N], cu_seqlens [N + 1] are int32 on the
 *    device and are read there: captured calls see their values at replay.
 *    cu_seqlens NULL means B sequences of T new tokens; packed sequences may be
 *    empty, and rows behind the last one have no effect and are not written.
 *  - Entries of page_table behind a sequence's last page are not read; slots
 *    behind its length, whatever they hold, have no effect.
 *  - Validate mode returns KDA_ERR_RANGE for cu_seqlens that do not start at 0
 *    or that decrease or pass the token count, a length below 0 or above
 *    max_pages * page_size, or a used page outside [0, num_pages).  Without it
 *    they are clamped (lengths and cu_seqlens to their ranges; a token whose page is
 *    outside is not stored, and its key and value are read from the nearest
 *    page), so that no call reads or writes outside the tensors.
 *  - A position below 0 (a length below the number of new tokens, as the entries
 *    that pad a batch have with length 0) is not stored, and under the causal mask
 *    attends to nothing.  A query without any key gets zeros and a log-sum of
 *    -infinity.
 */
typedef struct {
  int B;          /* batch; must be 1 when cu_seqlens is given                   */
  int T;          /* new tokens per sequence, or of all sequences when packed     */
  int Hq, Hk, d;
  int num_seqs;   /* packed: number of sequences N; 0 when cu_seqlens is NULL      */
  int page_size, num_pages, max_pages;
  kda_dtype dtype;           /* of every token tensor and of the cache            */
  int64_t q_stride, k_stride, v_stride; /* of q, k, v                             */
  int64_t out_stride;        /* of q_out or out                                   */
  int64_t cache_stride;      /* from page to page                                 */
  int rot;                   /* kda_kv_append: the rotation and the norm of q, k, */
  kda_rope_layout layout;    /*   as kda_rope_desc's                              */
  float rot_scale;
  int norm;
  float eps;
  int causal;                /* kda_paged_attn: 1: keys up to the query's own     */
                             /*   position; 0: all lens[n] keys                   */
  float scale;               /*   on the scores; above 0, scale / ln 2 finite     */
  int validate;              /* 1: range-check first (synchronises the stream)    */
} kda_paged_desc;

/*
 * kda_kv_append - stores the new tokens' keys and values in the cache; keys are
 * normed and rotated on the way (kda_qk_rope_fwd's arithmetic, at the tokens'
 * positions), and so are the queries, where given.
 *   q             [tokens, Hq, d], or NULL
 *   k, v          [tokens, Hk, d]
 *   lens, cu_seqlens, page_table  as above (lengths after the append)
 *   inv_freq      [rot / 2] fp32, or NULL with rot = 0
 *   q_weight, k_weight  [d] fp32, each or NULL (must be NULL without norm)
 *   q_out         as q, written (given exactly when q is); may be q itself
 *   k_cache, v_cache  written at the new tokens' slots only; values are copied as
 *                 they are, bit for bit
 * Two tokens must not share a slot.
 */
kda_status kda_kv_append(const kda_paged_desc *desc, const void *q, const void *k, const void *v,
                         const int32_t *lens, const int32_t *cu_seqlens, const int32_t *page_table,
                         const float *inv_freq, const float *q_weight, const float *k_weight, void *q_out,
                         void *k_cache, void *v_cache, kda_stream_t stream);

/*
 * kda_paged_attn - attention of the new tokens (one of each sequence when
 * generating, many in a prefill, or both in one packed call) over the cache:
 *     out_i = sum_j p_ij v_j,  p_ij = exp(scale q_i . k_j - lse_i)
 *     lse_i = log sum_j exp(scale q_i . k_j)
 *   q         [tokens, Hq, d]
 *   out       [tokens, Hq, d], written
 *   lse       [tokens, Hq] fp32, or NULL (written): what joins this result to one
 *             over other keys
 *   workspace kda_paged_attn_workspace_size bytes, 16-byte aligned, not in use by
 *             another call in flight; or NULL: allocated stream-ordered
 * Scores, the softmax's maxima and sums and the output sums are fp32, the sums
 * being of probabilities relative to a row's largest, at most 1 each; bf16
 * probabilities are rounded to bf16 for their product with the values.  A
 * non-finite key or value reaches the queries that attend to it, and no others; an
 * infinite value comes out as an infinity, or as NaN where its probability or a
 * factor of the running maximum underflows (0 times infinity).
 * Results are deterministic.  Where a bounded wait inside the kernel runs out the
 * outputs are undefined, and kda_device_watchdog says so.
 */
kda_status kda_paged_attn_workspace_size(const kda_paged_desc *desc, size_t *bytes);
kda_status kda_paged_attn(const kda_paged_desc *desc, const void *q, const void *k_cache, const void *v_cache,
                          const int32_t *lens, const int32_t *cu_seqlens, const int32_t *page_table, void *out,
                          float *lse, void *workspace, size_t workspace_bytes, kda_stream_t stream);

/* Static description of a status code (never NULL). */
const char *kda_status_string(kda_status status);

/* The last CUDA error string seen by this thread's most recent failing call,
 * or "" (never NULL). */
const char *kda_last_cuda_error(void);

/* The tensor-core prefill and the tensor-core kernel of kda_paged_attn (bf16,
 * many query rows to a head of the cache) bound every wait on their internal
 * barriers (2 s).  A wait that runs out makes the kernel abandon its work,
 * release what it holds and OR a bit into a per-device word; the outputs of that
 * call, which has returned KDA_OK by then, are undefined.  This call waits for the
 * current device to go idle (cudaDeviceSynchronize), stores that word in *flags
 * (0 = no time-out since it was last cleared) and clears it when `clear` is
 * non-zero.  Bits within KDA_WATCHDOG_PREFILL are of the prefill, bits within
 * KDA_WATCHDOG_PAGED_ATTN of the attention. */
#define KDA_WATCHDOG_PREFILL 0x0f90ffffu
#define KDA_WATCHDOG_PAGED_ATTN 0x306f0000u
kda_status kda_device_watchdog(unsigned int *flags, int clear);

/* Size of the library's built-in scratch array used by kda_chunk_fwd_noalloc:
 * 32 MiB of device memory on every GPU that loads libkda.so, held until the
 * process exits. */
#define KDA_STATIC_WORKSPACE_BYTES (32u << 20)

/*
 * kda_chunk_fwd_noalloc - kda_chunk_fwd for callers that cannot allocate.
 * The paper has no counterpart: this is a property of the library, not of the
 * method.
 *
 * Some callers own every byte of device memory through their own allocator
 * (for example a serving process that reserves the GPU's memory in fixed pools
 * at start-up), or run in code paths where a device allocation could block on
 * or fail against memory pressure they do not control.  For them kda_chunk_fwd
 * is unusable whenever its planner splits long sequences, because it then
 * allocates a stream-ordered workspace, and kda_chunk_fwd_ex needs a buffer they
 * may have no way to provide.  This entry point takes the same arguments as
 * kda_chunk_fwd (with desc->validate = 0) and computes the same results, but
 * takes its workspace from a fixed array inside the library
 * (KDA_STATIC_WORKSPACE_BYTES); it never calls cudaMalloc, cudaMallocAsync,
 * cudaFree or any other allocating routine.  The caller still passes every
 * input and output buffer.
 *
 * - A call whose plan needs more scratch than KDA_STATIC_WORKSPACE_BYTES (see
 *   kda_chunk_fwd_workspace_size) returns KDA_ERR_SCRATCH_LIMIT before launching
 *   anything.  Validate mode needs an allocation and is refused with
 *   KDA_ERR_UNSUPPORTED.
 * - Every call looks up the array's address in the current device's context
 *   (cudaGetSymbolAddress, which allocates nothing), so the address stays
 *   right after that context is destroyed and created again.  The first call
 *   in a context may load the library's device code into it; make that first
 *   call before any stream capture.
 * - All calls in the process share the one array, and it keeps whatever the
 *   previous call left in it (every call writes all the scratch it reads, so
 *   nothing has to start at zero).  Calls whose work overlaps on the GPU (on
 *   different streams, or from different threads without ordering between
 *   them) race on that array and may return wrong results: order them.
 */
kda_status kda_chunk_fwd_noalloc(const kda_chunk_desc *desc, const void *q, const void *k,
                                 const void *v, const void *log_alpha, const void *beta,
                                 const float *initial_state, const int32_t *cu_seqlens, void *out,
                                 float *final_state, kda_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H_ */
