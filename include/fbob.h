/*
 * fbob.h - C ABI of the GB300 FlashBoB library (libfbob.so).
 *
 * FlashBoB ("FlashBoB: I/O-Efficient Exact Backward-over-Backward for Softmax
 * Attention", Abstract) computes the exact backward-over-backward (BoB) of
 * softmax attention without writing any N x N tensor to device memory.  This
 * library exposes that computation and the two calls it builds on:
 *
 *   fbob_forward   O = softmax(c Q K^T) V and the row log-sum-exp LSE
 *                  (the FlashAttention forward the abstract builds on)
 *   fbob_backward  dQ, dK, dV of <dO, O>          (the first backward)
 *   fbob_bob       the gradient of L = <gQ,dQ> + <gK,dK> + <gV,dV> with
 *                  respect to Q, K, V and dO       (the BoB, Abstract)
 *
 * Conventions shared by every call
 * --------------------------------
 *  - Layout: every [B,H,N,d] tensor is dense and row-major (d fastest), of
 *    the call's dtype; LSE and the row scalars are fp32 [B,H,N].  Device
 *    pointers must be 16-byte aligned.  Outputs must not alias inputs.
 *  - Masking: with causal != 0 key j is visible to query i iff j <= i
 *    (square, top-left aligned).  The scale c is passed in shape->scale
 *    (1/sqrt(d) is the usual choice) and is a constant, not differentiated.
 *  - Derivative convention: O and LSE are the forward's outputs for the same
 *    Q, K, V (not independent inputs); BoB is the total derivative.
 *  - Ownership: the caller owns every buffer, including the workspace `ws`
 *    of at least fbob_workspace_size() bytes.  The library allocates and
 *    frees nothing.
 *  - Asynchrony: every call only enqueues work on `stream` (a cudaStream_t,
 *    or NULL for the legacy default stream) and returns.  The return value
 *    reports errors detected on the host (bad arguments, launch failures).
 *    Device-side failures (a bounded wait that ran out) are recorded in the
 *    workspace's status word and read back with fbob_status().
 *  - Threading: calls are re-entrant as long as concurrent calls use distinct
 *    workspaces.  The process-wide settings (fbob_force_path,
 *    fbob_set_profile_events) are not synchronised.
 *  - Supported shapes: N >= 1, B*H <= 65535.  fp32: 1 <= d <= 128, computed
 *    on CUDA cores.  bf16: 1 <= d <= 128; d = 64 and d = 128 run the
 *    tensor-core (tcgen05) kernels, other d run on CUDA cores.
 */
#ifndef FBOB_H_
#define FBOB_H_

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { FBOB_BF16 = 0, FBOB_FP32 = 1 } fbob_dtype_t;

typedef enum {
  FBOB_OK = 0,
  FBOB_ERR_INVALID_ARG = 1, /* null pointer, misalignment, bad size/flag    */
  FBOB_ERR_UNSUPPORTED = 2, /* shape or dtype outside the supported set     */
  FBOB_ERR_WORKSPACE = 3,   /* ws_bytes smaller than fbob_workspace_size()  */
  FBOB_ERR_CUDA = 4,        /* a CUDA runtime call or launch failed         */
  FBOB_ERR_TIMEOUT = 5      /* a device-side bounded wait ran out           */
} fbob_status_t;

typedef enum {
  FBOB_OP_FORWARD = 0,
  FBOB_OP_BACKWARD = 1,
  FBOB_OP_BOB = 2
} fbob_op_t;

/* Kernel family that serves a call (see fbob_path). */
typedef enum { FBOB_PATH_SIMT = 0, FBOB_PATH_TCGEN05 = 1 } fbob_path_t;

/* Problem description.  B batches x H heads of length-N sequences with head
 * dimension d; dtype is an fbob_dtype_t; causal is 0 or 1; scale is the
 * factor c in S = c Q K^T. */
typedef struct {
  int B, H, N, d;
  int dtype;
  int causal;
  float scale;
} fbob_shape_t;

/* Bytes of workspace that `op` needs for `shape` (0 if the shape is invalid).
 * The workspace holds a status word, the fp32 row scalars and, on the
 * tensor-core path, an fp32 [B,H,N,d] accumulator for dQ / gradQ. */
size_t fbob_workspace_size(int op, const fbob_shape_t* shape);

/* Forward: O = softmax(c Q K^T) V and LSE_i = log sum_j exp(c Q_i.K_j).
 *   q, k, v : [B,H,N,d] inputs            o : [B,H,N,d] output
 *   lse     : [B,H,N] fp32 output (natural log, scaled scores)
 * FlashAttention forward, cited as the base of FlashBoB (Abstract). */
int fbob_forward(const fbob_shape_t* shape, const void* q, const void* k,
                 const void* v, void* o, float* lse, void* ws,
                 size_t ws_bytes, void* stream);

/* First backward of attention for upstream gradient dO:
 *   D = rowsum(dO * O), dS = P * (dO V^T - D),
 *   dQ = c dS K,  dK = c dS^T Q,  dV = P^T dO.
 *   q, k, v, o, dO : [B,H,N,d] inputs; lse : [B,H,N] fp32 from fbob_forward
 *   dq, dk, dv     : [B,H,N,d] outputs
 * The "first backward pass" of the FlashBoB abstract. */
int fbob_backward(const fbob_shape_t* shape, const void* q, const void* k,
                  const void* v, const void* o, const float* lse,
                  const void* dO, void* dq, void* dk, void* dv, void* ws,
                  size_t ws_bytes, void* stream);

/* Backward-over-backward: given cotangents gQ, gK, gV on the first
 * backward's outputs dQ, dK, dV, returns the gradient of
 *   L = <gQ,dQ> + <gK,dK> + <gV,dV>
 * with respect to Q, K, V and dO (gradq, gradk, gradv, graddo).
 *   q, k, v, o, dO, gq, gk, gv : [B,H,N,d] inputs
 *   lse                        : [B,H,N] fp32 from fbob_forward
 *   gradq, gradk, gradv, graddo: [B,H,N,d] outputs (fully overwritten)
 * Any of gq, gk, gv may be NULL: that cotangent is zero (a loss that reads
 * only some of dQ, dK, dV).  The kernels then skip its loads and the MMAs
 * it feeds.  With all three NULL, L = 0 and the four outputs are zeroed.
 * Exact BoB, "FlashBoB: I/O-Efficient Exact Backward-over-Backward for
 * Softmax Attention", Abstract: two row-wise scalars per query (r and sigma,
 * reduced in a row-stationary pass) determine every output through affine
 * maps, which a second, key-stationary pass applies.  No N x N tensor is
 * written. */
int fbob_bob(const fbob_shape_t* shape, const void* q, const void* k,
             const void* v, const void* o, const float* lse, const void* dO,
             const void* gq, const void* gk, const void* gv, void* gradq,
             void* gradk, void* gradv, void* graddo, void* ws,
             size_t ws_bytes, void* stream);

/* Size of the fixed device scratch array behind fbob_bob_noalloc: 32 MiB. */
#define FBOB_NOALLOC_SCRATCH_BYTES (32u << 20)

/* fbob_bob for callers that cannot allocate device memory.
 *
 * The paper has no counterpart to this call.  It exists for callers that are
 * handed only their input and output buffers: plugin or custom-operator
 * hosts that give a kernel no allocator and no workspace, and code that must
 * not call cudaMalloc / cudaFree, which can stall the whole device or fail
 * when a caching allocator already holds the free memory.  Arguments and
 * results are those of fbob_bob without `ws` / `ws_bytes`; this call itself
 * allocates nothing.
 *
 * Scratch comes from one array of FBOB_NOALLOC_SCRATCH_BYTES in the
 * library's device memory, which every GPU that loads the library keeps
 * reserved until the process exits.  The first call on a device (with that
 * device current) looks up the array's device address; make that first call
 * before any stream capture.  Problems whose fbob_workspace_size(
 * FBOB_OP_BOB, shape) exceeds FBOB_NOALLOC_SCRATCH_BYTES are rejected with
 * FBOB_ERR_WORKSPACE (the tensor-core path needs about B*H*N*(d+3)*4 bytes,
 * i.e. at most about 125,000 rows B*H*N at d = 64 or 63,000 at d = 128; the
 * CUDA-core path needs about B*H*N*12 bytes).  All calls share the one
 * array, so calls that can overlap on the GPU (different streams, or host
 * threads) race on it: serialise them.  Each call clears what must start at
 * zero, so contents left by an earlier call do not affect the result.  The
 * status word that device-side bounded waits write lives in that array:
 * read it with fbob_noalloc_status(), not fbob_status().  The array's
 * address is kept for the life of the process, so calls after a device
 * reset (cudaDeviceReset) are not supported. */
int fbob_bob_noalloc(const fbob_shape_t* shape, const void* q, const void* k,
                     const void* v, const void* o, const float* lse,
                     const void* dO, const void* gq, const void* gk,
                     const void* gv, void* gradq, void* gradk, void* gradv,
                     void* graddo, void* stream);

/* Status of the last fbob_bob_noalloc call on the current device: synchronises
 * `stream` (the stream that call used), then returns the first device-side
 * error it recorded in the scratch array's status word (FBOB_OK if none), or
 * FBOB_ERR_CUDA if the stream reports an error or the array cannot be reached.
 * Like fbob_bob_noalloc, it has no counterpart in the paper. */
int fbob_noalloc_status(void* stream);

/* Synchronises `stream`, then returns the first error recorded in the
 * workspace's status word by the last call that used `ws` (FBOB_OK if none),
 * or FBOB_ERR_CUDA if the stream itself reports an error. */
int fbob_status(const void* ws, void* stream);

/* Static description of a status code. */
const char* fbob_strerror(int code);

/* Kernel family (fbob_path_t) that serves `op` for `shape`, or -1 if the
 * shape is not supported. */
int fbob_path(int op, const fbob_shape_t* shape);

/* Process-wide override of the kernel family: -1 = automatic (default),
 * FBOB_PATH_SIMT = always CUDA cores.  Forcing FBOB_PATH_TCGEN05 on a shape
 * it cannot serve makes calls return FBOB_ERR_UNSUPPORTED.  Returns the
 * previous setting.  Intended for tests and benchmarks. */
int fbob_force_path(int path);

/* Benchmark hook.  With count >= 1, later fbob_bob / fbob_backward /
 * fbob_forward calls record events[0] before their first kernel and
 * events[m] after their m-th kernel (m < count), on the call's stream.
 * `events` are cudaEvent_t created by the caller; pass count = 0 to turn
 * the hook off.  Returns FBOB_OK or FBOB_ERR_INVALID_ARG. */
int fbob_set_profile_events(void* const* events, int count);

/* Process-wide limit, in nanoseconds, of one device-side bounded wait in the
 * tensor-core kernels (default 2 s, far above any legitimate wait).  A wait
 * that runs out records FBOB_ERR_TIMEOUT in the call's status word; every
 * role of that thread block then stops early (those of fbob_diff_* stop
 * loading, and run to their end without waiting), waits (with a fixed 100 ms
 * limit of its own) for the copies and MMAs it has in flight, and exits, and
 * the call's outputs are undefined.  The limit is checked each time the
 * waiting thread wakes, at least every 10 us.  ns = 0 restores the default;
 * 1 <= ns <= 6e10 sets it.
 * Applies to calls enqueued afterwards.  Returns the previous limit, or -1
 * (nothing changed) for a value out of range.  Not synchronised. */
long long fbob_set_wait_limit(long long ns);

/* Number of kernels the last enqueued call launched (for launch counting). */
int fbob_last_launch_count(void);

/* Failure-detection self-test: launches one block that waits, with the same
 * bounded wait the tensor-core kernels use, on a barrier that nothing ever
 * completes, giving up after `limit_us` microseconds (1..10^6) and recording
 * FBOB_ERR_TIMEOUT in the status word of `ws` (>= 256 bytes).  The GPU is
 * never hung.  Read the result with fbob_status(). */
int fbob_selftest_wait_timeout(void* ws, size_t ws_bytes, int limit_us,
                               void* stream);

/* ------------------------------------------------------------------------
 * Rotary positions
 * ------------------------------------------------------------------------
 * The first rotary_dim features of each row are pairs; the pair (a, b) with
 * frequency inv_freq[i] of the row at position p becomes
 *   magnitude * (a cos t - b sin t, a sin t + b cos t),  t = p inv_freq[i],
 * and the remaining features are copied.  Pair i holds features 2i, 2i + 1
 * when interleaved, i and i + rotary_dim / 2 otherwise.  inverse != 0 negates
 * t: the backward of the call (the map is linear), with the same magnitude.
 * Whole turns drop out exactly, so far positions keep their angles: the
 * error is p 2^-63 turns.  Frequencies are finite and below 2^40 in magnitude.
 *
 * x and y are [B,H,N,d] with feature stride 1 and strides over batch, head
 * and position in elements (so a projection's [B,N,H,d] output can be read in
 * place), each FBOB_BF16 or FBOB_FP32; y must not overlap x.  Arithmetic is
 * fp32, rounded once.  d <= 1024, H <= 65535, B*H*N*d <= 2^38. */
typedef struct {
  int B, H, N, d;
  int rotary_dim;          /* even, 0 <= rotary_dim <= d                     */
  int interleaved;         /* 0 or 1                                         */
  int inverse;             /* 0 or 1                                         */
  int in_dtype, out_dtype; /* fbob_dtype_t of x and y                        */
  float magnitude;
  long long x_strides[3], y_strides[3]; /* batch, head, position             */
  long long pos_stride;    /* elements between the batches of `positions`    */
  long long offset;        /* position of row 0 where `positions` is NULL    */
} fbob_rotary_t;

/* y = rotary(x).  inv_freq: rotary_dim / 2 fp64 frequencies in radians per
 * position, on the device.  positions: int64 on the device, row n of batch b
 * at [b * pos_stride + n], or NULL for positions offset + n. */
int fbob_rotary(const fbob_rotary_t* r, const void* x, const double* inv_freq,
                const long long* positions, void* y, void* stream);

/* ------------------------------------------------------------------------
 * Differential attention
 * ------------------------------------------------------------------------
 * Per head h of H, two softmax maps over the same values and their weighted
 * difference:
 *   P^m = softmax(c Q^m K^mT),  m = 1, 2,   O = P^1 V - lam P^2 V.
 * Layouts, all dense and row-major: q [B,2H,N,d] with Q^1, Q^2 of head h as
 * heads 2h, 2h + 1; k [B,2Hk,N,d] likewise; v [B,Hk,N,dv]; o, dO
 * [B,H,N,dv]; lse [B,2H,N] fp32; rest [B,H,N,R,dv], R = 1 for fp32: P^2 V, and
 * R = 3 for bf16: P^2 V, what its rounding left off, and what o's rounding
 * left off.  H is a multiple of Hk: query head h reads key head h / (H / Hk).
 * lam is one value, [H], or [B,H,N], bf16 or fp32.  Masking, ownership,
 * asynchrony and alignment as above (lam to its own size); 0 < scale <= 2e38.
 * 1 <= d, dv <= 128, B*H <= 32767.  bf16 at d and dv that are multiples of 8
 * runs the tensor-core kernels, the rest runs on CUDA cores (fbob_diff_path).
 * Scores, softmax statistics and sums are fp32 in both; the tensor-core kernels
 * take P, P^1 - lam P^2 and dS as bf16 operands of the second products, the
 * CUDA-core kernels keep them in fp32.
 * Every output is summed in a fixed order: equal inputs give equal bits. */
typedef enum { FBOB_LAM_ONE = 0, FBOB_LAM_HEAD = 1, FBOB_LAM_ROW = 2 } fbob_lam_t;

typedef struct {
  int B, H, Hk, N, d, dv;
  int dtype;               /* fbob_dtype_t of q, k, v and every [..,dv]      */
  int causal;              /* 0 or 1                                         */
  int lam_kind, lam_dtype; /* fbob_lam_t, fbob_dtype_t                       */
  float scale;
} fbob_diff_shape_t;

/* Bytes of workspace that `op` (FBOB_OP_FORWARD or FBOB_OP_BACKWARD) needs
 * for `shape`, 0 if it is invalid; and the kernel family that serves it, or
 * -1.  The workspace's status word is read with fbob_status(). */
size_t fbob_diff_workspace_size(int op, const fbob_diff_shape_t* shape);
int fbob_diff_path(int op, const fbob_diff_shape_t* shape);

/* o = O and lse = the log-sum-exp of both maps' rows.  rest is what else the
 * backward reads, or NULL where no backward follows. */
int fbob_diff_forward(const fbob_diff_shape_t* shape, const void* q, const void* k, const void* v,
                      const void* lam, void* o, void* rest, float* lse, void* ws, size_t ws_bytes,
                      void* stream);

/* Gradients of <dO, O>: with dP = dO V^T, D^m = rowsum(dO * P^m V),
 *   dS^1 = P^1 * (dP - D^1),  dS^2 = -lam P^2 * (dP - D^2),
 *   dQ^m = c dS^m K^m,  dK^m = c dS^mT Q^m,  dV = (P^1 - lam P^2)^T dO,
 *   dlam = -D^2 summed over the rows that share a value.
 * dk and dv sum over the query heads that share a key head.  dlam has lam's
 * shape and dtype. */
int fbob_diff_backward(const fbob_diff_shape_t* shape, const void* q, const void* k,
                       const void* v, const void* lam, const void* o, const void* rest,
                       const float* lse, const void* dO, void* dq, void* dk, void* dv, void* dlam,
                       void* ws, size_t ws_bytes, void* stream);

/* Library ABI version (major*100 + minor). */
int fbob_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FBOB_H_ */
