// Differential attention: entry points (validation, workspace, choice of the
// kernel family), the row scalars of its backward and the gradient of lam.
//
// D^m_i = dO_i . O^m_i comes from the saved O = O^1 - lam O^2 and O^2:
// D^2 = dO . O^2 and D^1 = dO . O + lam D^2.  With both rounded to bf16 the
// roundings would reach every dS of the row (and more so where the maps nearly
// cancel: with 16 keys and lam = 1 the gradients of q and k had 1.8 times the
// error of their own rounding, with 2048 keys 1.49 times); so what they left off
// is kept beside them, and the scalars are as good as fp32 (1.42 to 1.5 times,
// from dS as a bf16 operand).  lam's gradient, dlam_i = -D^2_i, is summed over
// what shares a value of lam (per head, or over everything): the pass that
// computes dQ sums P^2_ij dP_ij over j in fp32, the same number from unrounded
// factors, and the sums here add them up in a fixed order.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "fbob.h"
#include "internal.h"
#include "ops.h"

namespace fbob {
namespace {

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool given(std::initializer_list<const void*> ps) {
  for (const void* q : ps)
    if (!q || !aligned(q, 16)) return false;
  return true;
}

int check_shape(const fbob_diff_shape_t* s, DiffProblem* out) {
  if (!s) return FBOB_ERR_INVALID_ARG;
  if (s->B < 1 || s->H < 1 || s->Hk < 1 || s->N < 1 || s->d < 1 || s->dv < 1 || s->H % s->Hk)
    return FBOB_ERR_INVALID_ARG;
  if (s->causal != 0 && s->causal != 1) return FBOB_ERR_INVALID_ARG;
  // (the kernels take scale log2 e, which is finite then)
  if (!(s->scale > 0.f) || s->scale > 2.0e38f) return FBOB_ERR_INVALID_ARG;
  if (s->lam_kind < FBOB_LAM_ONE || s->lam_kind > FBOB_LAM_ROW) return FBOB_ERR_INVALID_ARG;
  for (int dt : {s->dtype, s->lam_dtype})
    if (dt != FBOB_BF16 && dt != FBOB_FP32) return FBOB_ERR_UNSUPPORTED;
  if (s->d > 128 || s->dv > 128) return FBOB_ERR_UNSUPPORTED;
  // 2 B H maps, within the 65,535 heads of the other calls; N leaves room for a
  // tile past the end
  if ((long long)s->B * s->H > 32767 || s->N > (1 << 30)) return FBOB_ERR_UNSUPPORTED;
  if ((double)s->B * s->H * s->N * 128.0 > (double)(1ll << 40)) return FBOB_ERR_UNSUPPORTED;
  *out = DiffProblem{s->B, s->H, s->Hk, s->N, s->d, s->dv, s->dtype == FBOB_BF16, s->causal,
                     s->lam_kind, s->lam_dtype == FBOB_BF16, s->scale};
  return FBOB_OK;
}

int choose_path(const DiffProblem& p) {
  const bool tc = diff_tc_supported(p);
  if (forced_path() == FBOB_PATH_SIMT) return FBOB_PATH_SIMT;
  if (forced_path() == FBOB_PATH_TCGEN05) return tc ? FBOB_PATH_TCGEN05 : -1;
  return tc ? FBOB_PATH_TCGEN05 : FBOB_PATH_SIMT;
}

// [status 256 B][D: B*2H*N fp32, or the tensor cores' row scalars][d2: B*H*N
// fp32][partial: B*H fp32][parts of dK and dV], each region aligned
size_t carve(int op, const DiffProblem& p, int path, char* base, DiffWorkspace* ws) {
  size_t off = kAlign;
  if (ws) ws->status = reinterpret_cast<int*>(base);
  if (op == FBOB_OP_BACKWARD) {
    if (ws) ws->D = ws->scal = reinterpret_cast<float*>(base + off);
    off += align_up((path == FBOB_PATH_TCGEN05 ? diff_tc_scalar_count(p) : 2 * p.rows()) * sizeof(float));
    if (ws) ws->d2 = reinterpret_cast<float*>(base + off);
    off += align_up(p.rows() * sizeof(float));
    if (ws) ws->partial = reinterpret_cast<float*>(base + off);
    off += align_up((size_t)p.B * p.H * sizeof(float));
    if (ws) ws->parts = reinterpret_cast<float*>(base + off);
    off += align_up((path == FBOB_PATH_TCGEN05 ? diff_tc_part_count(p) : diff_simt_part_count(p)) *
                    sizeof(float));
  }
  return off;
}

__device__ __forceinline__ float lam_load(const LamArg& l, size_t i) {
  return l.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(l.p)[i])
                : static_cast<const float*>(l.p)[i];
}
__device__ __forceinline__ void lam_store(void* p, int bf16, size_t i, float x) {
  if (bf16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(x);
  else static_cast<float*>(p)[i] = x;
}

// D^1 and D^2 of every row, one warp per row.
template <typename T>
__global__ void __launch_bounds__(256)
    diff_row_scalars(const T* __restrict__ o, const T* __restrict__ rest, const T* __restrict__ dO,
                     LamArg lam, float* __restrict__ D, size_t rows, int H, int N, int dv) {
  constexpr int R = sizeof(T) == 2 ? 3 : 1;
  const size_t row = (size_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= rows) return;
  float s1 = 0.f, s2 = 0.f;
  for (int c = lane; c < dv; c += 32) {
    const float g = to_f32<T>(dO[row * dv + c]);
    float out = to_f32<T>(o[row * dv + c]), o2 = to_f32<T>(rest[row * R * dv + c]);
    if (R == 3) {
      o2 += to_f32<T>(rest[(row * R + 1) * dv + c]);
      out += to_f32<T>(rest[(row * R + 2) * dv + c]);
    }
    s1 = fmaf(g, out, s1);
    s2 = fmaf(g, o2, s2);
  }
  s1 = warp_sum(s1);
  s2 = warp_sum(s2);
  if (lane != 0) return;
  const size_t bh = row / N, n = row - bh * N;
  const size_t at = lam.kind == FBOB_LAM_ONE ? 0 : lam.kind == FBOB_LAM_HEAD ? bh % H : row;
  D[(bh * 2 + 0) * N + n] = fmaf(lam_load(lam, at), s2, s1);
  D[(bh * 2 + 1) * N + n] = s2;
}

__device__ __forceinline__ float block_sum(float v, float* sm) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  v = threadIdx.x < blockDim.x / 32 ? sm[threadIdx.x] : 0.f;
  return threadIdx.x < 32 ? warp_sum(v) : 0.f;
}

// dlam per row
__global__ void __launch_bounds__(256)
    diff_lam_rows(const float* __restrict__ d2, void* dlam, int bf16, size_t rows) {
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i < rows) lam_store(dlam, bf16, i, -d2[i]);
}

// dlam per head (a block each), or of the one value, in a single launch: for as
// many rows as a block adds up in a few us
constexpr long long kOneBlock = 65536;
__global__ void __launch_bounds__(1024)
    diff_lam_sums(const float* __restrict__ d2, void* dlam, int bf16, int kind, int B, int H, int N) {
  __shared__ float sm[32];
  float s = 0.f;
  if (kind == FBOB_LAM_HEAD) {
    for (int b = 0; b < B; ++b) {
      const float* rows = d2 + ((size_t)b * H + blockIdx.x) * N;
      for (int i = threadIdx.x; i < N; i += 1024) s += rows[i];
    }
  } else {
    const int rows = B * H * N;
    for (int i = threadIdx.x; i < rows; i += 1024) s += d2[i];
  }
  s = block_sum(s, sm);
  if (threadIdx.x == 0) lam_store(dlam, bf16, blockIdx.x, -s);
}

// partial[b, h] = sum over rows of d2: one block per (batch, head)
__global__ void __launch_bounds__(256)
    diff_head_sums(const float* __restrict__ d2, float* __restrict__ partial, int N) {
  __shared__ float sm[8];
  d2 += (size_t)blockIdx.x * N;
  float s = 0.f;
  for (int i = threadIdx.x; i < N; i += 256) s += d2[i];
  s = block_sum(s, sm);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// dlam per head (sum over the batch), or of the one value (sum over all)
__global__ void __launch_bounds__(256)
    diff_lam_grad(const float* __restrict__ partial, void* dlam, int bf16, int kind, int B, int H) {
  __shared__ float sm[8];
  if (kind == FBOB_LAM_HEAD) {
    for (int h = threadIdx.x; h < H; h += 256) {
      float s = 0.f;
      for (int b = 0; b < B; ++b) s += partial[(size_t)b * H + h];
      lam_store(dlam, bf16, h, -s);
    }
    return;
  }
  float s = 0.f;
  for (int i = threadIdx.x; i < B * H; i += 256) s += partial[i];
  s = block_sum(s, sm);
  if (threadIdx.x == 0) lam_store(dlam, bf16, 0, -s);
}

template <typename T>
cudaError_t row_scalars(const DiffProblem& p, const DiffTensors& t, const DiffWorkspace& ws,
                        LaunchLog& log) {
  const size_t rows = p.rows();
  diff_row_scalars<T><<<(unsigned)((rows + 7) / 8), 256, 0, log.stream>>>(
      static_cast<const T*>(t.o), static_cast<const T*>(t.rest), static_cast<const T*>(t.dO), t.lam,
      ws.D, rows, p.H, p.N, p.dv);
  const cudaError_t e = cudaGetLastError();
  log.mark();
  return e;
}

cudaError_t lam_gradient(const DiffProblem& p, const DiffWorkspace& ws, void* dlam, LaunchLog& log) {
  cudaError_t e;
  if (p.lam_kind == FBOB_LAM_ROW) {
    diff_lam_rows<<<(unsigned)((p.rows() + 255) / 256), 256, 0, log.stream>>>(ws.d2, dlam, p.lam_bf16,
                                                                              p.rows());
    e = cudaGetLastError();
    log.mark();
    return e;
  }
  const bool head = p.lam_kind == FBOB_LAM_HEAD;
  if ((head ? (long long)p.B * p.N : (long long)p.rows()) <= kOneBlock) {
    diff_lam_sums<<<head ? p.H : 1, 1024, 0, log.stream>>>(ws.d2, dlam, p.lam_bf16, p.lam_kind, p.B,
                                                           p.H, p.N);
    e = cudaGetLastError();
    log.mark();
    return e;
  }
  diff_head_sums<<<p.B * p.H, 256, 0, log.stream>>>(ws.d2, ws.partial, p.N);
  e = cudaGetLastError();
  log.mark();
  if (e != cudaSuccess) return e;
  diff_lam_grad<<<1, 256, 0, log.stream>>>(ws.partial, dlam, p.lam_bf16, p.lam_kind, p.B, p.H);
  e = cudaGetLastError();
  log.mark();
  return e;
}

// Common prologue: validate, pick the path, carve the workspace, reset the
// status word (in a thread new to the GPU also what makes its context current).
int prologue(int op, const fbob_diff_shape_t* shape, void* ws_ptr, size_t ws_bytes,
             cudaStream_t stream, DiffProblem* p, int* path, DiffWorkspace* ws) {
  const int st = check_shape(shape, p);
  if (st != FBOB_OK) return st;
  *path = choose_path(*p);
  if (*path < 0) return FBOB_ERR_UNSUPPORTED;
  if (!ws_ptr || !aligned(ws_ptr, 16)) return FBOB_ERR_INVALID_ARG;
  if (ws_bytes < carve(op, *p, *path, static_cast<char*>(ws_ptr), ws)) return FBOB_ERR_WORKSPACE;
  return cudaMemsetAsync(ws->status, 0, sizeof(int), stream) == cudaSuccess ? FBOB_OK : FBOB_ERR_CUDA;
}

}  // namespace
}  // namespace fbob

using namespace fbob;

extern "C" {

size_t fbob_diff_workspace_size(int op, const fbob_diff_shape_t* shape) {
  DiffProblem p;
  if (op != FBOB_OP_FORWARD && op != FBOB_OP_BACKWARD) return 0;
  if (check_shape(shape, &p) != FBOB_OK) return 0;
  const int path = choose_path(p);
  return path < 0 ? 0 : carve(op, p, path, nullptr, nullptr);
}

int fbob_diff_path(int op, const fbob_diff_shape_t* shape) {
  DiffProblem p;
  if (op != FBOB_OP_FORWARD && op != FBOB_OP_BACKWARD) return -1;
  if (check_shape(shape, &p) != FBOB_OK) return -1;
  return choose_path(p);
}

int fbob_diff_forward(const fbob_diff_shape_t* shape, const void* q, const void* k, const void* v,
                      const void* lam, void* o, void* rest, float* lse, void* ws_ptr,
                      size_t ws_bytes, void* stream) {
  DiffProblem p;
  int path;
  DiffWorkspace ws;
  LaunchLog log{static_cast<cudaStream_t>(stream)};
  if (!given({q, k, v, o, lse}) || !aligned(rest, 16) || !lam) return FBOB_ERR_INVALID_ARG;
  const int st = prologue(FBOB_OP_FORWARD, shape, ws_ptr, ws_bytes, log.stream, &p, &path, &ws);
  if (st != FBOB_OK) return st;
  if (!aligned(lam, p.lam_bf16 ? 2 : 4)) return FBOB_ERR_INVALID_ARG;
  DiffTensors t{};
  t.q = q; t.k = k; t.v = v; t.o = o; t.rest = rest; t.lse = lse;
  t.lam = LamArg{lam, p.lam_kind, p.lam_bf16};
  begin_call(log);
  const cudaError_t e = path == FBOB_PATH_TCGEN05 ? diff_tc_forward(p, t, ws, log)
                                                  : diff_simt_forward(p, t, log);
  end_call(log);
  return e == cudaSuccess ? FBOB_OK : FBOB_ERR_CUDA;
}

int fbob_diff_backward(const fbob_diff_shape_t* shape, const void* q, const void* k, const void* v,
                       const void* lam, const void* o, const void* rest, const float* lse,
                       const void* dO, void* dq, void* dk, void* dv, void* dlam, void* ws_ptr,
                       size_t ws_bytes, void* stream) {
  DiffProblem p;
  int path;
  DiffWorkspace ws;
  LaunchLog log{static_cast<cudaStream_t>(stream)};
  if (!given({q, k, v, o, rest, lse, dO, dq, dk, dv}) || !lam || !dlam) return FBOB_ERR_INVALID_ARG;
  const int st = prologue(FBOB_OP_BACKWARD, shape, ws_ptr, ws_bytes, log.stream, &p, &path, &ws);
  if (st != FBOB_OK) return st;
  const size_t la = p.lam_bf16 ? 2 : 4;
  if (!aligned(lam, la) || !aligned(dlam, la)) return FBOB_ERR_INVALID_ARG;
  DiffTensors t{};
  t.q = q; t.k = k; t.v = v; t.dO = dO;
  t.o = const_cast<void*>(o);
  t.rest = const_cast<void*>(rest);
  t.lse = const_cast<float*>(lse);
  t.dq = dq; t.dk = dk; t.dv = dv;
  t.lam = LamArg{lam, p.lam_kind, p.lam_bf16};
  begin_call(log);
  cudaError_t e;
  if (path == FBOB_PATH_TCGEN05) {
    e = diff_tc_backward(p, t, ws, log);
  } else {
    e = p.bf16 ? row_scalars<__nv_bfloat16>(p, t, ws, log) : row_scalars<float>(p, t, ws, log);
    if (e == cudaSuccess) e = diff_simt_backward(p, t, ws, log);
  }
  if (e == cudaSuccess) e = lam_gradient(p, ws, dlam, log);
  end_call(log);
  return e == cudaSuccess ? FBOB_OK : FBOB_ERR_CUDA;
}

}  // extern "C"
