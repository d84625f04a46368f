// Internal declarations of the attention-layer operators (rotary positions,
// differential attention), next to those of internal.h.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <initializer_list>

#include "fbob.h"
#include "internal.h"

namespace fbob {

// SMs of a GB300: what these operators' launch rules are made for and measured on.
constexpr int kSms = 152;

// Profiling-event and launch-count bookkeeping around one entry point's work.
void begin_call(LaunchLog& log);
void end_call(const LaunchLog& log);
// Kernel family forced by fbob_force_path, or -1.
int forced_path();

// Differential attention after validation (see fbob_diff_shape_t).
struct DiffProblem {
  int B, H, Hk, N, d, dv;
  int bf16, causal;
  int lam_kind, lam_bf16;
  float scale;
  int G() const { return H / Hk; }
  size_t rows() const { return (size_t)B * H * N; }
};

// lam of row n of head bh = b H + h, in fp32.
struct LamArg {
  const void* p;
  int kind, bf16;
};

struct DiffWorkspace {
  int* status = nullptr;
  float* D = nullptr;        // [B, 2H, N]: D^1 and D^2 of each row (CUDA cores)
  float* scal = nullptr;     // the row scalars' blocks (tensor cores)
  float* d2 = nullptr;       // [B, H, N]: sum_j P^2_ij dP_ij, for lam's gradient
  float* partial = nullptr;  // [B, H]: its sums
  float* parts = nullptr;    // parts of dK and dV, where blocks are few
};

struct DiffTensors {
  const void *q, *k, *v;
  LamArg lam;
  // rest [B,H,N,R,dv]: P^2 V and, for bf16, what its and o's rounding left off
  // (null: not wanted)
  void *o, *rest;
  float* lse;    // [B, 2H, N]
  const void* dO;
  void *dq, *dk, *dv;
};

// ---- CUDA-core kernels: fp32 or bf16, any d and dv up to 128 -------------
size_t diff_simt_part_count(const DiffProblem& p);  // fp32 values of DiffWorkspace::parts
cudaError_t diff_simt_forward(const DiffProblem& p, const DiffTensors& t, LaunchLog& log);
cudaError_t diff_simt_backward(const DiffProblem& p, const DiffTensors& t, const DiffWorkspace& ws,
                               LaunchLog& log);

// ---- tensor-core kernels: bf16, d and dv multiples of 8 ---------------------
bool diff_tc_supported(const DiffProblem& p);
size_t diff_tc_scalar_count(const DiffProblem& p);  // fp32 values of DiffWorkspace::scal
size_t diff_tc_part_count(const DiffProblem& p);    // fp32 values of DiffWorkspace::parts
cudaError_t diff_tc_forward(const DiffProblem& p, const DiffTensors& t, const DiffWorkspace& ws,
                            LaunchLog& log);
cudaError_t diff_tc_backward(const DiffProblem& p, const DiffTensors& t, const DiffWorkspace& ws,
                             LaunchLog& log);

}  // namespace fbob
