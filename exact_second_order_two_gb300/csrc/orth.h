// What the host (orth.cu) and the chain of products (orth_chain.cu) of an
// orthogonalisation share.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "ops.h"

namespace fbob {
namespace orth {

// What is known of a matrix from its norm.
struct MatInfo {
  float norm, s;  // |G|_F and 1 / (norm + eps)
  float f;        // X_0 = f G 2^k: f in [1, 2)
  int k;
};

constexpr int kTile = 128;      // rows of a CTA's operand tiles
constexpr int kHigh = 256;      // rows of a pair's tile of a product
constexpr int kWide = 256;      // its columns, at most
constexpr int kPairs = kSms / 2;
constexpr int kDepth = 64;      // contraction elements of a stage (128-byte rows)
constexpr int kEpiWarps = 8;    // warps that finish tiles
constexpr int kGroups = 2;      // in groups of four
constexpr int kMaxSegs = 6;
constexpr int kMaxSteps = 16;
constexpr int kMaxPhases = 3 * kMaxSteps;
constexpr int kMaxMaps = 24;

// One product for every matrix of the stack:
//   value = (alpha sum over segments P Q^T (nn: P Q) + beta E) f^fpow 2^shift,
// the operands, E and the result given by map and by the number of the stack's first
// matrix in it.
struct Phase {
  unsigned char seg_a[kMaxSegs], seg_b[kMaxSegs];
  int at_a[kMaxSegs], at_b[kMaxSegs];
  int nseg, nn;
  int cols, depth;
  int sym;                      // symmetric: tiles on and below the diagonal
  int wide;                     // columns of a tile: 128 or 256
  unsigned char e_map[2], o_map[2];
  int e_terms, e_at;            // terms of E: 0 without
  int o_terms, o_at;            // of the result: 0 where it goes to the caller's tensor.  One
                                // term of a symmetric result is mirrored through o_map[1],
  __half* mirror[2];            // two terms by stores here
  int ld;
  float alpha, beta;
  int fpow;
  float* sums;                  // [count][parts of a matrix]: squares of the values, or null
  // shift: brings the norm of the phase's input, whose squares these are, to 2^target
  const float* scale_sums;
  int scale_parts, target;
  const int* exp_in;
  int* exp_out;
  int first, tiles;             // first item, tiles of a matrix
};

struct ChainArgs {
  CUtensorMap maps[kMaxMaps];
  Phase phase[kMaxPhases];
  int phases, items;
  int rows, cols, count;        // p, q of the caller's tensor, and matrices
  const MatInfo* info;
  void* y;
  int y_bf16, y_transposed, y_mapped;
  int* ticket;                  // the next item, from 0
  int* done;                    // [phase][matrix]: parts of tiles that are written, from 0
  int* status;
  unsigned long long wait_ns;
};

static_assert(sizeof(ChainArgs) <= 32000, "kernel argument budget");

inline long long tiles_of(int rows, int cols, bool sym, int wide) {  // of one matrix
  const long long tm = (rows + kHigh - 1) / kHigh, tn = (cols + wide - 1) / wide;
  return sym ? kHigh / wide * tm * (tm + 1) / 2 : tm * tn;
}

cudaError_t launch_chain(const ChainArgs& g, LaunchLog& log);

// Launches a kernel that may start while the one before it in the stream ends; it
// waits for that one's results by after_previous().
template <typename... P, typename... A>
cudaError_t launch_next(void (*kernel)(P...), dim3 grid, int threads, size_t smem, int cluster,
                        LaunchLog& log, const A&... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = dim3((unsigned)threads);
  c.dynamicSmemBytes = smem;
  c.stream = log.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  c.attrs = attr;
  c.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&c, kernel, args...);
  log.mark();
  return e;
}

#ifdef __CUDACC__
// The kernels of a call follow one another closely: each lets the next one start as soon as
// all its own blocks run, and begins to read and write when the one before is done.
__device__ __forceinline__ void let_next_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The exponent that brings a matrix with sum of squares nu2 to a norm in
// (2^(target - 1), 2^target], or nearly; 0 for zeros and for what is not finite.
__device__ __forceinline__ int rescaling(float nu2, int target) {
  if (!(nu2 > 0.f) || nu2 > 3.0e38f) return 0;
  int e;
  frexpf(nu2, &e);  // nu2 < 2^e
  return target - ((e + 1) >> 1);
}
#endif

}  // namespace orth
}  // namespace fbob
