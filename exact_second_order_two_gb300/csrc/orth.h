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

// What is known of a matrix from its norm.
struct MatInfo {
  float norm, s;  // |G|_F and 1 / (norm + eps)
  float f;        // X_0 = f G 2^k: f in [1, 2)
  int k;
  // Where eps takes part, X is smaller than the stack's bound: X of step i is stored 2^e[i]
  // larger than its exponent says, A and B 2^(2 e[i]), S 2^e[i].  The result is not
  // (e[steps] = 0).
  short e[kMaxSteps + 1];
};

// The steps' polynomials, and bounds on the singular values of any matrix's X.
struct Steps {
  int n;
  float a[kMaxSteps], b[kMaxSteps], c[kMaxSteps], bound[kMaxSteps];
};

// One product for every matrix of the stack:
//   value = (alpha 2^ea sum over segments P Q^T (nn: P Q) + beta 2^eb E) f^fpow 2^shift,
// the operands, E and the result given by map and by the number of the stack's first
// matrix in it; ea and eb are the sums of e_alpha and e_beta times the matrix's exponents of
// this step and the next.
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
  int step;                     // < 0: ea = eb = 0
  signed char e_alpha[2], e_beta[2];
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
  int part;                     // split: stages of an accumulator
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

// split: sums in parts, tiles of 128 columns.
cudaError_t launch_chain(const ChainArgs& g, bool split, LaunchLog& log);

// A small matrix's steps, or their gradient, in one block (orth_small.cu).  Factors of
// each step: A = to_a acc, B = to_b acc + a_to_b A, X' = to_x acc + x_to_x X; S = to_s acc,
// T = to_t acc + s_to_t S, H' = to_h acc + h_to_h H, times what brings the norm of H to
// 2^target[step]; dY is brought to 2^target[steps].
struct SmallArgs {
  CUtensorMap x_map[2], a_map[2], b_map[2];  // kept: [step][matrix]
  const void *g, *dy;
  void* y;  // or dG
  MatInfo* info;
  int* status;
  unsigned long long wait_ns;
  int L, p, q, tall, keep;
  float eps;
  Steps steps;
  int x_terms, h_terms;                      // most of X, and of H, S and T, in a step
  int x_tiles;                               // backward: tiles of X (64 columns) held at a time
  int xt[kMaxSteps], xe[kMaxSteps];
  // a bit for each step: two terms of S and T; of H where it is added; of H in products; of B,
  // and of X in products
  unsigned two_s, two_h, two_hp, two_b;
  float to_a[kMaxSteps], to_b[kMaxSteps], a_to_b[kMaxSteps], to_x[kMaxSteps], x_to_x[kMaxSteps];
  float to_s[kMaxSteps], to_t[kMaxSteps], s_to_t[kMaxSteps], to_h[kMaxSteps], h_to_h[kMaxSteps];
  int target[kMaxSteps + 1];
};
bool small_fits(int p, int q, bool bf16);
cudaError_t launch_small(const SmallArgs& g, bool bf16, bool backward, LaunchLog& log);

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

// A sum of squares, m 2^e.  Squares are added as they are (e = 0) where their sum shows
// that none was lost, and leaves room for 1024 such sums: the others, of less than 2^-60 or more
// than 2^100, are taken again of elements times a power of two that keeps any fp32 number's
// square, and a sum of 2^36 of them, inside fp32.
struct Squares {
  float m;
  int e;
};
constexpr float kScaleSmall = 0x1p80f, kScaleLarge = 0x1p-96f;
// sum(scale): the squares of elements times the scale; the same in all threads of a block.
template <typename F>
__device__ __forceinline__ Squares squares_of(F sum) {
  Squares r = {sum(1.f), 0};
  if (r.m < 0x1p-60f) {
    r = Squares{sum(kScaleSmall), -160};
  } else if (r.m > 0x1p100f) {
    r = Squares{sum(kScaleLarge), 192};
  }
  return r;
}

// The exponent that brings a matrix with this sum of squares to a norm in
// (2^(target - 1), 2^target], or nearly; 0 for zeros and for what is not finite.  (127 at
// most, for a finite factor.)
__device__ __forceinline__ int rescaling(Squares nu2, int target) {
  if (!(nu2.m > 0.f) || nu2.m > 3.0e38f) return 0;
  int e;
  frexpf(nu2.m, &e);
  e += nu2.e;  // nu2 < 2^e
  return min(127, target - ((e + 1) >> 1));
}

// x 2^e, nearly always x.
__device__ __forceinline__ float times_pow2(float x, int e) { return e == 0 ? x : ldexpf(x, e); }

// Powers of two that are sure to lie between m and the bound (by their exponents: none
// where m is infinite or NaN).
__device__ __forceinline__ int room_below(float bound, float m) {
  const int e = (__float_as_int(bound) >> 23) - (__float_as_int(fmaxf(m, 1e-27f)) >> 23) - 1;
  return m == m && e > 0 ? e : 0;
}
// Singular values behind step i, from those before (1.01 for what is rounded on the way).
__device__ __forceinline__ float next_bound(const Steps& s, int i, float m) {
  return 1.01f * m * (fabsf(s.a[i]) + m * m * (fabsf(s.b[i]) + m * m * fabsf(s.c[i])));
}

// A matrix's scales from its sum of squares, but for those behind X_0; returns what G is
// multiplied by to be X_0's terms, stored at 2^(x_exp + e[0]).
__device__ __forceinline__ float info_of(Squares nu2, float eps, int x_exp, const Steps& steps, MatInfo& r) {
  r.norm = ldexpf(sqrtf(nu2.m), nu2.e / 2);
  r.s = 1.f / (r.norm + eps);
  r.e[0] = 0;
  if (r.s > 0.f && r.s < 3.0e38f) {
    int e;
    r.f = 2.f * frexpf(r.s, &e);  // s = f 2^(e - 1)
    r.k = e - 1;
    r.e[0] = (short)room_below(steps.bound[0], r.norm * r.s);
    // (a finite factor: only zeros, and what is lost beside a norm of 0, have a larger one)
    const int most = 127 - r.k - x_exp;
    if (r.e[0] > most) r.e[0] = (short)(most > 0 ? most : 0);
    return ldexpf(1.f, most > 0 ? r.k + x_exp + r.e[0] : 127);
  }
  // an infinite or NaN norm, or 0 and eps = 0: zeros and NaN as s G gives them
  r.f = 1.f;
  r.k = 0;
  return r.s;
}

// dG = by_h H_0 - by_g (up G), for H_0 stored at 2^exp and its product with X_0's terms: s (H_0
// - G <H_0, G> s / norm).  A zero matrix has no direction to take off.  (up = 2^k brings G to
// a norm of about 1: s s / norm alone could be past fp32's range.)
__device__ __forceinline__ void end_factors(const MatInfo& r, float dot, int exp, int x_exp, float& by_h,
                                            float& by_g, float& up) {
  const double along = r.norm > 0.f ? ldexp((double)dot, -(r.k + x_exp + r.e[0])) * r.s / r.norm : 0.0;
  const double scale = ldexp((double)r.s, -exp);
  by_h = (float)scale;
  by_g = (float)ldexp(scale * along, -r.k);
  up = ldexpf(1.f, r.k);
}
#endif

}  // namespace orth
}  // namespace fbob
