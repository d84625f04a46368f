// Orthogonalised updates: Newton-Schulz products and their gradient.
//
// X_0 = s G, s = 1 / (|G|_F + eps), with the shorter side first (p <= q; a tall G
// is transposed on the way in and out).  A step with polynomial a x + b x^3 + c x^5:
//   A = X X^T,   B = b A + c A^2,   X' = a X + B X.
// For an upstream gradient H of X', with A and B symmetric,
//   S = H X^T + X H^T,   T = b S + c (A S + S A),   H' = a H + B H + T X,
// and at the end dG = s (H_0 - G <H_0, G> s / |G|_F).
//
// All of these are products P Q^T or P Q of matrices stored by rows, summed in one
// accumulator and finished by alpha acc + beta E: one kernel (orth_chain.cu) runs them
// all.  A, B, S and T are symmetric: only tiles on and below the diagonal are computed,
// and written in both places.  S and A S + S A are sums of a product and its transpose: as
// one accumulation [H | X] [X | H]^T they need half the tiles, too.
//
// Numbers.  Operands are fp16 with exponents chosen for each matrix, accumulation
// is fp32.  X has singular values up to M (bounded on the host from the
// polynomials), so that one power of two for all of X, A and B keeps them inside fp16's
// range, with 11 bits down to 2^-26 of the bound; a matrix that eps keeps below that bound
// is stored as many powers of two larger (300 x 400, fp32, of norm 3e-15 beside an eps of
// 1e-7: 4.9e-2 off without); H is rescaled every step by the norm
// that it was measured to have.  fp32 tensors are held as the sum of two fp16 (22 bits)
// and multiplied in three products; bf16 tensors in one.  There, a rounding error of X
// between its weak directions grows by a every step.  It reaches them through a X alone
// (B is small there, and an error of A or of B X lies in a strong direction on one side),
// so that X is kept in two terms, of which the products take the first and a X
// both, in steps whose rounding later steps would multiply by more than 16.
// (256 x 1024 of rank 16 with noise of a hundredth: 1.6e-2 of the norm off with one term,
// 2.2e-3 with two, 1.7e-3 for the result's own rounding.)  In the backward the same growth
// meets the errors of H, S and T, and S and T are factors only: they have two terms where the
// steps still to come multiply a rounding by more than 4, and products read H's second
// term where they do by more than 16.  (1024 x 1024 of rank 16 with noise of 0.3, dY among the
// strong directions: dG 1.7e-2 off with one term each, 2.4e-3 so, of which 1.7e-3 are its own
// rounding; 2.4e-3 with second terms everywhere.)
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <string.h>
#include <stdint.h>

#include "common.cuh"
#include "fbob.h"
#include "internal.h"
#include "ops.h"
#include "orth.h"
#include "tc_common.cuh"

namespace fbob {
namespace {

using namespace orth;
using tc::encode_fn;

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

__device__ __forceinline__ void split(float v, __half& hi, __half& lo) {
  hi = __float2half_rn(v);
  lo = __float2half_rn(v - __half2float(hi));
}

// ---------------------------------------------------------------------------
// Norms, packing, and the end of the gradient
// ---------------------------------------------------------------------------
constexpr int kSumThreads = 256;

// 16 aligned bytes of elements.
__device__ __forceinline__ void load_vector(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 x = *reinterpret_cast<const uint4*>(p);
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&x);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 t = __bfloat1622float2(h[k]);
    v[2 * k] = t.x;
    v[2 * k + 1] = t.y;
  }
}
__device__ __forceinline__ void load_vector(const float* p, float (&v)[4]) {
  const float4 x = *reinterpret_cast<const float4*>(p);
  v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
}
// Eight elements of which `valid` exist; `wide`: all do, at 16-byte steps.
template <typename T>
__device__ __forceinline__ void load8(const T* p, bool wide, int valid, float (&v)[8]) {
  constexpr int V = 16 / sizeof(T);
  if (wide) {
#pragma unroll
    for (int j = 0; j < 8; j += V) {
      float t[V];
      load_vector(p + j, t);
#pragma unroll
      for (int k = 0; k < V; ++k) v[j + k] = t[k];
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = k < valid ? to_f32<T>(p[k]) : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, bool wide, int valid, const float (&v)[8]) {
  if (wide) {
    alignas(16) T t[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) t[k] = from_f32<T>(v[k]);
#pragma unroll
    for (int j = 0; j < (int)sizeof(T) / 2; ++j)
      reinterpret_cast<uint4*>(p)[j] = reinterpret_cast<const uint4*>(t)[j];
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < valid) p[k] = from_f32<T>(v[k]);
  }
}
// Eight elements of a row of terms (rows are padded to eights).
__device__ __forceinline__ void load_terms(const __half* hi, const __half* lo, float (&v)[8]) {
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const __half* p = t ? lo : hi;
    if (!p) continue;
    const uint4 x = *reinterpret_cast<const uint4*>(p);
    const __half2* h = reinterpret_cast<const __half2*>(&x);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = __half22float2(h[k]);
      v[2 * k] = t ? v[2 * k] + f.x : f.x;
      v[2 * k + 1] = t ? v[2 * k + 1] + f.y : f.y;
    }
  }
}
__device__ __forceinline__ void store_terms(__half* hi, __half* lo, const float (&v)[8]) {
  alignas(16) __half h[8], l[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) split(v[k], h[k], l[k]);
  *reinterpret_cast<uint4*>(hi) = *reinterpret_cast<const uint4*>(h);
  if (lo) *reinterpret_cast<uint4*>(lo) = *reinterpret_cast<const uint4*>(l);
}

// partial[l][block] = the squares of a slice of matrix l; also clears the call's
// status word and the chain's counters, before the kernels that write them.
template <typename T>
__global__ void __launch_bounds__(kSumThreads)
    square_sums(const T* __restrict__ x, Squares* __restrict__ partial, size_t elems, int* status,
                int* counters, size_t n_counters) {
  __shared__ float sm[kSumThreads / 32];
  let_next_start();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *status = 0;
  for (size_t i = ((size_t)blockIdx.y * gridDim.x + blockIdx.x) * kSumThreads + threadIdx.x; i < n_counters;
       i += (size_t)gridDim.x * gridDim.y * kSumThreads)
    counters[i] = 0;
  x += (size_t)blockIdx.y * elems;
  const Squares r = squares_of([&](float scale) {
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    constexpr int V = 16 / sizeof(T);
    if (elems % V == 0 && (reinterpret_cast<uintptr_t>(x) & 15u) == 0) {
      const size_t chunks = elems / V, per = (chunks + gridDim.x - 1) / gridDim.x;
      const size_t first = blockIdx.x * per, last = min(chunks, first + per);
#pragma unroll 4
      for (size_t i = first + threadIdx.x; i < last; i += kSumThreads) {
        float v[V];
        load_vector(x + i * V, v);
#pragma unroll
        for (int k = 0; k < V; ++k) s[k & 3] = fmaf(v[k] * scale, v[k] * scale, s[k & 3]);
      }
    } else {
      const size_t per = (elems + gridDim.x - 1) / gridDim.x;
      const size_t first = blockIdx.x * per, last = min(elems, first + per);
      for (size_t i = first + threadIdx.x; i < last; i += kSumThreads) {
        const float v = to_f32<T>(x[i]) * scale;
        s[0] = fmaf(v, v, s[0]);
      }
    }
    const float w = warp_sum((s[0] + s[1]) + (s[2] + s[3]));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = w;
    __syncthreads();
    float t = 0.f;
    for (int k = 0; k < kSumThreads / 32; ++k) t += sm[k];
    return t;
  });
  if (threadIdx.x == 0) partial[(size_t)blockIdx.y * gridDim.x + blockIdx.x] = r;
}

__global__ void clear_status(int* status) {
  let_next_start();
  *status = 0;
}

// Sum of `parts` values, the same in every thread of the block.
__device__ __forceinline__ float parts_sum(const float* p, int parts, float* sm) {
  float s = 0.f;
  for (int i = threadIdx.x; i < parts; i += kSumThreads) s += p[i];
  s = warp_sum(s);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = s;
  __syncthreads();
  s = 0.f;
  for (int k = 0; k < kSumThreads / 32; ++k) s += sm[k];
  return s;
}

// The same of squares, of which those with the largest exponent count most.
__device__ __forceinline__ Squares parts_sum(const Squares* p, int parts, float* sm) {
  int most = -1000, least = 1000;
  for (int i = threadIdx.x; i < parts; i += kSumThreads) {
    if (p[i].m == 0.f) continue;
    most = max(most, p[i].e);
    least = min(least, p[i].e);
  }
  if (__syncthreads_or(most >= least && (most != 0 || least != 0))) {
    most = __reduce_max_sync(0xffffffffu, most);
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = (float)most;
    __syncthreads();
    for (int k = 0; k < kSumThreads / 32; ++k) most = max(most, (int)sm[k]);
  } else {
    most = 0;
  }
  float s = 0.f;
  for (int i = threadIdx.x; i < parts; i += kSumThreads)
    s += most == p[i].e || p[i].m == 0.f ? p[i].m : ldexpf(p[i].m, p[i].e - most);
  s = warp_sum(s);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = s;
  __syncthreads();
  s = 0.f;
  for (int k = 0; k < kSumThreads / 32; ++k) s += sm[k];
  return Squares{s, most};
}

struct PackArgs {
  const void* x;        // [count][m][n]
  const Squares* sums;  // [count][parts]
  int parts;
  __half *hi, *lo;     // [count][p][ld]
  int p, q, ld, tall;
  float eps;
  int target;
  Steps steps;
  // forward: the matrices' scales; backward (info null): their exponents and square sums
  MatInfo* info;
  int* exp_out;
  float* sums_out;
};

constexpr int kPack = 64;  // rows and columns of a tile of a tall matrix

// x times a power of two, in fp16 terms, the shorter side first.
template <typename T>
__global__ void __launch_bounds__(kSumThreads) pack(PackArgs a) {
  __shared__ float sm[kSumThreads / 32];
  __shared__ float tile[kPack][kPack + 1];
  const int l = blockIdx.y;
  let_next_start();
  after_previous();
  const Squares nu2 = parts_sum(a.sums + (size_t)l * a.parts, a.parts, sm);
  const bool writer = blockIdx.x == 0 && threadIdx.x == 0;
  float factor;
  if (a.info) {
    MatInfo r;
    factor = info_of(nu2, a.eps, a.target, a.steps, r);
    if (writer) {
      float m = fminf(r.norm * r.s, 1.f);  // (1 for NaN: no room)
      for (int i = 0; i < a.steps.n; ++i) {
        if (i > 0) r.e[i] = (short)room_below(a.steps.bound[i], m);
        m = next_bound(a.steps, i, m);
      }
      r.e[a.steps.n] = 0;
      a.info[l] = r;
    }
  } else {
    const int e = rescaling(nu2, a.target);
    factor = ldexpf(1.f, e);
    if (writer) {
      a.exp_out[l] = e;
      a.sums_out[l] = ldexpf(nu2.m, nu2.e + 2 * e);
    }
  }
  const T* x = static_cast<const T*>(a.x) + (size_t)l * a.p * a.q;
  const size_t base = (size_t)l * a.p * a.ld;
  const int chunks = a.ld / 8;
  if (a.tall) {  // x is [q][p]: tiles through shared memory
    const int across = (a.q + kPack - 1) / kPack, all = across * ((a.p + kPack - 1) / kPack);
    for (int t = blockIdx.x; t < all; t += gridDim.x) {
      const int r0 = t / across * kPack, c0 = t % across * kPack;  // of the packed matrix
      __syncthreads();
      for (int i = threadIdx.x; i < kPack * kPack; i += kSumThreads) {
        const int c = i / kPack, r = i % kPack;
        tile[r][c] = c0 + c < a.q && r0 + r < a.p ? to_f32<T>(x[(size_t)(c0 + c) * a.p + r0 + r]) * factor : 0.f;
      }
      __syncthreads();
      for (int i = threadIdx.x; i < kPack * kPack / 8; i += kSumThreads) {
        const int r = i / (kPack / 8), c = i % (kPack / 8) * 8;
        if (r0 + r >= a.p || c0 + c >= a.q) continue;
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = tile[r][c + k];
        const size_t at = base + (size_t)(r0 + r) * a.ld + c0 + c;
        store_terms(a.hi + at, a.lo ? a.lo + at : nullptr, v);
      }
    }
    return;
  }
  const bool wide = a.q % 8 == 0 && (reinterpret_cast<uintptr_t>(x) & 15u) == 0;
  const long long all = (long long)a.p * chunks;
#pragma unroll 2
  for (long long i = (long long)blockIdx.x * kSumThreads + threadIdx.x; i < all;
       i += (long long)gridDim.x * kSumThreads) {
    const int r = (int)(i / chunks), c = (int)(i - (long long)r * chunks) * 8;
    float v[8];
    load8(x + (size_t)r * a.q + c, wide, a.q - c, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= factor;
    const size_t at = base + (size_t)r * a.ld + c;
    store_terms(a.hi + at, a.lo ? a.lo + at : nullptr, v);
  }
}

// partial[l][block] = part of <H, X> over a slice of rows of matrix l, both in terms.
struct DotArgs {
  const __half *h[2], *x[2];  // [count][p][ld]
  float* partial;
  int p, q, ld;
};
__global__ void __launch_bounds__(kSumThreads) term_dots(DotArgs a) {
  __shared__ float sm[kSumThreads / 32];
  let_next_start();
  after_previous();
  const size_t base = (size_t)blockIdx.y * a.p * a.ld;
  const int chunks = a.ld / 8;
  const long long all = (long long)a.p * chunks, per = (all + gridDim.x - 1) / gridDim.x;
  const long long first = blockIdx.x * per, last = min(all, first + per);
  float s = 0.f;
  for (long long i = first + threadIdx.x; i < last; i += kSumThreads) {
    const int row = (int)(i / chunks), c = (int)(i - (long long)row * chunks) * 8;
    const size_t at = base + (size_t)row * a.ld + c;
    float h[8], x[8];
    load_terms(a.h[0] + at, a.h[1] ? a.h[1] + at : nullptr, h);
    load_terms(a.x[0] + at, a.x[1] ? a.x[1] + at : nullptr, x);
#pragma unroll
    for (int k = 0; k < 8; ++k)  // (the padding of a row holds anything)
      if (c + k < a.q) s = fmaf(h[k], x[k], s);
  }
  s = warp_sum(s);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    float t = 0.f;
    for (int k = 0; k < kSumThreads / 32; ++k) t += sm[k];
    a.partial[(size_t)blockIdx.y * gridDim.x + blockIdx.x] = t;
  }
}

struct EndArgs {
  const void* g;      // [count][m][n]
  void* dg;
  const __half* h[2]; // [count][p][ld]: dX_0 2^exp
  const float* dots;  // [count][parts]: <h, X_0's terms>
  int parts;
  int p, q, ld, tall, x_exp;
  const MatInfo* info;
  const int* exp;
};

// dG = s (H_0 - G <H_0, G> s / norm), as end_factors has it
template <typename T>
__global__ void __launch_bounds__(kSumThreads) end_gradient(EndArgs a) {
  __shared__ float sm[kSumThreads / 32];
  __shared__ float tile[kPack][kPack + 1];
  const int l = blockIdx.y;
  after_previous();
  const MatInfo r = a.info[l];
  const float dot = parts_sum(a.dots + (size_t)l * a.parts, a.parts, sm);
  float by_h, by_g, up;
  end_factors(r, dot, a.exp[l], a.x_exp, by_h, by_g, up);
  const size_t n = (size_t)l * a.p * a.q;
  const size_t base = (size_t)l * a.p * a.ld;
  const T* g = static_cast<const T*>(a.g) + n;
  T* dg = static_cast<T*>(a.dg) + n;
  const int chunks = a.ld / 8;
  if (a.tall) {  // g is [q][p]: tiles of h through shared memory
    const int across = (a.q + kPack - 1) / kPack, all = across * ((a.p + kPack - 1) / kPack);
    for (int t = blockIdx.x; t < all; t += gridDim.x) {
      const int r0 = t / across * kPack, c0 = t % across * kPack;  // of h
      __syncthreads();
      for (int i = threadIdx.x; i < kPack * kPack / 8; i += kSumThreads) {
        const int r = i / (kPack / 8), c = i % (kPack / 8) * 8;
        if (r0 + r >= a.p || c0 + c >= a.q) continue;
        const size_t at = base + (size_t)(r0 + r) * a.ld + c0 + c;
        float v[8];
        load_terms(a.h[0] + at, a.h[1] ? a.h[1] + at : nullptr, v);
#pragma unroll
        for (int k = 0; k < 8; ++k) tile[r][c + k] = v[k];
      }
      __syncthreads();
      for (int i = threadIdx.x; i < kPack * kPack; i += kSumThreads) {
        const int c = i / kPack, r = i % kPack;
        if (r0 + r >= a.p || c0 + c >= a.q) continue;
        const size_t at = (size_t)(c0 + c) * a.p + r0 + r;
        dg[at] = from_f32<T>(fmaf(-by_g, to_f32<T>(g[at]) * up, by_h * tile[r][c]));
      }
    }
    return;
  }
  const bool wide = a.q % 8 == 0 && ((reinterpret_cast<uintptr_t>(g) | reinterpret_cast<uintptr_t>(dg)) & 15u) == 0;
  const long long all = (long long)a.p * chunks;
#pragma unroll 2
  for (long long i = (long long)blockIdx.x * kSumThreads + threadIdx.x; i < all;
       i += (long long)gridDim.x * kSumThreads) {
    const int r = (int)(i / chunks), c = (int)(i - (long long)r * chunks) * 8;
    const size_t at = base + (size_t)r * a.ld + c, to = (size_t)r * a.q + c;
    float v[8], x[8];
    load_terms(a.h[0] + at, a.h[1] ? a.h[1] + at : nullptr, v);
    load8(g + to, wide, a.q - c, x);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = fmaf(-by_g, x[k] * up, by_h * v[k]);
    store8(dg + to, wide, a.q - c, v);
  }
}

// ---------------------------------------------------------------------------
// Host: scales, workspace, launches
// ---------------------------------------------------------------------------
struct Plan {
  int L, m, n, p, q, ldq, ldp, steps, bf16, keep, tall;
  float eps;
  float a[kMaxSteps], b[kMaxSteps], c[kMaxSteps];
  int xe[kMaxSteps], ae[kMaxSteps], be[kMaxSteps];  // exponents of X, A, B as stored
  int xt[kMaxSteps];                                // terms of X
  int st[kMaxSteps], ht[kMaxSteps];                 // of S and T, and of the H that a step takes,
  int hp[kMaxSteps];                                // in its sum and in its products
  double M[kMaxSteps];                              // bound on X's singular values
  Steps device;                                     // the same for the kernels
  int square_parts;
  // sums of products are added up in parts (orth_chain.cu)
  bool split() const { return !bf16 || q > 65536; }
};

// Columns of a product's tiles: 128 where that fills more of the GPU.  A tile costs its
// multiplications (128 columns 0.8 of what 256 do: half, less well fed), in stages of
// 64 elements, and as much as 8 stages beside them.
int choose_wide(const Plan& p, int cols, int depth, bool sym, int segs) {
  if (p.split()) return 128;  // the finishing warps hold sums of 128 columns
  double best = 0;
  int wide = 0;
  for (int w : {256, 128}) {
    const long long tiles = p.L * tiles_of(p.p, cols, sym, w);
    const double stages = (double)segs * ((depth + kDepth - 1) / kDepth);
    const double t = (double)((tiles + kPairs - 1) / kPairs) * (stages * (w == 256 ? 1.0 : 0.8) + 8);
    if (!wide || t < best) {
      best = t;
      wide = w;
    }
  }
  return wide;
}

int floor_log2(double x) { return (int)floor(log2(x)); }
int store_exp(double bound) {  // entries up to 2^15
  const int e = bound > 0 ? floor_log2(32768.0 / bound) : 12;
  return e < 12 ? e : 12;
}

int make_plan(const fbob_orth_t* o, Plan* out) {
  if (!o || !o->coefficients) return FBOB_ERR_INVALID_ARG;
  if (o->L < 1 || o->m < 1 || o->n < 1 || o->steps < 1 || (o->keep & ~1)) return FBOB_ERR_INVALID_ARG;
  if (!(o->eps >= 0.f) || o->eps > 3.0e38f) return FBOB_ERR_INVALID_ARG;
  if (o->dtype != FBOB_BF16 && o->dtype != FBOB_FP32) return FBOB_ERR_UNSUPPORTED;
  if (o->steps > kMaxSteps || o->L > 65535) return FBOB_ERR_UNSUPPORTED;
  Plan p;
  p.L = o->L; p.m = o->m; p.n = o->n;
  p.p = o->m < o->n ? o->m : o->n;
  p.q = o->m < o->n ? o->n : o->m;
  p.tall = o->m > o->n;
  // tiles and 64-wide pieces are counted in 32 bits, pieces of rows in a grid's y
  if (p.p > (1 << 16) || p.q > (1 << 22) || (double)p.L * p.p * p.q > (double)(1ll << 36))
    return FBOB_ERR_UNSUPPORTED;
  p.ldq = (p.q + 7) / 8 * 8;
  p.ldp = (p.p + 7) / 8 * 8;
  p.steps = o->steps;
  p.bf16 = o->dtype == FBOB_BF16;
  p.keep = o->keep;
  p.eps = o->eps;
  double M = 1.0, falls = 1.0;
  for (int i = 0; i < p.steps; ++i) {
    const double a = o->coefficients[3 * i], b = o->coefficients[3 * i + 1], c = o->coefficients[3 * i + 2];
    if (!(fabs(a) < 1e6 && fabs(b) < 1e6 && fabs(c) < 1e6)) return FBOB_ERR_INVALID_ARG;
    p.a[i] = (float)a; p.b[i] = (float)b; p.c[i] = (float)c;
    p.M[i] = M;
    p.xe[i] = store_exp(M);
    p.ae[i] = store_exp(M * M);
    p.be[i] = store_exp(fabs(b) * M * M + fabs(c) * M * M * M * M);
    // the polynomial's most up to M, which rounding may pass a little: at the end, or
    // where a + 3 b t + 5 c t^2 = 0, t = x^2
    const double end = 1.01 * M, root = 9 * b * b - 20 * a * c;
    double at[3] = {end, 0, 0}, most = 0;
    if (c != 0 && root >= 0) {
      at[1] = sqrt(fmax(0.0, (-3 * b + sqrt(root)) / (10 * c)));
      at[2] = sqrt(fmax(0.0, (-3 * b - sqrt(root)) / (10 * c)));
    } else if (c == 0 && b != 0) {
      at[1] = sqrt(fmax(0.0, -a / (3 * b)));
    }
    for (double x : at) {
      if (x > end) continue;
      const double y = fabs(x * (a + x * x * (b + x * x * c)));
      if (!(y <= most)) most = y;
    }
    M = 1.01 * most;
    if (!(M < 64.0)) return FBOB_ERR_INVALID_ARG;  // singular values that run away
    // exponents come from bounds: where small singular values, which go with a, fall far
    // behind those, fp16 has no digits left for them
    falls *= fmin(1.0, fabs(a));
    if (!(falls >= 1.0 / 256)) return FBOB_ERR_INVALID_ARG;
  }
  p.device.n = p.steps;
  for (int i = 0; i < p.steps; ++i) {
    p.device.a[i] = p.a[i]; p.device.b[i] = p.b[i]; p.device.c[i] = p.c[i];
    p.device.bound[i] = (float)p.M[i];
  }
  // terms of X: the growth of a rounding error by the steps that follow
  double growth = 1;
  for (int i = p.steps - 1; i >= 0; --i) {
    growth *= fabs(p.a[i]) > 1 ? fabs(p.a[i]) : 1;
    // (a bf16 G is one fp16 term, times a power of two)
    p.xt[i] = !p.bf16 || (growth > 16 && i > 0) ? 2 : 1;
  }
  growth = 1;  // by the steps that the backward takes behind step i
  for (int i = 0; i < p.steps; ++i) {
    p.st[i] = !p.bf16 || growth > 4 ? 2 : 1;
    const bool much = growth > 16;
    growth *= fabs(p.a[i]) > 1 ? fabs(p.a[i]) : 1;
    // (a bf16 dY is one fp16 term, times a power of two)
    p.ht[i] = !p.bf16 || (growth > 4 && i + 1 < p.steps) ? 2 : 1;
    p.hp[i] = !p.bf16 || (p.ht[i] == 2 && much) ? 2 : 1;
  }
  const long long elems = (long long)p.p * p.q;
  const long long parts = (elems + 8191) / 8192;
  p.square_parts = (int)(parts < 1024 ? parts : 1024);
  // items of a chain are counted in 32 bits
  const double tiles = 2.0 * tiles_of(p.p, p.p, true, 128) + (double)tiles_of(p.p, p.q, false, 128);
  if (tiles * p.L * p.steps > (double)(1 << 30)) return FBOB_ERR_UNSUPPORTED;
  *out = p;
  return FBOB_OK;
}

// A map of [count][rows][ld] elements, cols of each row; a box: 128 bytes of box_rows rows.
bool make_map(CUtensorMap* m, CUtensorMapDataType type, int size, const void* ptr, long long count, int rows,
              int cols, long long ld, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)count};
  cuuint64_t strides[2] = {(cuuint64_t)ld * size, (cuuint64_t)rows * ld * size};
  cuuint32_t box[3] = {(cuuint32_t)(128 / size), (cuuint32_t)box_rows, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return fn(m, type, 3, const_cast<void*>(ptr), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Slots of L matrices of p rows each, in one fp16 term, the first low_slots in two.
struct Mats {
  __half *hi, *lo;
  int slots, low_slots, cols, ld;
  size_t slot;              // elements
  unsigned char tile[2];    // maps in boxes of 128 rows: left operands, right ones of P Q^T, what
  unsigned char step[2];    // is added, results; and of 64 rows: right operands of P Q, mirrors
};

struct Carver {
  char* base;
  size_t off;
  void* take(size_t bytes) {
    void* r = base ? base + off : nullptr;
    off += align_up(bytes);
    return r;
  }
  Mats mats(const Plan& p, int cols, int ld, int slots, int low_slots) {
    Mats t = {};
    t.slot = (size_t)p.L * p.p * ld;
    t.hi = static_cast<__half*>(take(slots * t.slot * sizeof(__half)));
    t.lo = low_slots ? static_cast<__half*>(take(low_slots * t.slot * sizeof(__half))) : nullptr;
    t.slots = slots;
    t.low_slots = low_slots;
    t.cols = cols;
    t.ld = ld;
    return t;
  }
};

size_t counters(const Plan& p) { return 1 + (size_t)3 * p.steps * p.L; }  // ticket, done

// Forward: [status][counters][info][square sums], then X, A and B of every step (keep), or
// of two and one.
struct Forward {
  int *status, *counters;
  MatInfo* info;
  Squares* sums;
  Mats X, A, B;
  size_t bytes;
  int keep;
  int x(int i) const { return keep ? i : i & 1; }
  int a(int i) const { return keep ? i : 0; }
};
Forward carve_forward(const Plan& p, char* base) {
  Forward w;
  Carver c{base, 0};
  w.keep = p.keep;
  w.status = static_cast<int*>(c.take(sizeof(int)));
  w.counters = static_cast<int*>(c.take(sizeof(int) * counters(p)));
  w.info = static_cast<MatInfo*>(c.take(sizeof(MatInfo) * p.L));
  w.sums = static_cast<Squares*>(c.take(sizeof(Squares) * p.L * p.square_parts));
  const int xs = p.keep ? p.steps : p.steps > 1 ? 2 : 1, as = p.keep ? p.steps : 1;
  int low = 0;
  for (int i = 0; i < p.steps; ++i)
    if (p.xt[i] == 2 && w.x(i) >= low) low = w.x(i) + 1;
  w.X = c.mats(p, p.q, p.ldq, xs, low);
  w.A = c.mats(p, p.p, p.ldp, as, p.bf16 ? 0 : as);
  w.B = c.mats(p, p.p, p.ldp, as, p.bf16 ? 0 : as);
  w.bytes = c.off;
  return w;
}

// Backward: [status][counters][square sums of dY][the same of H as packed][exponents:
// steps + 1][sums of the steps' results: two in turn][<H, X>], H in turn, S, T.
struct Backward {
  int *status, *counters;
  Squares* sums;
  float *first, *step_sums[2], *dots;
  int* exp[kMaxSteps + 1];
  Mats H, S, T;
  size_t bytes;
};
int step_parts(const Plan& p, int i) {  // of the squares of B H + T X
  const int segs = p.bf16 ? p.hp[i] + p.st[i] : 6;
  return (int)tiles_of(p.p, p.q, false, choose_wide(p, p.q, p.p, false, segs)) * 2 * kEpiWarps;
}
Backward carve_backward(const Plan& p, char* base) {
  Backward w;
  Carver c{base, 0};
  int h_two = 0, s_two = 0, most = 0;
  for (int i = 0; i < p.steps; ++i) {
    if (p.ht[i] == 2) h_two = 1;
    if (p.st[i] == 2) s_two = 1;
    if (step_parts(p, i) > most) most = step_parts(p, i);
  }
  w.status = static_cast<int*>(c.take(sizeof(int)));
  w.counters = static_cast<int*>(c.take(sizeof(int) * counters(p)));
  w.sums = static_cast<Squares*>(c.take(sizeof(Squares) * p.L * p.square_parts));
  w.dots = static_cast<float*>(c.take(sizeof(float) * p.L * p.square_parts));
  w.first = static_cast<float*>(c.take(sizeof(float) * p.L));
  for (float*& s : w.step_sums) s = static_cast<float*>(c.take(sizeof(float) * p.L * most));
  for (int i = 0; i <= p.steps; ++i) w.exp[i] = static_cast<int*>(c.take(sizeof(int) * p.L));
  w.H = c.mats(p, p.q, p.ldq, 2, 2 * h_two);
  w.S = c.mats(p, p.p, p.ldp, 1, s_two);
  w.T = c.mats(p, p.p, p.ldp, 1, s_two);
  w.bytes = c.off;
  return w;
}

// A matrix (L of them) as a product takes it: a family's slot, in one or two terms.
struct Ref {
  const Mats* m;
  int slot, terms;
};

// Builds a chain, phase by phase.
struct Chain {
  ChainArgs g;
  const Plan& p;
  int maps = 0, items = 0;
  bool ok = true;
  int q_terms[kMaxSegs];
  const Mats* q_of[kMaxSegs];
  Chain(const Plan& plan, int* status, int* counts, const MatInfo* info) : p(plan) {
    g.phases = 0;
    g.rows = p.p;
    g.cols = p.q;
    g.count = p.L;
    g.info = info;
    g.y = nullptr;
    g.y_bf16 = p.bf16;
    g.y_transposed = p.tall;
    g.y_mapped = 0;
    g.status = status;
    g.ticket = counts;
    g.done = counts + 1;
    g.wait_ns = wait_limit_ns();
  }
  void use(Mats& m) {
    for (int t = 0; t < 2; ++t) {
      const int slots = t ? m.low_slots : m.slots;
      if (!slots) continue;
      const __half* at = t ? m.lo : m.hi;
      const auto half = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
      m.tile[t] = (unsigned char)maps;
      ok = ok && make_map(&g.maps[maps++], half, 2, at, (long long)slots * p.L, p.p, m.cols, m.ld, kTile);
      m.step[t] = (unsigned char)maps;
      ok = ok && make_map(&g.maps[maps++], half, 2, at, (long long)slots * p.L, p.p, m.cols, m.ld, kDepth);
    }
  }
  Phase& phase() { return g.phase[g.phases]; }
  void begin(int cols, int depth, bool nn, bool sym) {
    Phase& f = phase();
    memset(&f, 0, sizeof f);
    f.cols = cols;
    f.depth = depth;
    f.nn = nn;
    f.sym = sym;
    f.step = -1;
    f.first = items;
  }
  void pair(const Ref& P, int tp, const Ref& Q, int tq) {
    Phase& f = phase();
    f.seg_a[f.nseg] = P.m->tile[tp];
    f.at_a[f.nseg] = P.slot * p.L;
    q_terms[f.nseg] = tq;
    q_of[f.nseg] = Q.m;
    f.at_b[f.nseg++] = Q.slot * p.L;
  }
  // acc += P Q^T (or P Q): every pair of terms but the two low ones
  void add(const Ref& P, const Ref& Q) {
    if (Q.terms == 2) pair(P, 0, Q, 1);
    if (P.terms == 2) pair(P, 1, Q, 0);
    pair(P, 0, Q, 0);
  }
  // exponents of alpha and of beta for a matrix with exponents e[i], e[i + 1]
  void by_matrix(int i, int alpha0, int alpha1, int beta0, int beta1) {
    Phase& f = phase();
    f.step = i;
    f.e_alpha[0] = (signed char)alpha0;
    f.e_alpha[1] = (signed char)alpha1;
    f.e_beta[0] = (signed char)beta0;
    f.e_beta[1] = (signed char)beta1;
  }
  void plus(const Ref& E) {
    Phase& f = phase();
    f.e_terms = E.terms;
    f.e_map[0] = E.m->tile[0];
    f.e_map[1] = E.m->tile[1];
    f.e_at = E.slot * p.L;
  }
  void to(const Ref& O) {
    Phase& f = phase();
    f.o_terms = O.terms;
    f.o_map[0] = O.m->tile[0];
    f.o_map[1] = O.terms == 2 ? O.m->tile[1] : O.m->step[0];
    f.o_at = O.slot * p.L;
    f.mirror[0] = O.m->hi;
    f.mirror[1] = O.m->lo;
    f.ld = O.m->ld;
  }
  // the caller's tensor, by rows (through a map where one can be made) or transposed
  void to_caller(void* y) {
    const int size = p.bf16 ? 2 : 4;
    g.y = y;
    g.y_mapped = !p.tall && (reinterpret_cast<uintptr_t>(y) & 15u) == 0 && (long long)p.q * size % 16 == 0 &&
                 make_map(&g.maps[maps], p.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                          size, y, p.L, p.p, p.q, p.q, kTile);
    phase().o_map[0] = (unsigned char)maps++;
  }
  void end() {
    Phase& f = phase();
    f.wide = choose_wide(p, f.cols, f.depth, f.sym, f.nseg);
    f.tiles = (int)tiles_of(p.p, f.cols, f.sym, f.wide);
    // a CTA's half of the right operand's tile: 64 or 128 rows of it, or columns 64 at a time
    for (int i = 0; i < f.nseg; ++i)
      f.seg_b[i] = (f.nn || f.wide == 128 ? q_of[i]->step : q_of[i]->tile)[q_terms[i]];
    items += p.L * f.tiles;
    ++g.phases;
  }
  cudaError_t launch(LaunchLog& log) {
    if (!ok) return cudaErrorUnknown;
    g.items = items;
    // parts of 64 elements, longer where there would be more than 4096 of them to add
    g.part = p.bf16 ? 64 : 3 * ((p.q + 64 * 4096 - 1) / (64 * 4096));
    return launch_chain(g, p.split(), log);
  }
};

// Blocks of a pass over every matrix: 2048 elements (a tile of 4096 of a tall one) each,
// up to eight blocks an SM.
dim3 passes(const Plan& p) {
  const long long tiles = (long long)((p.p + kPack - 1) / kPack) * ((p.q + kPack - 1) / kPack);
  const long long n = p.tall ? tiles : ((long long)p.p * p.ldq + 2047) / 2048;
  const long long most = (8ll * kSms + p.L - 1) / p.L;
  return dim3((unsigned)(n < most ? n : most), (unsigned)p.L);
}

cudaError_t squares_and_pack(const Plan& p, const void* x, Squares* sums, int* status, int* counts,
                             PackArgs a, LaunchLog& log) {
  const size_t elems = (size_t)p.p * p.q;
  const dim3 grid((unsigned)p.square_parts, (unsigned)p.L);
  if (p.bf16)
    square_sums<<<grid, kSumThreads, 0, log.stream>>>(static_cast<const __nv_bfloat16*>(x), sums, elems, status,
                                                      counts, counters(p));
  else
    square_sums<<<grid, kSumThreads, 0, log.stream>>>(static_cast<const float*>(x), sums, elems, status, counts,
                                                      counters(p));
  cudaError_t e = cudaGetLastError();
  log.mark();
  if (e != cudaSuccess) return e;
  a.x = x;
  a.sums = sums;
  a.parts = p.square_parts;
  a.p = p.p; a.q = p.q; a.ld = p.ldq; a.tall = p.tall;
  a.eps = p.eps;
  a.steps = p.device;
  return launch_next(p.bf16 ? pack<__nv_bfloat16> : pack<float>, passes(p), kSumThreads, 0, 1, log, a);
}

float pow2(int e) { return ldexpf(1.f, e); }

// Exponents of the gradient.  A step multiplies the norm of H by growth = max |p'| over X's
// singular values at most (on blocks of singular vectors it is a divided difference of
// p, which is odd: a mean of p' between them).  H may have a norm of 2^room as step i takes
// it, so that every entry of H, S (stored at 2^se), T and H' is below 2^15, whatever their
// directions.  What step i is to scale its H' by comes from the norm of its own H:
// that is brought to 2^target[i], and H' by growth further; dY to 2^target[steps].
void backward_scales(const Plan& p, int* target, int* se) {
  double after = 15;  // the room of what step i makes: the caller's gradient is past all products
  for (int i = 0; i < p.steps; ++i) {
    const double M = p.M[i], a = p.a[i], b = p.b[i], c = p.c[i], end = 1.01 * M * 1.01 * M;
    double growth = fmax(1.0, fmax(fabs(a), fabs(a + end * (3 * b + end * 5 * c))));
    const double middle = c != 0 ? -3 * b / (10 * c) : -1;
    if (middle > 0 && middle < end) growth = fmax(growth, fabs(a + middle * (3 * b + middle * 5 * c)));
    const double t = (fabs(b) + 2 * fabs(c) * M * M) * 2 * M;
    // (T of the first step is stored times f < 2)
    const double by_t = (i > 0 ? 15 : 14) - log2(t > 1e-30 ? t : 1e-30) - (p.be[i] - p.xe[i]);
    const double room = fmin(12.0, fmin(15 - log2(growth), by_t));
    target[i] = (int)floor(fmin(12.0, after - log2(growth)));
    se[i] = store_exp(exp2(room) * 2 * M);
    after = room;
  }
  target[p.steps] = (int)floor(after);
}

// A call for small matrices: one launch, and one that clears the status word.
cudaError_t small(const Plan& p, const void* G, const void* dY, void* out, Forward& f, int* status,
                  LaunchLog& log) {
  SmallArgs g = {};
  g.g = G;
  g.dy = dY;
  g.y = out;
  g.info = f.info;
  g.status = status;
  g.wait_ns = wait_limit_ns();
  g.L = p.L; g.p = p.p; g.q = p.q; g.tall = p.tall; g.keep = p.keep;
  g.eps = p.eps;
  g.steps = p.device;
  int se[kMaxSteps];
  backward_scales(p, g.target, se);
  g.x_terms = g.h_terms = 1;
  for (int i = 0; i < p.steps; ++i) {
    const int te = p.be[i] - p.xe[i], out_exp = i + 1 < p.steps ? p.xe[i + 1] : 0;
    if (p.ht[i] == 2 || p.st[i] == 2) g.h_terms = 2;
    double left = 1;  // what small singular values still grow by
    for (int j = i; j < p.steps; ++j) left *= fabs(p.a[j]) > 1 ? fabs(p.a[j]) : 1;
    const bool two = !p.bf16 || left <= 64;
    g.two_b |= (unsigned)two << i;
    g.xt[i] = !p.bf16 || (two && i > 0) ? 2 : p.xt[i];  // (a bf16 X_0 is one term)
    if (g.xt[i] == 2) g.x_terms = 2;
    g.two_s |= (unsigned)(p.st[i] == 2) << i;
    g.two_h |= (unsigned)(p.ht[i] == 2) << i;
    g.two_hp |= (unsigned)(p.hp[i] == 2) << i;
    g.xe[i] = p.xe[i];
    g.to_a[i] = pow2(p.ae[i] - 2 * p.xe[i]);
    g.to_b[i] = p.c[i] * pow2(p.be[i] - 2 * p.ae[i]);
    g.a_to_b[i] = p.b[i] * pow2(p.be[i] - p.ae[i]);
    g.to_x[i] = pow2(out_exp - p.be[i] - p.xe[i]);
    g.x_to_x[i] = p.a[i] * pow2(out_exp - p.xe[i]);
    g.to_s[i] = pow2(se[i] - p.xe[i]);
    g.to_t[i] = p.c[i] * pow2(te - p.ae[i] - se[i]);
    g.s_to_t[i] = p.b[i] * pow2(te - se[i]);
    g.to_h[i] = pow2(-p.be[i]);
    g.h_to_h[i] = p.a[i];
  }
  const auto half = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const Mats* from[3] = {&f.X, &f.A, &f.B};
  CUtensorMap* maps[3] = {g.x_map, g.a_map, g.b_map};
  for (int k = 0; p.keep && k < 3; ++k)
    for (int t = 0; t < 2; ++t) {
      const int slots = t ? from[k]->low_slots : from[k]->slots;
      if (slots && !make_map(&maps[k][t], half, 2, t ? from[k]->lo : from[k]->hi, (long long)slots * p.L, p.p,
                             from[k]->cols, from[k]->ld, kTile))
        return cudaErrorUnknown;
    }
  // (in the stream's order: no block of the kernel clears it behind another's report.  A memset
  // would have to be over before the kernel starts: 2 us of 22.)
  clear_status<<<1, 1, 0, log.stream>>>(status);
  const cudaError_t e = cudaGetLastError();
  log.mark();
  return e == cudaSuccess ? launch_small(g, p.bf16, dY != nullptr, log) : e;
}

cudaError_t forward(const Plan& p, const void* G, void* Y, Forward& w, LaunchLog& log) {
  if (small_fits(p.p, p.q, p.bf16)) return small(p, G, nullptr, Y, w, w.status, log);
  Chain c(p, w.status, w.counters, w.info);
  c.use(w.X);
  c.use(w.A);
  c.use(w.B);
  const int terms = p.bf16 ? 1 : 2;
  for (int i = 0; i < p.steps; ++i) {
    const Ref X{&w.X, w.x(i), p.xt[i]}, Xm{&w.X, w.x(i), terms};  // as it is added, and multiplied
    const Ref A{&w.A, w.a(i), terms}, B{&w.B, w.a(i), terms};
    const bool last = i + 1 == p.steps;
    c.begin(p.p, p.q, false, true);
    c.add(Xm, Xm);
    c.phase().alpha = pow2(p.ae[i] - 2 * p.xe[i]);
    c.phase().fpow = i == 0 ? 2 : 0;
    c.to(A);
    c.end();
    c.begin(p.p, p.p, false, true);
    c.add(A, A);
    c.plus(A);
    c.phase().alpha = p.c[i] * pow2(p.be[i] - 2 * p.ae[i]);
    c.phase().beta = p.b[i] * pow2(p.be[i] - p.ae[i]);
    c.by_matrix(i, -2, 0, 0, 0);
    c.to(B);
    c.end();
    c.begin(p.q, p.p, true, false);
    c.add(B, Xm);
    c.plus(X);
    const int out = last ? 0 : p.xe[i + 1];
    c.phase().alpha = pow2(out - p.be[i] - p.xe[i]);
    c.phase().beta = p.a[i] * pow2(out - p.xe[i]);
    c.phase().fpow = i == 0 ? 1 : 0;
    c.by_matrix(i, -3, 1, -1, 1);
    if (last) c.to_caller(Y);
    else c.to(Ref{&w.X, w.x(i + 1), p.xt[i + 1]});
    c.end();
  }
  if (!c.ok) return cudaErrorUnknown;
  PackArgs a = {};
  a.hi = w.X.hi;
  a.lo = p.xt[0] == 2 ? w.X.lo : nullptr;
  a.target = p.xe[0];
  a.info = w.info;
  const cudaError_t e = squares_and_pack(p, G, w.sums, w.status, w.counters, a, log);
  return e == cudaSuccess ? c.launch(log) : e;
}

cudaError_t backward(const Plan& p, const void* G, const void* dY, void* dG, Forward& f, Backward& w,
                     LaunchLog& log) {
  if (small_fits(p.p, p.q, p.bf16)) return small(p, G, dY, dG, f, w.status, log);
  int target[kMaxSteps + 1], se[kMaxSteps];
  backward_scales(p, target, se);
  const int top = p.steps - 1, terms = p.bf16 ? 1 : 2;
  Chain c(p, w.status, w.counters, f.info);
  for (Mats* m : {&f.X, &f.A, &f.B, &w.H, &w.S, &w.T}) c.use(*m);
  const float* sums = w.first;
  int parts = 1, turn = 0;
  for (int i = top; i >= 0; --i, turn ^= 1) {
    const Ref H{&w.H, turn, p.ht[i]}, Hm{&w.H, turn, p.hp[i]};  // as it is added, and multiplied
    const Ref X{&f.X, i, terms}, A{&f.A, i, terms}, B{&f.B, i, terms};
    const Ref S{&w.S, 0, p.st[i]}, T{&w.T, 0, p.st[i]};
    const int by_f = i == 0 ? 1 : 0;  // X_0 is f times what is stored
    c.begin(p.p, p.q, false, true);
    c.add(Hm, X);
    c.add(X, Hm);
    c.phase().alpha = pow2(se[i] - p.xe[i]);
    c.phase().fpow = by_f;
    c.to(S);
    c.end();
    // T X and B H share an accumulator: T is stored 2^e[i] larger, as S and X are
    const int te = p.be[i] - p.xe[i];
    c.begin(p.p, p.p, false, true);
    c.add(A, S);
    c.add(S, A);
    c.plus(S);
    c.phase().alpha = p.c[i] * pow2(te - p.ae[i] - se[i]);
    c.phase().beta = p.b[i] * pow2(te - se[i]);
    c.phase().fpow = by_f;
    c.by_matrix(i, -2, 0, 0, 0);
    c.to(T);
    c.end();
    c.begin(p.q, p.p, true, false);
    c.add(B, Hm);
    c.add(T, X);
    c.plus(H);
    Phase& h = c.phase();
    h.alpha = pow2(-p.be[i]);
    h.beta = p.a[i];
    c.by_matrix(i, -2, 0, 0, 0);
    h.sums = i > 0 ? w.step_sums[turn] : nullptr;
    h.scale_sums = sums;
    h.scale_parts = parts;
    h.target = target[i];
    h.exp_in = w.exp[i + 1];
    h.exp_out = w.exp[i];
    c.to(Ref{&w.H, turn ^ 1, i > 0 ? p.ht[i - 1] : terms});
    c.end();
    sums = w.step_sums[turn];
    parts = step_parts(p, i);
  }
  if (!c.ok) return cudaErrorUnknown;
  PackArgs a = {};
  a.hi = w.H.hi;
  a.lo = p.bf16 ? nullptr : w.H.lo;
  a.target = target[p.steps];
  a.exp_out = w.exp[p.steps];
  a.sums_out = w.first;
  cudaError_t e = squares_and_pack(p, dY, w.sums, w.status, w.counters, a, log);
  if (e == cudaSuccess) e = c.launch(log);
  if (e != cudaSuccess) return e;
  DotArgs d = {};
  d.h[0] = w.H.hi + turn * w.H.slot;
  d.h[1] = p.bf16 ? nullptr : w.H.lo + turn * w.H.slot;
  d.x[0] = f.X.hi;
  d.x[1] = p.xt[0] == 2 ? f.X.lo : nullptr;
  d.partial = w.dots;
  d.p = p.p; d.q = p.q; d.ld = p.ldq;
  e = launch_next(term_dots, dim3((unsigned)p.square_parts, (unsigned)p.L), kSumThreads, 0, 1, log, d);
  if (e != cudaSuccess) return e;
  EndArgs n = {};
  n.g = G;
  n.dg = dG;
  n.h[0] = d.h[0];
  n.h[1] = d.h[1];
  n.dots = w.dots;
  n.parts = p.square_parts;
  n.p = p.p; n.q = p.q; n.ld = p.ldq; n.tall = p.tall; n.x_exp = p.xe[0];
  n.info = f.info;
  n.exp = w.exp[0];
  return launch_next(p.bf16 ? end_gradient<__nv_bfloat16> : end_gradient<float>, passes(p), kSumThreads, 0, 1,
                     log, n);
}

// Makes the device's context current in a thread that is new to the GPU (autograd's
// are), as making tensor maps needs.
bool enter() {
  int dev;
  return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess;
}

bool off(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

}  // namespace
}  // namespace fbob

using namespace fbob;

extern "C" {

size_t fbob_orth_workspace_size(int op, const fbob_orth_t* o) {
  Plan p;
  if (op != FBOB_OP_FORWARD && op != FBOB_OP_BACKWARD) return 0;
  if (make_plan(o, &p) != FBOB_OK) return 0;
  return op == FBOB_OP_FORWARD ? carve_forward(p, nullptr).bytes : carve_backward(p, nullptr).bytes;
}

int fbob_orth_forward(const fbob_orth_t* o, const void* g, void* y, void* ws, size_t ws_bytes,
                      void* stream) {
  Plan p;
  const int st = make_plan(o, &p);
  if (st != FBOB_OK) return st;
  const size_t size = p.bf16 ? 2 : 4;
  if (!g || !y || !ws || off(g, size) || off(y, size) || off(ws, 256)) return FBOB_ERR_INVALID_ARG;
  if (ws_bytes < carve_forward(p, nullptr).bytes) return FBOB_ERR_WORKSPACE;
  if (!enter()) return FBOB_ERR_CUDA;
  Forward w = carve_forward(p, static_cast<char*>(ws));
  LaunchLog log{static_cast<cudaStream_t>(stream)};
  begin_call(log);
  const cudaError_t e = forward(p, g, y, w, log);
  end_call(log);
  return e == cudaSuccess ? FBOB_OK : FBOB_ERR_CUDA;
}

int fbob_orth_backward(const fbob_orth_t* o, const void* g, const void* dy, void* dg, const void* kept,
                       size_t kept_bytes, void* ws, size_t ws_bytes, void* stream) {
  Plan p;
  const int st = make_plan(o, &p);
  if (st != FBOB_OK) return st;
  const size_t size = p.bf16 ? 2 : 4;
  if (!p.keep || !g || !dy || !dg || !kept || !ws || off(g, size) || off(dy, size) || off(dg, size) ||
      off(kept, 256) || off(ws, 256))
    return FBOB_ERR_INVALID_ARG;
  if (kept_bytes < carve_forward(p, nullptr).bytes || ws_bytes < carve_backward(p, nullptr).bytes)
    return FBOB_ERR_WORKSPACE;
  if (!enter()) return FBOB_ERR_CUDA;
  Forward f = carve_forward(p, const_cast<char*>(static_cast<const char*>(kept)));
  Backward w = carve_backward(p, static_cast<char*>(ws));
  LaunchLog log{static_cast<cudaStream_t>(stream)};
  begin_call(log);
  const cudaError_t e = backward(p, g, dy, dg, f, w, log);
  end_call(log);
  return e == cudaSuccess ? FBOB_OK : FBOB_ERR_CUDA;
}

}  // extern "C"
