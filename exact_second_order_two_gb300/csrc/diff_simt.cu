// CUDA-core kernels of differential attention: fp32 tensors, and bf16 with
// head sizes that are no multiples of 8.  Per head, with m = 1, 2,
//   S^m = c Q^m K^mT, P^m = softmax(S^m), O = P^1 V - lam P^2 V;
//   dP = dO V^T, D^m = dO . O^m, dS^1 = P^1*(dP - D^1),
//   dS^2 = -lam P^2*(dP - D^2), dQ^m = c dS^m K^m, dK^m = c dS^mT Q^m,
//   dV = (P^1 - lam P^2)^T dO, dlam_i = -sum_j P^2_ij dP_ij.
//
// Arithmetic is fp32 throughout.  A group of 8 x 16 threads holds a 32-row
// tile (queries, or keys for dK and dV) against 64-row tiles of the other side
// in shared memory; thread (ty, tx) computes the 4 x 4 scores of rows 4 ty.. and
// columns tx + 16 j.  A row of scores lives in 16 lanes of one warp, so row
// maxima and sums are shuffles, and the probabilities pass to their product
// through shared memory inside the warp.  The floor is FFMA issue, at 8 FFMA per
// 16-byte shared-memory read; with one or two warps per scheduler latency counts
// more, so several groups share a stationary tile: in the forward one per map,
// which read the same values; and where shared memory allows (SPLIT = 2) twice
// as many, which take every other streamed tile with tiles of their own, and
// add up at the end.  Everything a row accumulates is summed by one block in a
// fixed order; a key's sums too, or by one block per part (col_parts), with the
// parts added in their order.
//
// Measured, fp32, d = 64: forward at 4 heads x 2049 tokens, dv = 128, causal
// 208 us (31 TFLOP/s; 254 us with both maps in one group and two groups), dQ 249,
// dK and dV 320; at 2 x 8 heads x 4096 tokens, dv = 64 1.86 ms (2.39), 2.90 and
// 3.45 ms.
#include <cuda_bf16.h>
#include <math.h>

#include "common.cuh"
#include "diff_rows.h"
#include "internal.h"
#include "ops.h"

namespace fbob {
namespace {

constexpr int kM = 32;       // rows of the stationary tile
constexpr int kT = 64;       // rows of a streamed tile
constexpr int kThreads = 128;  // of a group
constexpr int kLdp = kT + 4;  // row stride of the score tile

// Row stride of a [64][width] tile in floats: whole 16-byte steps, and rows
// shifted by four banks against one another.
__host__ __device__ inline int ld_of(int width) {
  const int w = (width + 3) / 4 * 4;
  return (w % 32 == 0 || w % 8 == 0) ? w + 4 : w;
}

// Floats of one group's area: `tiles`, or the sums it hands over at the end
// (`sums` per thread).
__host__ __device__ inline int group_floats(int tiles, int sums) {
  return tiles > sums * kThreads ? tiles : sums * kThreads;
}

struct Args {
  const void *q, *k, *v, *dO;
  void *o, *rest, *dq, *dk, *dv;
  float* lse;
  const float* D;
  float* d2;
  float* parts;  // [gridDim.y][heads][N][2 d + dv]: partial dK^1, dK^2, dV
  LamArg lam;
  int H, G, N, d, dv_, causal;
  int heads;  // of the grid: B H, or B Hk
  float scale;
};

__device__ __forceinline__ float lam_at(const LamArg& l, int H, int N, int b, int h, int n) {
  const size_t i = l.kind == 0 ? 0 : l.kind == 1 ? (size_t)h : ((size_t)b * H + h) * N + n;
  return l.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(l.p)[i])
                : static_cast<const float*>(l.p)[i];
}

// Rows row0.. of src [N][width] into dst [ROWS][ld]; rows past N and the
// columns up to the next multiple of four read as zero.  fp32 rows of whole
// 16-byte steps go by asynchronous copies, which the caller awaits
// (loads_done) before its barrier.
template <int ROWS, typename T>
__device__ __forceinline__ void load_rows(int tid, float* dst, int ld, const T* src, int row0, int N,
                                          int width) {
  const int w4 = (width + 3) / 4;
  const bool whole = (width & 3) == 0;
  const int sh = 32 - __clz(w4 - 1);  // a row takes 2^sh threads (w4 <= 32)
  for (int e = tid; e < ROWS << sh; e += kThreads) {
    const int r = e >> sh, c = (e & ((1 << sh) - 1)) * 4;
    if (c >= width) continue;
    const bool in = row0 + r < N;
    const T* p = src + (size_t)(in ? row0 + r : 0) * width + c;
    float* d = dst + r * ld + c;
    if (sizeof(T) == 4 && whole) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(d)), "l"(p),
                   "r"(in ? 16 : 0)
                   : "memory");
      continue;
    }
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
    if (in && sizeof(T) == 2 && whole) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v.x));
      const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v.y));
      f = make_float4(a.x, a.y, b.x, b.y);
    } else if (in) {
      f.x = to_f32<T>(p[0]);
      if (c + 1 < width) f.y = to_f32<T>(p[1]);
      if (c + 2 < width) f.z = to_f32<T>(p[2]);
      if (c + 3 < width) f.w = to_f32<T>(p[3]);
    }
    *reinterpret_cast<float4*>(d) = f;
  }
}
__device__ __forceinline__ void loads_done() {
  asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
}

// fp32 pairs: one instruction, each half rounded as the scalar form is
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

// s[i][j] = sum_c A[4 ty + i][c] B[tx + 16 j][c]
__device__ __forceinline__ void tile_dot(float (&s)[4][4], const float* A, const float* B, int ld,
                                         int width, int ty, int tx) {
  float2 acc[4][4];  // sums over even and odd pairs of c
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = make_float2(0.f, 0.f);
  const float* a0 = A + 4 * ty * ld;
  const float* b0 = B + tx * ld;
#pragma unroll 4
  for (int c = 0; c < width; c += 4) {
    float4 a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(a0 + i * ld + c);
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(b0 + 16 * j * ld + c);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = fma2({a[i].x, a[i].y}, {b[j].x, b[j].y}, acc[i][j]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = fma2({a[i].z, a[i].w}, {b[j].z, b[j].w}, acc[i][j]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = acc[i][j].x + acc[i][j].y;
}

// acc[i][4 g + e] += sum_k P[4 ty + i][k] X[k][4 tx + 64 g + e], over the
// column groups g that hold some of the width's columns.
template <int NG>
__device__ __forceinline__ void tile_add(float (&acc)[4][4 * NG], const float* P, const float* X,
                                         int ld, int width, int ty, int tx) {
  const float* p0 = P + 4 * ty * kLdp;
#pragma unroll 4
  for (int k = 0; k < kT; k += 4) {
    float4 p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4*>(p0 + i * kLdp + k);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const int col = 4 * tx + 64 * g;
      if (col < width) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float4 x = *reinterpret_cast<const float4*>(X + (k + u) * ld + col);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float w = u == 0 ? p[i].x : u == 1 ? p[i].y : u == 2 ? p[i].z : p[i].w;
            float2* a = reinterpret_cast<float2*>(&acc[i][4 * g]);
            a[0] = fma2({w, w}, {x.x, x.y}, a[0]);
            a[1] = fma2({w, w}, {x.z, x.w}, a[1]);
          }
        }
      }
    }
  }
}

// The warp's own rows of the score tile: written, and visible to its product.
__device__ __forceinline__ void put_tile(float* P, const float (&s)[4][4], int ty, int tx) {
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) P[(4 * ty + i) * kLdp + tx + 16 * j] = s[i][j];
  __syncwarp();
}

template <typename T, int NG>
__device__ __forceinline__ void store_rows(T* dst, const float (&acc)[4][4 * NG], float mul, int row0,
                                           int N, int width, int stride, int ty, int tx) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = row0 + 4 * ty + i;
    if (r >= N) continue;
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = 4 * tx + 64 * g + e;
        if (c < width) dst[(size_t)r * stride + c] = from_f32<T>(mul * acc[i][4 * g + e]);
      }
  }
}

// What rounding to T leaves off.
template <typename T, int NG>
__device__ __forceinline__ void left_off(float (&acc)[4][4 * NG]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < 4 * NG; ++e) acc[i][e] -= to_f32<T>(from_f32<T>(acc[i][e]));
}

// A group's threads only (the block's, where there is one group)
template <int SPLIT>
__device__ __forceinline__ void group_sync(int grp) {
  if constexpr (SPLIT == 1) __syncthreads();
  else asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "n"(kThreads) : "memory");
}

__device__ __forceinline__ float row16_max(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float row16_sum(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Floats of one pair's area: its tiles, or what it hands over at the end.
__host__ __device__ inline int fwd_area(int d, int dv) {
  const int tiles = kT * (2 * ld_of(d) + ld_of(dv)) + 2 * kM * kLdp;
  const int sums = (16 * (dv <= 64 ? 1 : 2) + 8) * 2 * kThreads;
  return tiles > sums ? tiles : sums;
}

// ---- forward: one block per 32 query rows of a head, a group of threads per
// map; SPLIT = 2: two such pairs of groups take every other key tile, and the
// first adds up --------------------------------------------------------------
template <typename T, int NGV, int SPLIT>
__global__ void __launch_bounds__(SPLIT * 2 * kThreads, 2 / SPLIT) diff_fwd(Args a) {
  extern __shared__ __align__(16) float sm[];
  const int ld = ld_of(a.d), ldv = ld_of(a.dv_), N = a.N;
  const int m = threadIdx.x / kThreads % 2, tid = threadIdx.x % kThreads;
  const int half = threadIdx.x / (2 * kThreads);
  const int ty = tid >> 4, tx = tid & 15;
  float* qs = sm + m * kM * ld;                    // [2][32][ld]
  float* pair = sm + 2 * kM * ld;                  // the pair's area
  const int area = fwd_area(a.d, a.dv_);
  const float* other = pair + area;                // the second pair's, for the first
  if (half == 1) pair += area;
  float* ks = pair + m * kT * ld;                  // [2][64][ld]
  float* vs = pair + 2 * kT * ld;                  // [64][ldv]
  float* ps = vs + kT * ldv + m * kM * kLdp;       // [2][32][kLdp]
  // barrier of the pair
  auto pair_sync = [&] {
    if constexpr (SPLIT == 1) __syncthreads();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + half), "n"(2 * kThreads) : "memory");
  };
  // heads vary fastest, and the long rows of all of them start first
  const int bh = blockIdx.x % a.heads, b = bh / a.H, h = bh % a.H;
  const int kvh = b * (a.H / a.G) + h / a.G;
  const int blk = blockIdx.x / a.heads;
  const int row0 = (a.causal ? (int)(gridDim.x / a.heads) - 1 - blk : blk) * kM;
  const size_t qsz = (size_t)N * a.d;
  const T* q = static_cast<const T*>(a.q) + ((size_t)bh * 2 + m) * qsz;
  const T* k = static_cast<const T*>(a.k) + ((size_t)kvh * 2 + m) * qsz;
  const T* v = static_cast<const T*>(a.v) + (size_t)kvh * N * a.dv_;
  if (half == 0) load_rows<kM>(tid, qs, ld, q, row0, N, a.d);
  if (SPLIT > 1) {
    loads_done();
    __syncthreads();
  }

  float acc[4][4 * NGV], mx[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    mx[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int e = 0; e < 4 * NGV; ++e) acc[i][e] = 0.f;
  }
  const int kend = a.causal ? min(N, row0 + kM) : N;
  for (int j0 = half * kT; j0 < kend; j0 += SPLIT * kT) {
    pair_sync();
    load_rows<kT>(tid, ks, ld, k, j0, N, a.d);
    load_rows<kT / 2>(tid, vs + m * (kT / 2) * ldv, ldv, v, j0 + m * (kT / 2), N, a.dv_);
    loads_done();
    pair_sync();
    float s[4][4];
    tile_dot(s, qs, ks, ld, a.d, ty, tx);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = row0 + 4 * ty + i;
      float t = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int col = j0 + tx + 16 * j;
        s[i][j] = (col < N && (!a.causal || col <= r)) ? s[i][j] * a.scale : -INFINITY;
        t = fmaxf(t, s[i][j]);
      }
      // A row that has seen no key yet (the second pair's at the diagonal; keys
      // of infinite features) keeps a maximum of -inf: it counts as 0 then, and
      // every term and sum stays 0
      t = fmaxf(mx[i], row16_max(t));
      const float ref = t == -INFINITY ? 0.f : t;
      const float alpha = expf(mx[i] - ref);
      mx[i] = t;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = expf(s[i][j] - ref);
        sum += s[i][j];
      }
      l[i] = l[i] * alpha + row16_sum(sum);
#pragma unroll
      for (int e = 0; e < 4 * NGV; ++e) acc[i][e] *= alpha;
    }
    put_tile(ps, s, ty, tx);
    tile_add<NGV>(acc, ps, vs, ldv, a.dv_, ty, tx);
  }
  if constexpr (SPLIT > 1) {
    // the second pair hands over; the first combines against the joint maximum
    constexpr int S = 2 * kThreads;
    const int at = m * kThreads + tid;
    pair_sync();
    if (half == 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int e = 0; e < 4 * NGV; ++e) pair[(i * 4 * NGV + e) * S + at] = acc[i][e];
        pair[(16 * NGV + i) * S + at] = mx[i];
        pair[(16 * NGV + 4 + i) * S + at] = l[i];
      }
    }
    __syncthreads();
    if (half == 1) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float m2 = other[(16 * NGV + i) * S + at];
      const float top = fmaxf(mx[i], m2);
      const float f1 = expf(mx[i] - top), f2 = expf(m2 - top);
      mx[i] = top;
      l[i] = l[i] * f1 + other[(16 * NGV + 4 + i) * S + at] * f2;
#pragma unroll
      for (int e = 0; e < 4 * NGV; ++e)
        acc[i][e] = acc[i][e] * f1 + other[(i * 4 * NGV + e) * S + at] * f2;
    }
  }
  const size_t ob = (size_t)bh * N * a.dv_;
  constexpr int R = sizeof(T) == 2 ? 3 : 1;
  T* rest = static_cast<T*>(a.rest) + R * ob;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = row0 + 4 * ty + i;
    const float inv = 1.f / l[i];
#pragma unroll
    for (int e = 0; e < 4 * NGV; ++e) acc[i][e] *= inv;
    if (r < N && tx == 0 && a.lse) a.lse[((size_t)bh * 2 + m) * N + r] = mx[i] + logf(l[i]);
  }
  pair_sync();
  if (m == 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4 * NGV; ++e) pair[(i * 4 * NGV + e) * kThreads + tid] = acc[i][e];
  }
  pair_sync();
  if (m == 1) {
    if (!a.rest) return;
    store_rows<T, NGV>(rest, acc, 1.f, row0, N, a.dv_, R * a.dv_, ty, tx);
    if constexpr (R == 3) {
      left_off<T, NGV>(acc);
      store_rows<T, NGV>(rest + a.dv_, acc, 1.f, row0, N, a.dv_, R * a.dv_, ty, tx);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = row0 + 4 * ty + i;
    const float w = r < N ? lam_at(a.lam, a.H, N, b, h, r) : 0.f;
#pragma unroll
    for (int e = 0; e < 4 * NGV; ++e) acc[i][e] -= w * pair[(i * 4 * NGV + e) * kThreads + tid];
  }
  store_rows<T, NGV>(static_cast<T*>(a.o) + ob, acc, 1.f, row0, N, a.dv_, a.dv_, ty, tx);
  if constexpr (R == 3) {
    if (!a.rest) return;
    left_off<T, NGV>(acc);
    store_rows<T, NGV>(rest + 2 * a.dv_, acc, 1.f, row0, N, a.dv_, R * a.dv_, ty, tx);
  }
}

// ---- dQ: one block per 32 query rows of a head -----------------------------
template <typename T, int NGD, int SPLIT>
__global__ void __launch_bounds__(SPLIT * kThreads) diff_bwd_row(Args a) {
  extern __shared__ __align__(16) float sm[];
  const int ld = ld_of(a.d), ldv = ld_of(a.dv_), N = a.N;
  const int grp = threadIdx.x / kThreads, tid = threadIdx.x % kThreads;
  const int ty = tid >> 4, tx = tid & 15;
  float* qs = sm;                      // [2][32][ld]
  float* dos = qs + 2 * kM * ld;       // [32][ldv]
  float* mine = dos + kM * ldv;        // the group's area
  const int area = group_floats(kT * (2 * ld + ldv) + kM * kLdp, 32 * NGD + 4);
  const float* other = mine + area;
  if (grp == 1) mine += area;
  float* ks = mine;                    // [2][64][ld]
  float* vs = ks + 2 * kT * ld;        // [64][ldv]
  float* ps = vs + kT * ldv;           // [32][kLdp]
  const int bh = blockIdx.x % a.heads, b = bh / a.H, h = bh % a.H;
  const int kvh = b * (a.H / a.G) + h / a.G;
  // heads vary fastest, and the long rows of all of them start first
  const int blk = blockIdx.x / a.heads;
  const int row0 = (a.causal ? (int)(gridDim.x / a.heads) - 1 - blk : blk) * kM;
  const size_t qsz = (size_t)N * a.d;
  const T* q = static_cast<const T*>(a.q) + (size_t)bh * 2 * qsz;
  const T* k = static_cast<const T*>(a.k) + (size_t)kvh * 2 * qsz;
  const T* v = static_cast<const T*>(a.v) + (size_t)kvh * N * a.dv_;
  if (grp == 0) {
    load_rows<kM>(tid, qs, ld, q, row0, N, a.d);
    load_rows<kM>(tid, qs + kM * ld, ld, q + qsz, row0, N, a.d);
  }
  if (grp == SPLIT - 1)
    load_rows<kM>(tid, dos, ldv, static_cast<const T*>(a.dO) + (size_t)bh * N * a.dv_, row0, N, a.dv_);
  loads_done();
  __syncthreads();
  float lse[2][4], D[2][4], w[4], d2[4], acc[2][4][4 * NGD];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = row0 + 4 * ty + i;
    d2[i] = 0.f;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const size_t at = ((size_t)bh * 2 + m) * N + (r < N ? r : 0);
      lse[m][i] = a.lse[at];
      D[m][i] = a.D[at];
#pragma unroll
      for (int e = 0; e < 4 * NGD; ++e) acc[m][i][e] = 0.f;
    }
    w[i] = lam_at(a.lam, a.H, N, b, h, r < N ? r : 0);
  }
  const int kend = a.causal ? min(N, row0 + kM) : N;
  for (int j0 = grp * kT; j0 < kend; j0 += SPLIT * kT) {
    group_sync<SPLIT>(grp);
    load_rows<kT>(tid, ks, ld, k, j0, N, a.d);
    load_rows<kT>(tid, ks + kT * ld, ld, k + qsz, j0, N, a.d);
    load_rows<kT>(tid, vs, ldv, v, j0, N, a.dv_);
    loads_done();
    group_sync<SPLIT>(grp);
    float dp[4][4];
    tile_dot(dp, dos, vs, ldv, a.dv_, ty, tx);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      float s[4][4];
      tile_dot(s, qs + m * kM * ld, ks + m * kT * ld, ld, a.d, ty, tx);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = row0 + 4 * ty + i;
        const float f = m == 0 ? 1.f : -w[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int col = j0 + tx + 16 * j;
          const bool in = r < N && col < N && (!a.causal || col <= r);
          const float pr = in ? expf(s[i][j] * a.scale - lse[m][i]) : 0.f;
          if (m == 1) d2[i] = fmaf(pr, dp[i][j], d2[i]);
          s[i][j] = in ? f * pr * (dp[i][j] - D[m][i]) : 0.f;
        }
      }
      put_tile(ps, s, ty, tx);
      tile_add<NGD>(acc[m], ps, ks + m * kT * ld, ld, a.d, ty, tx);
    }
  }
  if constexpr (SPLIT > 1) {
    group_sync<SPLIT>(grp);
    if (grp == 1) {
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4 * NGD; ++e)
            mine[((m * 4 + i) * 4 * NGD + e) * kThreads + tid] = acc[m][i][e];
#pragma unroll
      for (int i = 0; i < 4; ++i) mine[(32 * NGD + i) * kThreads + tid] = d2[i];
    }
    __syncthreads();
    if (grp == 1) return;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4 * NGD; ++e)
          acc[m][i][e] += other[((m * 4 + i) * 4 * NGD + e) * kThreads + tid];
#pragma unroll
    for (int i = 0; i < 4; ++i) d2[i] += other[(32 * NGD + i) * kThreads + tid];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = row0 + 4 * ty + i;
    const float s = row16_sum(d2[i]);
    if (tx == 0 && r < N) a.d2[(size_t)bh * N + r] = s;
  }
#pragma unroll
  for (int m = 0; m < 2; ++m)
    store_rows<T, NGD>(static_cast<T*>(a.dq) + ((size_t)bh * 2 + m) * qsz, acc[m], a.scale, row0, N,
                       a.d, a.d, ty, tx);
}

// ---- dK, dV: one block per 32 keys of a key head, over its query heads, or over
// one of gridDim.y parts of their tiles ---------------------------------------
template <typename T, int NGD, int NGV, int SPLIT>
__global__ void __launch_bounds__(SPLIT * kThreads) diff_bwd_col(Args a) {
  extern __shared__ __align__(16) float sm[];
  const int ld = ld_of(a.d), ldv = ld_of(a.dv_), N = a.N;
  const int grp = threadIdx.x / kThreads, tid = threadIdx.x % kThreads;
  const int ty = tid >> 4, tx = tid & 15;
  float* ks = sm;                      // [2][32][ld]
  float* vs = ks + 2 * kM * ld;        // [32][ldv]
  float* mine = vs + kM * ldv;         // the group's area
  const int area = group_floats(kT * (2 * ld + ldv + 5) + kM * kLdp, 32 * NGD + 16 * NGV);
  const float* other = mine + area;
  if (grp == 1) mine += area;
  float* qs = mine;                    // [2][64][ld]
  float* dos = qs + 2 * kT * ld;       // [64][ldv]
  float* ps = dos + kT * ldv;          // [32][kLdp]
  float* sc = ps + kM * kLdp;          // [5][64]: LSE^1, LSE^2, D^1, D^2, lam
  const int kvh = blockIdx.x % a.heads, Hk = a.H / a.G;
  const int b = kvh / Hk;
  const int col0 = blockIdx.x / a.heads * kM;
  const size_t qsz = (size_t)N * a.d;
  const T* k = static_cast<const T*>(a.k) + (size_t)kvh * 2 * qsz;
  if (grp == 0) {
    load_rows<kM>(tid, ks, ld, k, col0, N, a.d);
    load_rows<kM>(tid, ks + kM * ld, ld, k + qsz, col0, N, a.d);
  }
  if (grp == SPLIT - 1)
    load_rows<kM>(tid, vs, ldv, static_cast<const T*>(a.v) + (size_t)kvh * N * a.dv_, col0, N, a.dv_);
  loads_done();
  __syncthreads();
  float ak[2][4][4 * NGD], av[4][4 * NGV];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int e = 0; e < 4 * NGD; ++e) ak[0][i][e] = ak[1][i][e] = 0.f;
#pragma unroll
    for (int e = 0; e < 4 * NGV; ++e) av[i][e] = 0.f;
  }
  const int start = a.causal ? col0 / kT * kT : 0, per_head = (N - start + kT - 1) / kT;
  const int split = gridDim.y, part = blockIdx.y;
  const int t0 = (int)((long long)per_head * a.G * part / split);
  const int t1 = (int)((long long)per_head * a.G * (part + 1) / split);
  for (int g = t0 / per_head; g * per_head < t1; ++g) {
    const int h = (kvh % Hk) * a.G + g;
    const size_t bh = (size_t)b * a.H + h;
    const T* q = static_cast<const T*>(a.q) + bh * 2 * qsz;
    const T* dO = static_cast<const T*>(a.dO) + bh * N * a.dv_;
    const RowRange rows = part_rows(t0, t1, g, per_head, start, N, kT);
    for (int i0 = rows.first + grp * kT; i0 < rows.end; i0 += SPLIT * kT) {
      group_sync<SPLIT>(grp);
      load_rows<kT>(tid, qs, ld, q, i0, N, a.d);
      load_rows<kT>(tid, qs + kT * ld, ld, q + qsz, i0, N, a.d);
      load_rows<kT>(tid, dos, ldv, dO, i0, N, a.dv_);
      if (tid < kT) {
        const int r = min(i0 + tid, N - 1);
        sc[0 * kT + tid] = a.lse[(bh * 2 + 0) * N + r];
        sc[1 * kT + tid] = a.lse[(bh * 2 + 1) * N + r];
        sc[2 * kT + tid] = a.D[(bh * 2 + 0) * N + r];
        sc[3 * kT + tid] = a.D[(bh * 2 + 1) * N + r];
        sc[4 * kT + tid] = lam_at(a.lam, a.H, N, b, h, r);
      }
      loads_done();
      group_sync<SPLIT>(grp);
      float dp[4][4], wt[4][4];
      tile_dot(dp, vs, dos, ldv, a.dv_, ty, tx);
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        float s[4][4];
        tile_dot(s, ks + m * kM * ld, qs + m * kT * ld, ld, a.d, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int key = col0 + 4 * ty + i, c = tx + 16 * j, r = i0 + c;
            const bool in = r < N && key < N && (!a.causal || key <= r);
            const float p = in ? expf(s[i][j] * a.scale - sc[m * kT + c]) : 0.f;
            const float f = m == 0 ? p : -sc[4 * kT + c] * p;
            wt[i][j] = m == 0 ? f : wt[i][j] + f;
            s[i][j] = in ? f * (dp[i][j] - sc[(2 + m) * kT + c]) : 0.f;
          }
        put_tile(ps, s, ty, tx);
        tile_add<NGD>(ak[m], ps, qs + m * kT * ld, ld, a.d, ty, tx);
      }
      put_tile(ps, wt, ty, tx);
      tile_add<NGV>(av, ps, dos, ldv, a.dv_, ty, tx);
    }
  }
  if constexpr (SPLIT > 1) {
    group_sync<SPLIT>(grp);
    if (grp == 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int e = 0; e < 4 * NGD; ++e)
            mine[((m * 4 + i) * 4 * NGD + e) * kThreads + tid] = ak[m][i][e];
#pragma unroll
        for (int e = 0; e < 4 * NGV; ++e)
          mine[(32 * NGD + i * 4 * NGV + e) * kThreads + tid] = av[i][e];
      }
    }
    __syncthreads();
    if (grp == 1) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int e = 0; e < 4 * NGD; ++e)
          ak[m][i][e] += other[((m * 4 + i) * 4 * NGD + e) * kThreads + tid];
#pragma unroll
      for (int e = 0; e < 4 * NGV; ++e)
        av[i][e] += other[(32 * NGD + i * 4 * NGV + e) * kThreads + tid];
    }
  }
  if (split > 1) {
    const int W = 2 * a.d + a.dv_;
    float* dst = a.parts + ((size_t)part * a.heads + kvh) * N * W;
    store_rows<float, NGD>(dst, ak[0], 1.f, col0, N, a.d, W, ty, tx);
    store_rows<float, NGD>(dst + a.d, ak[1], 1.f, col0, N, a.d, W, ty, tx);
    store_rows<float, NGV>(dst + 2 * a.d, av, 1.f, col0, N, a.dv_, W, ty, tx);
    return;
  }
#pragma unroll
  for (int m = 0; m < 2; ++m)
    store_rows<T, NGD>(static_cast<T*>(a.dk) + ((size_t)kvh * 2 + m) * qsz, ak[m], a.scale, col0, N,
                       a.d, a.d, ty, tx);
  store_rows<T, NGV>(static_cast<T*>(a.dv) + (size_t)kvh * N * a.dv_, av, 1.f, col0, N, a.dv_, a.dv_,
                     ty, tx);
}

// dK (scaled) and dV from the parts, added in their order: a thread per element.
template <typename T>
__global__ void __launch_bounds__(256) diff_join(Args a, int split) {
  const size_t W = 2 * a.d + a.dv_, total = (size_t)a.heads * a.N * W;
  const size_t e = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= total) return;
  float x = a.parts[e];
  for (int s = 1; s < split; ++s) x += a.parts[s * total + e];
  const size_t row = e / W, kvh = row / a.N, j = row - kvh * a.N;
  const int f = (int)(e - row * W);
  if (f < 2 * a.d) {
    const int m = f / a.d;
    static_cast<T*>(a.dk)[((2 * kvh + m) * a.N + j) * a.d + f - m * a.d] = from_f32<T>(x * a.scale);
  } else {
    static_cast<T*>(a.dv)[row * a.dv_ + f - 2 * a.d] = from_f32<T>(x);
  }
}

// Parts of the dK/dV pass, where its blocks are fewer than the SMs: as many as
// leave each 4 or more tiles.  Whole and cut, fp32: 2 x 4 heads on one key head x
// 796, d = 40, dv = 128 489, 176 + 4 us; 1 x 4 on one x 1500, d = 64 900, 303 + 4;
// 2 heads x 700 116, 64 + 4.
int col_parts(const DiffProblem& p) {
  const long long blocks = (long long)((p.N + kM - 1) / kM) * p.B * p.Hk;
  const long long tiles = (long long)((p.N + kT - 1) / kT) * p.G();
  return (int)max(1ll, min(kSms / blocks, tiles / 4));
}

Args make_args(const DiffProblem& p, const DiffTensors& t) {
  Args a{};
  a.q = t.q; a.k = t.k; a.v = t.v; a.dO = t.dO;
  a.o = t.o; a.rest = t.rest; a.dq = t.dq; a.dk = t.dk; a.dv = t.dv;
  a.lse = t.lse;
  a.lam = t.lam;
  a.H = p.H; a.G = p.G(); a.N = p.N; a.d = p.d; a.dv_ = p.dv; a.causal = p.causal;
  a.scale = p.scale;
  return a;
}

constexpr size_t kMaxShared = 232448;

template <typename K>
cudaError_t launch(K kernel, int blocks, int split, size_t floats, const Args& a, LaunchLog& log,
                   int parts = 1) {
  const size_t bytes = floats * sizeof(float);
  // (the limit belongs to the kernel, which another thread may be about to launch: it is always
  // set to the most there is)
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxShared);
  if (e != cudaSuccess) return e;
  kernel<<<dim3(blocks * a.heads, parts), split * kThreads, bytes, log.stream>>>(a);
  e = cudaGetLastError();
  log.mark();
  return e;
}

// Two groups per block where their areas fit in shared memory.
template <typename K1, typename K2>
cudaError_t run(K1 one, K2 two, int blocks, int heads, size_t fixed, size_t area, Args a,
                LaunchLog& log, int parts = 1) {
  a.heads = heads;
  if ((fixed + 2 * area) * sizeof(float) <= kMaxShared)
    return launch(two, blocks, 2, fixed + 2 * area, a, log, parts);
  return launch(one, blocks, 1, fixed + area, a, log, parts);
}

template <typename T>
cudaError_t forward_t(const DiffProblem& p, const DiffTensors& t, LaunchLog& log) {
  const int blocks = (p.N + kM - 1) / kM;
  const size_t q = (size_t)2 * kM * ld_of(p.d), area = fwd_area(p.d, p.dv);
  Args a = make_args(p, t);
  a.heads = p.B * p.H;
  // With few blocks the longest row's time counts: two pairs of groups share
  // one.  With many the SMs' throughput does: two blocks of a pair per SM, which
  // need not add up.  One pair, two, in us (fp32, d = 64, dv = 128): causal, 128
  // blocks 262, 204; 192 209, 157; 256 296, 205; 288 339, 230; 368 466, 395; 512
  // 723, 712; 1024 1315, 1355; without mask 128 264, 204; 192 305, 304; 256 404,
  // 400; 288 452, 448; 512 1551, 1524.  At dv = 64 without mask two are 3% slower
  // from 192 to 288 blocks.
  const bool split = (long long)blocks * a.heads <= 2 * kSms &&
                     (q + 2 * area) * sizeof(float) <= kMaxShared;
  if (split)
    return p.dv <= 64 ? launch(diff_fwd<T, 1, 2>, blocks, 4, q + 2 * area, a, log)
                      : launch(diff_fwd<T, 2, 2>, blocks, 4, q + 2 * area, a, log);
  return p.dv <= 64 ? launch(diff_fwd<T, 1, 1>, blocks, 2, q + area, a, log)
                    : launch(diff_fwd<T, 2, 1>, blocks, 2, q + area, a, log);
}

template <typename T, int NGD, int NGV>
cudaError_t columns(int blocks, int heads, size_t fixed, int tiles, const Args& a, LaunchLog& log,
                    int parts) {
  return run(diff_bwd_col<T, NGD, NGV, 1>, diff_bwd_col<T, NGD, NGV, 2>, blocks, heads, fixed,
             group_floats(tiles, 32 * NGD + 16 * NGV), a, log, parts);
}

template <typename T>
cudaError_t backward_t(const DiffProblem& p, const DiffTensors& t, const DiffWorkspace& ws,
                       LaunchLog& log) {
  Args a = make_args(p, t);
  a.D = ws.D;
  a.d2 = ws.d2;
  a.parts = ws.parts;
  const int ld = ld_of(p.d), ldv = ld_of(p.dv), tiles = kT * (2 * ld + ldv) + kM * kLdp;
  const int blocks = (p.N + kM - 1) / kM, rows = p.B * p.H, cols = p.B * p.Hk;
  const size_t fixed = (size_t)kM * (2 * ld + ldv);
  cudaError_t e = p.d <= 64 ? run(diff_bwd_row<T, 1, 1>, diff_bwd_row<T, 1, 2>, blocks, rows, fixed,
                                  group_floats(tiles, 32 + 4), a, log)
                            : run(diff_bwd_row<T, 2, 1>, diff_bwd_row<T, 2, 2>, blocks, rows, fixed,
                                  group_floats(tiles, 64 + 4), a, log);
  if (e != cudaSuccess) return e;
  const int ct = tiles + 5 * kT, parts = col_parts(p);
  e = p.d <= 64 ? p.dv <= 64 ? columns<T, 1, 1>(blocks, cols, fixed, ct, a, log, parts)
                             : columns<T, 1, 2>(blocks, cols, fixed, ct, a, log, parts)
      : p.dv <= 64 ? columns<T, 2, 1>(blocks, cols, fixed, ct, a, log, parts)
                   : columns<T, 2, 2>(blocks, cols, fixed, ct, a, log, parts);
  if (e != cudaSuccess || parts == 1) return e;
  a.heads = cols;
  const size_t total = (size_t)cols * p.N * (2 * p.d + p.dv);
  diff_join<T><<<(unsigned)((total + 255) / 256), 256, 0, log.stream>>>(a, parts);
  e = cudaGetLastError();
  log.mark();
  return e;
}

}  // namespace

size_t diff_simt_part_count(const DiffProblem& p) {
  const int parts = col_parts(p);
  return parts == 1 ? 0 : (size_t)parts * p.B * p.Hk * p.N * (2 * p.d + p.dv);
}

cudaError_t diff_simt_forward(const DiffProblem& p, const DiffTensors& t, LaunchLog& log) {
  return p.bf16 ? forward_t<__nv_bfloat16>(p, t, log) : forward_t<float>(p, t, log);
}

cudaError_t diff_simt_backward(const DiffProblem& p, const DiffTensors& t, const DiffWorkspace& ws,
                               LaunchLog& log) {
  return p.bf16 ? backward_t<__nv_bfloat16>(p, t, ws, log) : backward_t<float>(p, t, ws, log);
}

}  // namespace fbob
