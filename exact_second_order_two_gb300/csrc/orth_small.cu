// Orthogonalisation of small matrices: one block takes a matrix through all its steps.
//
// Up to 128 rows (p) and 128 columns (256 for bf16), X, A and B stay in shared memory, as
// tiles that are left operands, right operands by rows (P Q^T) and by columns (P Q) as
// they lie; the accumulator is in TMEM.  A product is at most 64 MMAs of 64 clocks, so what
// counts is the way between them: MMAs done, accumulator read, values rounded and
// written, MMAs issued: three times a step, 1.2 us each for bf16 in one term, 2.3 for fp32 (a
// warp to 32 rows and 32 columns; with half as many warps 3).  As products in memory over the
// whole GPU (orth_chain.cu) each takes 8.  16 x 64 x 64, bf16: 93 us there, 25 here in one
// term; 4 x 128 x 128, fp32, with its gradient: 168 us, of 357.  Symmetric results are computed whole, which saves the mirroring.
//
// bf16: X and B have two terms in products, too, in the steps behind which small singular values
// grow by 64 at most (before, X is small, and what B adds smaller).  In a large matrix each
// result is a sum of many roundings, in a small one of few, and MMAs cost little: 16 x 24 to
// 64 x 96, the result 2.1e-3 to 2.3e-3 off with one term and the gradient 2.7e-3 to 3.9e-3,
// 1.8e-3 and 2.3e-3 to 2.6e-3 so; 16 x 64 x 64 takes 26.6 us, 22.6 with one.
//
// With a backward to follow, X, A and B of every step leave for the workspace by TMA.  The
// backward holds H, S (then T) and, in turn in one place, X (in two parts where second terms of
// H and S leave no room for more), A, B and X again.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "fbob.h"
#include "orth.h"
#include "orth_tile.cuh"
#include "sm103.cuh"
#include "tc_common.cuh"

namespace fbob {
namespace orth {
namespace {

constexpr int kThreads = 512;  // a warp to 32 rows and 32 columns of a square result
constexpr int kSquare = 2;  // tiles (64 columns) of A, B, S and T

// A matrix in shared memory: `terms` times `tiles` tiles.
struct Held {
  uint8_t* at;
  int tiles;
  __device__ __forceinline__ uint8_t* tile(int term, int c) const {
    return at + (term * tiles + c) * kTileBytes;
  }
};

struct Shared {
  uint64_t mma, load;  // barriers
  uint32_t tmem;
  Abort ab;
  float red[kThreads / 32];
  short e[kMaxSteps + 1];
};
constexpr uint32_t kMisc = 256;
constexpr int kMostTiles = 14;  // in shared memory
static_assert(kMostTiles * kTileBytes + kMisc <= 232448, "small orthogonalisation: shared memory");
static_assert(sizeof(Shared) <= kMisc, "small orthogonalisation: shared memory");

__device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
#pragma unroll
  for (int k = 0; k < kThreads / 32; ++k) v += red[k];
  return v;
}

// Element (r, c) of a matrix with the shorter side first, kept as the caller has it.
template <typename T>
__device__ __forceinline__ const T* element(const T* x, int r, int c, int p, int q, int tall) {
  return x + (tall ? (size_t)c * p + r : (size_t)r * q + c);
}

template <typename T>
__device__ __forceinline__ Squares squares(const T* x, int elems, float* red) {
  return squares_of([&](float scale) {
    float s = 0.f;
#pragma unroll 4
    for (int i = threadIdx.x; i < elems; i += kThreads) {
      const float v = to_f32<T>(x[i]) * scale;
      s = fmaf(v, v, s);
    }
    return block_sum(s, red);
  });
}

// factor x into tiles of `terms` terms, zeros around it.
template <typename T>
__device__ __forceinline__ void take_in(const T* x, const Held& h, int terms, float factor, int p, int q,
                                        int tall) {
  for (int i = threadIdx.x; i < kTile * 8 * h.tiles; i += kThreads) {
    // lanes on neighbouring elements: along a row's chunks of eight, or down the rows
    const int r = tall ? i % kTile : i / (8 * h.tiles), ch = tall ? i / kTile : i % (8 * h.tiles);
    f2 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = 8 * ch + 2 * k;
      v[k].x = r < p && c < q ? to_f32<T>(*element(x, r, c, p, q, tall)) * factor : 0.f;
      v[k].y = r < p && c + 1 < q ? to_f32<T>(*element(x, r, c + 1, p, q, tall)) * factor : 0.f;
    }
    uint32_t w[4], lo[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      w[k] = to_halves(v[k]);
      lo[k] = to_halves(fma2(f2{-1.f, -1.f}, halves(w[k]), v[k]));
    }
    *slot_chunk(h.tile(0, ch / 8), r, ch % 8) = make_uint4(w[0], w[1], w[2], w[3]);
    if (terms == 2) *slot_chunk(h.tile(1, ch / 8), r, ch % 8) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}

// Issued by one thread: acc (+)= P Q^T over tile k of columns, or P Q over tile k of Q's
// rows (64 each).
__device__ __forceinline__ void multiply(uint32_t acc, const Held& P, int tp, const Held& Q, int tq, bool nn,
                                         int k, bool begun) {
  const uint32_t id = idesc_f16(kTile, nn ? 64 * Q.tiles : kTile, nn);
  const uint32_t a = lo_kmajor(smem_u32(P.tile(tp, k)));
  const uint32_t b = nn ? lo_mnmajor(smem_u32(Q.tile(tq, 0)), kTileBytes) + 4 * k * kstep_off(1)
                        : lo_kmajor(smem_u32(Q.tile(tq, k)));
#pragma unroll
  for (int u = 0; u < 4; ++u)
    mma_ss(acc, a + 2 * u, b + (nn ? kstep_off(u) : 2 * u), id, begun || u > 0 ? 1u : 0u);
}
// A product over `depth` tiles: every pair of terms but the two low ones, the high ones
// last.  For fp32, sums of 64 products of high terms each in an accumulator of their own
// (of four; at most two tiles, two products), for what the tensor cores cut off their
// additions; `first` is the product's first accumulator, or not 0 where the one that there is
// has been begun.  pt, qt: terms of P and Q for bf16.
template <int TERMS>
__device__ __forceinline__ void multiply_terms(uint32_t acc, const Held& P, int pt, const Held& Q, int qt, bool nn,
                                               int depth, int first) {
  for (int k = 0; k < depth; ++k) {
    if (TERMS == 2) {
      const uint32_t own = acc + 128 * (first + k);
      multiply(own, P, 0, Q, 1, nn, k, false);
      multiply(own, P, 1, Q, 0, nn, k, true);
      multiply(own, P, 0, Q, 0, nn, k, true);
    } else {
      bool begun = first + k > 0;
      if (qt == 2) {
        multiply(acc, P, 0, Q, 1, nn, k, begun);
        begun = true;
      }
      if (pt == 2) {
        multiply(acc, P, 1, Q, 0, nn, k, begun);
        begun = true;
      }
      multiply(acc, P, 0, Q, 0, nn, k, begun);
    }
  }
}

__device__ __forceinline__ void store_held(const CUtensorMap* hi, const CUtensorMap* lo, const Held& h, int at,
                                           int cols, int rows) {
  for (int t = 0; t < (lo ? 2 : 1); ++t)
    for (int c = 0; c < h.tiles && 64 * c < cols; ++c) tma_store_3d(t ? lo : hi, h.tile(t, c), 64 * c, 0, at);
  bulk_commit_group();
}
// tiles first .. first + tiles - 1 of the columns, to h's first
__device__ __forceinline__ void load_held(const CUtensorMap* hi, const CUtensorMap* lo, const Held& h, int first,
                                          int tiles, uint64_t* bar, int at) {
  mbar_arrive_expect_tx(bar, (lo ? 2 : 1) * tiles * kTileBytes);
  for (int t = 0; t < (lo ? 2 : 1); ++t)
    for (int c = 0; c < tiles; ++c) tma_load_3d(h.tile(t, c), t ? lo : hi, bar, 64 * (first + c), 0, at);
}

__device__ __forceinline__ void begin_block(Shared* sh, uint32_t cols, const SmallArgs& g) {
  if (threadIdx.x == 0) {
    mbar_init(&sh->mma, 1);
    mbar_init(&sh->load, 1);
    sh->ab.flag = 0;
    sh->ab.limit_ns = g.wait_ns;
    fence_mbar_init();
  }
  if (threadIdx.x < 32) {
    tmem_alloc(&sh->tmem, cols);
    tmem_relinquish();
  }
  tc_fence_before();
  after_previous();
  __syncthreads();
  tc_fence_after();
}
__device__ __forceinline__ void end_block(Shared* sh, uint32_t cols) {
  if (threadIdx.x == 0 && sh->ab.flag)  // what an abort leaves in flight lands
    for (const uint64_t t0 = global_ns(); global_ns() - t0 < 10000000ull;) __nanosleep(10000);
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x < 32) {
    tc_fence_after();
    tmem_dealloc(sh->tmem, cols);
  }
}

// The tiles just written are seen by MMAs and TMA; every thread is past its reads of the
// accumulator.
__device__ __forceinline__ void hand_over() {
  fence_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
}

// The thread's 32 columns (32 u on) of the sum of `count` accumulators, times alpha.
__device__ __forceinline__ void read_acc(uint32_t acc, int count, int u, float alpha, f2 (&v)[16]) {
  acc += ((uint32_t)(32 * ((threadIdx.x >> 5) & 3)) << 16) + 32 * u;
#pragma unroll
  for (int k = 0; k < 16; ++k) v[k] = f2{0.f, 0.f};
  for (int i = 0; i < count; ++i) {
    uint32_t w[32];
    tmem_ld32(acc + 128 * i, w);
#pragma unroll
    for (int k = 0; k < 16; ++k)
      v[k] = add2(v[k], f2{__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1])});
  }
#pragma unroll
  for (int k = 0; k < 16; ++k) v[k] = mul2(f2{alpha, alpha}, v[k]);
}
// in `terms` terms to columns 32 u .. of h
__device__ __forceinline__ void put(const f2 (&v)[16], const Held& h, int terms, int row, int u) {
  uint32_t w[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) w[k] = to_halves(v[k]);
  put_slot(w, h.tile(0, u >> 1), row, u & 1);
  if (terms == 2) {
    uint32_t lo[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) lo[k] = to_halves(fma2(f2{-1.f, -1.f}, halves(w[k]), v[k]));
    put_slot(lo, h.tile(1, u >> 1), row, u & 1);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1) small_forward(const __grid_constant__ SmallArgs g) {
  constexpr int TERMS = sizeof(T) == 2 ? 1 : 2;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {
    after_previous();
    if (threadIdx.x == 0) report_status(g.status, FBOB_ERR_CUDA);
    return;
  }
  const int tiles = (g.q + 63) / 64, l = blockIdx.x;
  const Held X{smem, tiles}, A{smem + g.x_terms * tiles * kTileBytes, kSquare};  // B in A's place
  Shared* sh = reinterpret_cast<Shared*>(A.at + 2 * kSquare * kTileBytes);
  const uint32_t cols = TERMS == 2 ? 512 : tiles > 2 ? 256 : 128;
  begin_block(sh, cols, g);
  const uint32_t acc = sh->tmem;
  const int row = 32 * ((threadIdx.x >> 5) & 3) + (threadIdx.x & 31), unit = threadIdx.x >> 7;
  const T* x = static_cast<const T*>(g.g) + (size_t)l * g.p * g.q;
  MatInfo info;
  const float factor = info_of(squares(x, g.p * g.q, sh->red), g.eps, g.xe[0], g.steps, info);
  float bound = fminf(info.norm * info.s, 1.f);  // of X's singular values (1 for NaN: no room)
  int e = info.e[0];
  if (threadIdx.x == 32) g.info[l] = info;
  take_in(x, X, g.xt[0], factor, g.p, g.q, g.tall);
  const int deep = (g.p + 63) / 64;  // tiles of A's columns
  const int wide_sums = TERMS == 2 ? tiles : 1, deep_sums = TERMS == 2 ? deep : 1;
  int n = 0;                         // products so far
  bool ok = true;
  // one product: what `store` sends off is read before the tiles can be written again
  auto product = [&](const Held& P, int pt, const Held& Q, int qt, bool nn, int depth, auto store) {
    hand_over();
    if (threadIdx.x == 0 && !sh->ab.flag) {
      store();
      multiply_terms<TERMS>(acc, P, pt, Q, qt, nn, depth, 0);
      bulk_wait_read_all();
      mma_commit(&sh->mma);
    }
    __syncwarp();
    ok = ok && warp_wait(&sh->mma, n++ & 1, &sh->ab, g.status);
    tc_fence_after();
  };
  for (int i = 0; i < g.steps.n; ++i) {
    const float f = i == 0 ? info.f : 1.f;
    const bool last = i + 1 == g.steps.n;
    bound = next_bound(g.steps, i, bound);
    const int e1 = last ? 0 : room_below(g.steps.bound[i + 1], bound);
    if (threadIdx.x == 32) g.info[l].e[i + 1] = (short)e1;
    f2 v[16];
    // terms of B, and of X in products
    const int bt = TERMS == 2 ? 2 : 1 + (g.two_b >> i & 1), xp = min(bt, g.xt[i]);
    product(X, xp, X, xp, false, tiles, [&] {
      if (g.keep) store_held(&g.x_map[0], TERMS == 2 ? &g.x_map[1] : nullptr, X, i * g.L + l, g.q, g.p);
    });
    read_acc(acc, wide_sums, unit, f * f * g.to_a[i], v);
    put(v, A, TERMS, row, unit);
    product(A, 1, A, 1, false, deep, [&] {
      if (g.keep) store_held(&g.a_map[0], TERMS == 2 ? &g.a_map[1] : nullptr, A, i * g.L + l, g.p, g.p);
    });
    read_acc(acc, deep_sums, unit, times_pow2(g.to_b[i], -2 * e), v);
    add_slot(v, A.tile(0, unit >> 1), row, unit & 1, g.a_to_b[i]);
    if (TERMS == 2) add_slot(v, A.tile(1, unit >> 1), row, unit & 1, g.a_to_b[i]);
    put(v, A, bt, row, unit);
    product(A, bt, X, xp, true, deep, [&] {
      if (g.keep) store_held(&g.b_map[0], TERMS == 2 ? &g.b_map[1] : nullptr, A, i * g.L + l, g.p, g.p);
    });
    const float to_x = times_pow2(f * g.to_x[i], e1 - 3 * e), x_to_x = times_pow2(f * g.x_to_x[i], e1 - e);
    e = e1;
    for (int u = unit; u < 2 * tiles; u += 4) {
      read_acc(acc, deep_sums, u, to_x, v);
      add_slot(v, X.tile(0, u >> 1), row, u & 1, x_to_x);
      if (g.xt[i] == 2) add_slot(v, X.tile(1, u >> 1), row, u & 1, x_to_x);
      if (!last) {
        put(v, X, g.xt[i + 1], row, u);
        continue;
      }
      T* y = static_cast<T*>(g.y) + (size_t)l * g.p * g.q;
#pragma unroll
      for (int k = 0; k < 32; ++k)
        if (row < g.p && 32 * u + k < g.q)
          *const_cast<T*>(element(y, row, 32 * u + k, g.p, g.q, g.tall)) = from_f32<T>(k & 1 ? v[k / 2].y : v[k / 2].x);
    }
  }
  if (threadIdx.x == 0) bulk_wait_all();
  end_block(sh, cols);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1) small_backward(const __grid_constant__ SmallArgs g) {
  constexpr int TERMS = sizeof(T) == 2 ? 1 : 2;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {
    after_previous();
    if (threadIdx.x == 0) report_status(g.status, FBOB_ERR_CUDA);
    return;
  }
  const int tiles = (g.q + 63) / 64, l = blockIdx.x, room = g.x_tiles > kSquare ? g.x_tiles : kSquare;
  const Held H{smem, tiles}, S{smem + g.h_terms * tiles * kTileBytes, kSquare};
  // what comes from memory: X, x_tiles of it at a time, or A or B
  const Held X{S.at + g.h_terms * kSquare * kTileBytes, g.x_tiles}, A{X.at, kSquare};
  Shared* sh = reinterpret_cast<Shared*>(X.at + TERMS * room * kTileBytes);
  const uint32_t cols = TERMS == 2 ? 512 : tiles > 2 ? 256 : 128;
  begin_block(sh, cols, g);
  if (threadIdx.x < g.steps.n) sh->e[threadIdx.x] = g.info[l].e[threadIdx.x];
  const uint32_t acc = sh->tmem;
  const int row = 32 * ((threadIdx.x >> 5) & 3) + (threadIdx.x & 31), unit = threadIdx.x >> 7;
  const int deep = (g.p + 63) / 64;
  const int wide_sums = TERMS == 2 ? 2 * tiles : 1, deep_sums = TERMS == 2 ? 2 * deep : 1;
  const T* dy = static_cast<const T*>(g.dy) + (size_t)l * g.p * g.q;
  const MatInfo info = g.info[l];
  int n = 0, m = 0;  // products and loads so far
  bool ok = true;
  auto load = [&](const CUtensorMap* maps, const Held& to, int first, int count, int i) {  // by thread 0
    if (!sh->ab.flag) load_held(&maps[0], TERMS == 2 ? &maps[1] : nullptr, to, first, count, &sh->load, i * g.L + l);
  };
  auto part = [&](int first) { return min(g.x_tiles, tiles - first); };  // of X from a tile on
  auto loaded = [&] { ok = ok && warp_wait(&sh->load, m++ & 1, &sh->ab, g.status); };
  auto product = [&](auto issue) {
    hand_over();
    if (threadIdx.x == 0 && !sh->ab.flag) {
      issue();
      mma_commit(&sh->mma);
    }
    __syncwarp();
    ok = ok && warp_wait(&sh->mma, n++ & 1, &sh->ab, g.status);
    tc_fence_after();
  };
  if (threadIdx.x == 0) load(g.x_map, X, 0, part(0), g.steps.n - 1);
  const Squares dy2 = squares(dy, g.p * g.q, sh->red);
  int exp = rescaling(dy2, g.target[g.steps.n]);
  const float factor = ldexpf(1.f, exp);
  take_in(dy, H, TERMS, factor, g.p, g.q, g.tall);
  float nu2 = ldexpf(dy2.m, dy2.e + 2 * exp);
  float dots = 0.f;
  for (int i = g.steps.n - 1; i >= 0; --i) {
    const int e = sh->e[i];  // X, S and T are 2^e larger in store, A and B 2^(2 e)
    const float f = i == 0 ? info.f : 1.f;  // X_0 is f times what is stored
    // terms of S and T, of H, and of H in products
    const int st = TERMS == 2 ? 2 : 1 + (g.two_s >> i & 1), ht = TERMS == 2 ? 2 : 1 + (g.two_h >> i & 1);
    const int hp = TERMS == 2 ? 2 : 1 + (g.two_hp >> i & 1);
    f2 v[16];
    for (int c = 0; c < tiles; c += g.x_tiles) {
      loaded();
      product([&] {
        const Held Hc{H.at + c * kTileBytes, tiles};  // the columns that are here of X
        multiply_terms<TERMS>(acc, Hc, hp, X, 1, false, part(c), c);
        multiply_terms<TERMS>(acc, X, 1, Hc, hp, false, part(c), TERMS == 2 ? tiles : 1);
      });
      if (threadIdx.x == 0 && c + g.x_tiles < tiles) load(g.x_map, X, c + g.x_tiles, part(c + g.x_tiles), i);
    }
    if (threadIdx.x == 0) load(g.a_map, A, 0, kSquare, i);
    read_acc(acc, wide_sums, unit, f * g.to_s[i], v);
    put(v, S, st, row, unit);
    loaded();
    product([&] {
      multiply_terms<TERMS>(acc, A, 1, S, st, false, deep, 0);
      multiply_terms<TERMS>(acc, S, st, A, 1, false, deep, deep);
    });
    if (threadIdx.x == 0) load(g.b_map, A, 0, kSquare, i);
    read_acc(acc, deep_sums, unit, times_pow2(f * g.to_t[i], -2 * e), v);  // T in S's place
    add_slot(v, S.tile(0, unit >> 1), row, unit & 1, f * g.s_to_t[i]);
    if (st == 2) add_slot(v, S.tile(1, unit >> 1), row, unit & 1, f * g.s_to_t[i]);
    put(v, S, st, row, unit);
    loaded();
    product([&] { multiply_terms<TERMS>(acc, A, 1, H, hp, true, deep, 0); });
    const int shift = rescaling(Squares{nu2, 0}, g.target[i]);
    exp += shift;
    const float alpha = ldexpf(g.to_h[i], shift - 2 * e), beta = ldexpf(g.h_to_h[i], shift);
    float sum = 0.f;
    for (int c = 0; c < tiles; c += g.x_tiles) {
      if (threadIdx.x == 0) load(g.x_map, X, c, part(c), i);
      loaded();
      product([&] {
        multiply_terms<TERMS>(acc + 64 * c, S, st, Held{X.at, part(c)}, 1, true, deep, deep);
      });
      for (int u = 2 * c + unit; u < 2 * (c + part(c)); u += 4) {
        read_acc(acc, deep_sums, u, alpha, v);
        add_slot(v, H.tile(0, u >> 1), row, u & 1, beta);
        if (ht == 2) add_slot(v, H.tile(1, u >> 1), row, u & 1, beta);
        f2 w[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) w[k] = i > 0 ? v[k] : f2{0.f, 0.f};
        if (i == 0) {  // <H_0, X_0>, which is still there
          add_slot(w, X.tile(0, (u >> 1) - c), row, u & 1, 1.f);
          if (TERMS == 2) add_slot(w, X.tile(1, (u >> 1) - c), row, u & 1, 1.f);
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) sum = fmaf(v[k].x, w[k].x, fmaf(v[k].y, w[k].y, sum));
        put(v, H, TERMS == 2 ? 2 : i > 0 ? 1 + (g.two_h >> (i - 1) & 1) : 1, row, u);
      }
      if (i == 0) __syncthreads();  // every thread is past its reads of this part of X
    }
    sum = block_sum(sum, sh->red);
    if (i > 0) {
      nu2 = sum;
      if (threadIdx.x == 0) load(g.x_map, X, 0, part(0), i - 1);
    } else {
      dots = sum;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) end_factors(info, dots, exp, g.xe[0], sh->red[0], sh->red[1], sh->red[2]);
  __syncthreads();  // (64-bit arithmetic is slow: once is enough)
  const float by_h = sh->red[0], by_g = sh->red[1], up = sh->red[2];
  const T* x = static_cast<const T*>(g.g) + (size_t)l * g.p * g.q;
  T* out = static_cast<T*>(g.y) + (size_t)l * g.p * g.q;
  for (int i = threadIdx.x; i < g.p * g.q; i += kThreads) {
    const int major = i / (g.tall ? g.p : g.q), minor = i - major * (g.tall ? g.p : g.q);
    const int r = g.tall ? minor : major, c = g.tall ? major : minor;
    float h = 0.f;
#pragma unroll
    for (int t = 0; t < TERMS; ++t)
      h += __half2float(*reinterpret_cast<const __half*>(H.tile(t, c >> 6) + sw128_offset(r, (c & 63) >> 3) +
                                                         2 * (c & 7)));
    out[i] = from_f32<T>(fmaf(-by_g, to_f32<T>(x[i]) * up, by_h * h));
  }
  end_block(sh, cols);
}

}  // namespace

bool small_fits(int p, int q, bool bf16) { return p <= kTile && q <= (bf16 ? 256 : 128); }

template <typename T>
cudaError_t launch(const SmallArgs& g, bool backward, LaunchLog& log) {
  const int terms = sizeof(T) == 2 ? 1 : 2, tiles = (g.q + 63) / 64;
  const int held = backward ? g.h_terms * (tiles + kSquare) + terms * (g.x_tiles > kSquare ? g.x_tiles : kSquare)
                            : g.x_terms * tiles + 2 * kSquare;
  const int smem = held * (int)kTileBytes + (int)kMisc;
  auto kernel = backward ? small_backward<T> : small_forward<T>;
  // (the limit belongs to the kernel, which another thread may be about to launch: it is always
  // set to the most that a call takes)
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kMostTiles * (int)kTileBytes + (int)kMisc);
  if (e != cudaSuccess) return e;
  return launch_next(kernel, dim3((unsigned)g.L), kThreads, smem, 1, log, g);
}
cudaError_t launch_small(const SmallArgs& args, bool bf16, bool backward, LaunchLog& log) {
  SmallArgs g = args;
  // all of X, or, where shared memory would not hold that, two tiles at a time: 4 of H, and S, in
  // two terms each
  const int tiles = (g.q + 63) / 64;
  g.x_tiles = g.h_terms * (tiles + kSquare) + tiles <= kMostTiles || !bf16 ? tiles : kSquare;
  return bf16 ? launch<__nv_bfloat16>(g, backward, log) : launch<float>(g, backward, log);
}

}  // namespace orth
}  // namespace fbob
