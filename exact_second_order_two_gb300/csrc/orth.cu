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
// accumulator and finished by alpha acc + beta E: one kernel (product) serves them
// all.  A, B, S and T are symmetric: only tiles on and below the diagonal are computed,
// and written in both places.  S and A S + S A are sums of a product and its transpose: as
// one accumulation [H | X] [X | H]^T they need half the tiles, too.
//
// Numbers.  Operands are fp16 with exponents chosen for each matrix, accumulation
// is fp32.  X has singular values up to M (bounded on the host from the
// polynomials), so that one power of two for all of X, A and B keeps them inside fp16's
// range, with 11 bits down to 2^-26 of the bound; H is rescaled every step by the norm
// that it was measured to have.  fp32 tensors are held as the sum of two fp16 (22 bits)
// and multiplied in three products; bf16 tensors in one.  There, a rounding error of X
// between its weak directions grows by a every step.  It reaches them through a X alone
// (B is small there, and an error of A or of B X lies in a strong direction on one side),
// so that X is kept in two terms, of which the products take the first and a X
// both, in steps whose rounding later steps would multiply by more than 16.
// (256 x 1024 of rank 16 with noise of a hundredth: 1.6e-2 of the norm off with one term,
// 2.2e-3 with two, 1.7e-3 for the result's own rounding.)
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdlib.h>
#include <string.h>
#include <stdint.h>

#include "common.cuh"
#include "fbob.h"
#include "internal.h"
#include "ops.h"
#include "sm103.cuh"
#include "tc_common.cuh"

namespace fbob {
namespace {

using namespace tc;

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

// ---------------------------------------------------------------------------
// What is kept of a matrix
// ---------------------------------------------------------------------------
struct MatInfo {
  float norm, s;  // |G|_F and 1 / (norm + eps)
  float f;        // X_0 = f G 2^k: f in [1, 2)
  int k;
};

// A matrix in one or two fp16 terms: rows of ld elements, [count] matrices.  Its maps:
// tiles of 128 rows and 64 columns (left operands, right ones of P Q^T, what is added,
// results) and of 64 rows and 64 columns (right operands of P Q).
struct Terms {
  __half *hi = nullptr, *lo = nullptr;
  int rows = 0, cols = 0, ld = 0;
  CUtensorMap tile[2], step[2];
};

// ---------------------------------------------------------------------------
// The product kernel
// ---------------------------------------------------------------------------
constexpr int kTile = 128;        // rows, and columns, of a CTA's operand tiles
constexpr int kDepth = 64;        // contraction elements of a stage (128-byte rows)
constexpr int kStages = 5;
constexpr uint32_t kTileBytes = kTile * kDepth * 2;
constexpr uint32_t kStageBytes = 2 * kTileBytes;
constexpr int kEpiWarps = 8, kProducerWarp = 8, kMmaWarp = 9;
constexpr int kThreads = 320;
constexpr int kMaxSegs = 6;
// Two groups of four warps finish 64 columns at a time, each through two slots of
// 128 rows x 64 columns: what is added comes in by TMA, the result is written in its place and
// leaves by TMA.  Values of two terms take both slots; of one term, where the result is
// symmetric, the second holds the tile transposed.  (Mirrored by stores from registers
// a tile of 128 x 64 took 4 us, with a box more to store 2.)
constexpr int kGroups = 2;
constexpr uint32_t kOffSlots = kStages * kStageBytes;
constexpr uint32_t kOffMisc = kOffSlots + kGroups * 2 * kTileBytes;
constexpr uint32_t kSmem = kOffMisc + 512;
static_assert(kSmem <= 232448, "shared memory budget");

struct Epilogue {
  float alpha, beta;            // value = (alpha acc + beta E) f^fpow, times the rescaling
  int e_terms;                  // of E: 0 without
  const MatInfo* info;          // f of each matrix
  int fpow;
  // results: o_terms terms by rows (sym: also mirrored, two terms at o), or the caller's tensor y,
  // through maps as well where its rows are at 16-byte steps (o_terms 0)
  int o_terms;
  __half* o[2];
  int old;
  void* y;
  int y_bf16, y_transposed, y_mapped;
  float* sums;                  // [count][parts of a matrix]: squares of the values, or null
  // rescaling by the norm of the step's input: [count][scale_parts] squares
  const float* scale_sums;
  int scale_parts, target;
  const int* exp_in;
  int* exp_out;
};

struct ProductArgs {
  CUtensorMap a[4], b[4], e[2], o[2];
  unsigned char seg_a[kMaxSegs], seg_b[kMaxSegs];
  int nseg;
  int rows, cols, depth, count;
  int sym;
  Epilogue ep;
  int* status;
  unsigned long long wait_ns;
};

// Instruction descriptor: fp16 operands (formats 0), fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

// The kernels of a call follow one another closely: each lets the next one start as soon as
// all its own blocks run, and begins to read and write when the one before is done.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

struct TileAt {
  int l, i, j, index;  // matrix, tile row and column, its number within the matrix
};
__device__ __forceinline__ TileAt tile_at(const ProductArgs& g, int t, int side) {
  const int tm = (g.rows + side - 1) / side, tn = (g.cols + side - 1) / side;
  const int per = g.sym ? tm * (tm + 1) / 2 : tm * tn;
  TileAt r;
  r.l = t / per;
  r.index = t - r.l * per;
  if (g.sym) {
    int i = (int)((sqrtf(8.f * r.index + 1.f) - 1.f) * 0.5f);
    while (i * (i + 1) / 2 > r.index) --i;
    while ((i + 1) * (i + 2) / 2 <= r.index) ++i;
    r.i = i;
    r.j = r.index - i * (i + 1) / 2;
  } else {  // a column of tiles after the other: its operand tile is shared
    r.j = r.index / tm;
    r.i = r.index - r.j * tm;
  }
  return r;
}

__device__ __forceinline__ void split(float v, __half& hi, __half& lo) {
  hi = __float2half_rn(v);
  lo = __float2half_rn(v - __half2float(hi));
}

// 32 columns (half h) of a thread's row in a slot: 16-byte chunks 4 h .. 4 h + 3.
__device__ __forceinline__ uint4* slot_chunk(uint8_t* slot, int row, int c) {
  return reinterpret_cast<uint4*>(slot + sw128_offset(row, c));
}
__device__ __forceinline__ f2 halves(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ uint32_t to_halves(f2 v) {
  const __half2 h = __floats2half2_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void add_slot(f2 (&v)[16], uint8_t* slot, int row, int h, float beta) {
  const f2 b = {beta, beta};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint4 x = *slot_chunk(slot, row, 4 * h + q);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) v[4 * q + k] = fma2(b, halves(w[k]), v[4 * q + k]);
  }
}
__device__ __forceinline__ void put_slot(const uint32_t (&w)[16], uint8_t* slot, int row, int h) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
    *slot_chunk(slot, row, 4 * h + q) = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
}
__device__ __forceinline__ void put_floats(const f2 (&v)[16], uint8_t* slot, int row) {
#pragma unroll
  for (int k = 0; k < 8; ++k)
    *reinterpret_cast<float4*>(slot_chunk(slot, row, k)) =
        make_float4(v[2 * k].x, v[2 * k].y, v[2 * k + 1].x, v[2 * k + 1].y);
}
// The same columns as rows of the transposed tile: two boxes of 64 rows x 64 columns,
// the tile's rows 0 .. 63 and 64 .. 127.  A warp's lanes write neighbouring elements.
__device__ __forceinline__ void put_slot_transposed(const uint32_t (&w)[16], uint8_t* slot, int row, int h) {
  const uint32_t box = smem_u32(slot) + (row >> 6) * (kTileBytes / 2) + (row & 7) * 2;
  const uint32_t chunk = (row & 63) >> 3;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const uint32_t c = 32 * h + 2 * k;
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(box + sw128_offset(c, chunk)),
                 "h"((unsigned short)(w[k] & 0xffffu))
                 : "memory");
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(box + sw128_offset(c + 1, chunk)),
                 "h"((unsigned short)(w[k] >> 16))
                 : "memory");
  }
}

// Writes 32 columns of a row in two terms to the mirrored place.  Neighbouring lanes hold
// neighbouring rows: they exchange halves, so that each writes two rows of every other
// column at once.  (An odd matrix's last pair reaches into the padding of its rows.)
__device__ __forceinline__ void put_mirrored(const uint32_t (&hi)[16], const uint32_t (&lo)[16],
                                             const Epilogue& e, size_t base, int row, int col, int rows,
                                             int cols) {
  const bool odd = row & 1;
  const int pair = row & ~1;
#pragma unroll
  for (int k = 0; k < 16; ++k) {  // columns 2k (low half) and 2k + 1
    // hi and lo of the column that the partner writes
    const uint32_t mine = odd ? (hi[k] & 0xffffu) | (lo[k] << 16) : (hi[k] >> 16) | (lo[k] & 0xffff0000u);
    const uint32_t other = __shfl_xor_sync(0xffffffffu, mine, 1);
    const int c = col + 2 * k + odd;
    const uint32_t h = odd ? (other & 0xffffu) | (hi[k] & 0xffff0000u) : (hi[k] & 0xffffu) | (other << 16);
    const uint32_t l = odd ? (other >> 16) | (lo[k] & 0xffff0000u) : (lo[k] & 0xffffu) | (other & 0xffff0000u);
    if (pair < rows && c < cols) {
      const size_t at = base + (size_t)c * e.old + pair;
      *reinterpret_cast<uint32_t*>(e.o[0] + at) = h;
      *reinterpret_cast<uint32_t*>(e.o[1] + at) = l;
    }
  }
}

// 32 values of a row straight to the caller's tensor, where no map can take them.
__device__ __forceinline__ void put_caller(const f2 (&v)[16], const ProductArgs& g, int l, int row, int col) {
  const Epilogue& e = g.ep;
  if (row >= g.rows) return;
  const size_t first = (size_t)l * g.rows * g.cols +
                       (e.y_transposed ? (size_t)col * g.rows + row : (size_t)row * g.cols + col);
  const size_t step = e.y_transposed ? g.rows : 1;
#pragma unroll
  for (int c = 0; c < 32; ++c)
    if (col + c < g.cols) {
      const float x = c & 1 ? v[c / 2].y : v[c / 2].x;
      if (e.y_bf16) static_cast<__nv_bfloat16*>(e.y)[first + c * step] = __float2bfloat16_rn(x);
      else static_cast<float*>(e.y)[first + c * step] = x;
    }
}

// The exponent that brings a matrix with sum of squares nu2 to a norm in
// (2^(target - 1), 2^target], or nearly; 0 for zeros and for what is not finite.
__device__ __forceinline__ int rescaling(float nu2, int target) {
  if (!(nu2 > 0.f) || nu2 > 3.0e38f) return 0;
  int e;
  frexpf(nu2, &e);  // nu2 < 2^e
  return target - ((e + 1) >> 1);
}

// acc = sum over segments of P Q^T (Q stored [cols, depth]) or P Q (NN: Q stored
// [depth, cols]); blocks stay and take tiles in turn.  Warps: 8 finish tiles, one
// loads, one multiplies; two accumulators, so that a tile is finished while the next
// is multiplied.  CTAS = 2: a pair of CTAs multiplies a tile of 256 x 256, each loading its
// 128 rows of P and 128 columns of Q, CTA 0 issuing for both.
template <int CTAS, bool NN>
__global__ void __launch_bounds__(kThreads, 1) product(const __grid_constant__ ProductArgs g) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  let_next_start();
  if (sb & 1023u) {  // 128-byte swizzled tiles need a 1024-byte aligned base
    if (threadIdx.x == 0) report_status(g.status, FBOB_ERR_CUDA);
    return;
  }
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kOffMisc);  // [kStages]
  uint64_t* empty = full + kStages;                               // [kStages]
  uint64_t* t_full = empty + kStages;                             // [2]
  uint64_t* t_empty = t_full + 2;                                 // [2]
  uint64_t* e_full = t_empty + 2;                                 // [kGroups][2]
  uint64_t* drain = e_full + 2 * kGroups;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc + 256);
  Abort* ab = reinterpret_cast<Abort*>(smem + kOffMisc + 264);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CTAS == 2 ? cluster_rank() : 0;
  constexpr int kSide = kTile * CTAS;
  constexpr uint32_t kCols = 2 * kSide;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(t_full + b, 1);
      mbar_init(t_empty + b, kEpiWarps * CTAS);
    }
    for (int i = 0; i < 2 * kGroups; ++i) mbar_init(e_full + i, 1);
    mbar_init(drain, 1);
    ab->flag = 0;
    ab->limit_ns = g.wait_ns;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    if (CTAS == 2) {
      tmem_alloc_pair(tmem_slot, kCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, kCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (CTAS == 2) cluster_sync();  // the other's barriers are there
  tc_fence_after();
  after_previous();
  const uint32_t tmem = *tmem_slot;
  const int tm = (g.rows + kSide - 1) / kSide, tn = (g.cols + kSide - 1) / kSide;
  const int per = g.sym ? tm * (tm + 1) / 2 : tm * tn;
  const int tiles = g.count * per;
  const int blocks = (g.depth + kDepth - 1) / kDepth;
  const int first = blockIdx.x / CTAS, step = gridDim.x / CTAS;

  if (warp == kProducerWarp) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int t = first; ok && t < tiles; t += step) {
        const TileAt at = tile_at(g, t, kSide);
        const int row = at.i * kSide + rank * kTile, col = at.j * kSide + rank * kTile;
        for (int sg = 0; ok && sg < g.nseg; ++sg) {
          const CUtensorMap* ma = &g.a[g.seg_a[sg]];
          const CUtensorMap* mb = &g.b[g.seg_b[sg]];
          for (int k = 0; k < blocks; ++k, ++it) {
            const int s = it % kStages;
            if (it >= kStages && !wait_bar(empty + s, ((it / kStages) - 1) & 1, ab, g.status)) {
              ok = false;
              break;
            }
            if (ab->flag) {
              ok = false;
              break;
            }
            uint8_t *pa = smem + s * kStageBytes, *pb = pa + kTileBytes;
            if (rank == 0) mbar_arrive_expect_tx(full + s, CTAS * kStageBytes);
            if (CTAS == 2) {
              const uint32_t bar = cluster_addr(full + s, 0);
              tma_load_3d_pair(pa, ma, bar, k * kDepth, row, at.l);
              if (NN) {
                tma_load_3d_pair(pb, mb, bar, col, k * kDepth, at.l);
                tma_load_3d_pair(pb + kTileBytes / 2, mb, bar, col + 64, k * kDepth, at.l);
              } else {
                tma_load_3d_pair(pb, mb, bar, k * kDepth, col, at.l);
              }
            } else {
              tma_load_3d(pa, ma, full + s, k * kDepth, row, at.l);
              if (NN) {
                tma_load_3d(pb, mb, full + s, col, k * kDepth, at.l);
                tma_load_3d(pb + kTileBytes / 2, mb, full + s, col + 64, k * kDepth, at.l);
              } else {
                tma_load_3d(pb, mb, full + s, k * kDepth, col, at.l);
              }
            }
          }
        }
      }
      // every load issued has landed before the block exits: CTA 0 sees the barriers
      // that count both CTAs' loads; what an abort leaves uncounted gets a fixed time
      if (rank == 0)
        for (int u = max(0, it - kStages); u < it; ++u)
          mbar_wait_bounded(full + u % kStages, (u / kStages) & 1, g.status, 100000000ull);
      if (CTAS == 2 && ab->flag) {
        const uint64_t t0 = global_ns();
        while (global_ns() - t0 < 10000000ull) __nanosleep(10000);
      }
    }
  } else if (warp == kMmaWarp) {
    if (rank == 0) {
      constexpr uint32_t id = idesc_f16(kSide, kSide, NN);
      int it = 0, n = 0;
      bool ok = true;
      for (int t = first; ok && t < tiles; t += step, ++n) {
        const uint32_t d = tmem + (n & 1) * kSide;
        if (n >= 2 && !warp_wait(t_empty + (n & 1), ((n >> 1) - 1) & 1, ab, g.status)) break;
        tc_fence_after();
        const int total = g.nseg * blocks;
        for (int k = 0; k < total; ++k, ++it) {
          const int s = it % kStages;
          if (!warp_wait(full + s, (it / kStages) & 1, ab, g.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a_lo = opaque(lo_kmajor(sb + s * kStageBytes));
          const uint32_t b_at = sb + s * kStageBytes + kTileBytes;
          const uint32_t b_lo = opaque(NN ? lo_mnmajor(b_at, kTileBytes / 2) : lo_kmajor(b_at));
#pragma unroll
          for (int u = 0; u < kDepth / 16; ++u) {
            const uint32_t al = a_lo + 2 * u, bl = b_lo + (NN ? kstep_off(u) : 2 * u);
            if (CTAS == 2) mma_ss_pair_w(d, al, bl, id, k + u > 0 ? 1u : 0u);
            else mma_ss_w(d, al, bl, id, k + u > 0 ? 1u : 0u);
          }
          if (CTAS == 2) mma_commit_pair_w(empty + s, 3);
          else mma_commit_w(empty + s);
        }
        if (!ok) break;
        if (CTAS == 2) mma_commit_pair_w(t_full + (n & 1), 3);
        else mma_commit_w(t_full + (n & 1));
      }
      // every MMA this warp issued has completed before TMEM is released
      if (CTAS == 2) mma_commit_pair_w(drain, 1);
      else mma_commit_w(drain);
      mbar_wait_bounded(drain, 0, g.status, 100000000ull);
    }
  } else {
    const Epilogue& e = g.ep;
    const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
    const int group = warp >> 2, r = 32 * (warp & 3) + lane;
    const bool issuer = (threadIdx.x & 127) == 0;
    uint8_t* const slots = smem + kOffSlots + group * 2 * kTileBytes;
    uint64_t* const e_bar = e_full + 2 * group;
    constexpr int kChunks = kSide / 64 / kGroups;  // of a tile, for each group
    const bool two = g.sym || e.e_terms == 2 || e.o_terms == 2 || (e.y_mapped && !e.y_bf16);
    const int nslots = two ? 1 : 2;
    const int mine = first < tiles ? ((tiles - 1 - first) / step + 1) * kChunks : 0;
    // the slot of chunk u is free once the result before it has left; then what is
    // added comes in
    auto prepare = [&](int u) {
      const int s = u % nslots;
      if (e.e_terms) {
        const TileAt at = tile_at(g, first + u / kChunks * step, kSide);
        const int row = at.i * kSide + rank * kTile;
        const int col = at.j * kSide + (group + u % kChunks * kGroups) * 64;
        mbar_arrive_expect_tx(e_bar + s, e.e_terms * kTileBytes);
        tma_load_3d(slots + s * kTileBytes, &g.e[0], e_bar + s, col, row, at.l);
        if (e.e_terms == 2) tma_load_3d(slots + kTileBytes, &g.e[1], e_bar + s, col, row, at.l);
      } else {
        mbar_arrive(e_bar + s);
      }
    };
    int ahead = 0;  // chunks prepared
    if (issuer)
      for (; ahead < nslots && ahead < mine; ++ahead) prepare(ahead);
    int n = 0, u = 0, scaled = -1, shift = 0;
    bool ok = true;
    // after an abort the loops run to their end without waiting, so that a group's warps
    // keep meeting at its barrier
    for (int t = first; t < tiles; t += step, ++n) {
      const TileAt at = tile_at(g, t, kSide);
      float alpha = e.alpha, beta = e.beta;
      if (e.fpow) {
        const float f = e.info[at.l].f, ff = e.fpow == 2 ? f * f : f;
        alpha *= ff;
        beta *= ff;
      }
      if (e.scale_sums) {
        if (scaled != at.l) {
          const float* p = e.scale_sums + (size_t)at.l * e.scale_parts;
          float nu2 = 0.f;
          for (int i = lane; i < e.scale_parts; i += 32) nu2 += p[i];
          shift = rescaling(warp_sum(nu2), e.target);
          scaled = at.l;
        }
        alpha = ldexpf(alpha, shift);
        beta = ldexpf(beta, shift);
        if (at.index == 0 && threadIdx.x == 0 && rank == 0) e.exp_out[at.l] = e.exp_in[at.l] + shift;
      }
      ok = ok && warp_wait(t_full + (n & 1), (n >> 1) & 1, ab, g.status);
      tc_fence_after();
      float sum = 0.f;
      const int row0 = at.i * kSide + rank * kTile, row = row0 + r;
#pragma unroll 1
      for (int c = 0; c < kChunks; ++c, ++u) {
        const int in_tile = (group + c * kGroups) * 64, col0 = at.j * kSide + in_tile;
        const int s = u % nslots;
        uint8_t* const slot = slots + s * kTileBytes;
        ok = ok && warp_wait(e_bar + s, (u / nslots) & 1, ab, g.status);
        const bool mirror = g.sym && at.i != at.j;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          const int col = col0 + 32 * h;
          uint32_t acc[32];
          tmem_ld32(tmem + lane_off + (n & 1) * kSide + in_tile + 32 * h, acc);
          f2 v[16];
#pragma unroll
          for (int k = 0; k < 16; ++k)
            v[k] = mul2(f2{alpha, alpha}, f2{__uint_as_float(acc[2 * k]), __uint_as_float(acc[2 * k + 1])});
          if (e.e_terms) add_slot(v, slot, r, h, beta);
          if (e.e_terms == 2) add_slot(v, slot + kTileBytes, r, h, beta);
          if (e.sums) {  // (what lies outside is zero)
#pragma unroll
            for (int k = 0; k < 16; ++k) sum = fmaf(v[k].x, v[k].x, fmaf(v[k].y, v[k].y, sum));
          }
          uint32_t w[16];
          if (e.o_terms) {
#pragma unroll
            for (int k = 0; k < 16; ++k) w[k] = to_halves(v[k]);
            put_slot(w, slot, r, h);
            if (e.o_terms == 2) {
              uint32_t lo[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) lo[k] = to_halves(fma2(f2{-1.f, -1.f}, halves(w[k]), v[k]));
              put_slot(lo, slot + kTileBytes, r, h);
              if (mirror)
                put_mirrored(w, lo, e, (size_t)at.l * g.rows * e.old, row, col, g.rows, g.cols);
            } else if (mirror) {
              put_slot_transposed(w, slot + kTileBytes, r, h);
            }
          } else if (!e.y_mapped) {
            put_caller(v, g, at.l, row, col);
          } else if (e.y_bf16) {
#pragma unroll
            for (int k = 0; k < 16; ++k) w[k] = pack_bf16(v[k].x, v[k].y);
            put_slot(w, slot, r, h);
          } else if (h == 0) {  // 32 fp32 columns fill a slot row: kept in both until all is read
#pragma unroll
            for (int k = 0; k < 8; ++k)
              *reinterpret_cast<float4*>(slot_chunk(slot + (k >> 2) * kTileBytes, r, k & 3)) =
                  make_float4(v[2 * k].x, v[2 * k].y, v[2 * k + 1].x, v[2 * k + 1].y);
          } else {
            float4 f[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              f[k] = *reinterpret_cast<float4*>(slot_chunk(slot + kTileBytes, r, k));
            put_floats(v, slot + kTileBytes, r);
#pragma unroll
            for (int k = 0; k < 4; ++k) *reinterpret_cast<float4*>(slot_chunk(slot, r, 4 + k)) = f[k];
          }
        }
        if (c == kChunks - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (CTAS == 2) mbar_arrive_cluster(cluster_addr(t_empty + (n & 1), 0));
            else mbar_arrive(t_empty + (n & 1));
          }
        }
        fence_async_smem();
        named_sync<128>(1 + group);
        if (issuer) {
          if ((e.o_terms || e.y_mapped) && row0 < g.rows && col0 < g.cols && !ab->flag) {
            tma_store_3d(&g.o[0], slot, col0, row0, at.l);
            if (e.o_terms == 2) {
              tma_store_3d(&g.o[1], slot + kTileBytes, col0, row0, at.l);
            } else if (mirror) {
              tma_store_3d(&g.o[1], slot + kTileBytes, row0, col0, at.l);
              if (row0 + 64 < g.rows)
                tma_store_3d(&g.o[1], slot + kTileBytes + kTileBytes / 2, row0 + 64, col0, at.l);
            }
            if (!e.o_terms && !e.y_bf16 && col0 + 32 < g.cols)
              tma_store_3d(&g.o[0], slot + kTileBytes, col0 + 32, row0, at.l);
            bulk_commit_group();
            bulk_wait_read_all();
          }
          if (ahead < mine && !ab->flag) prepare(ahead++);
        }
      }
      if (e.sums) {
        sum = warp_sum(sum);
        if (lane == 0)
          e.sums[((size_t)at.l * per + at.index) * (CTAS * kEpiWarps) + rank * kEpiWarps + warp] = sum;
      }
    }
    if (issuer) {
      bulk_wait_all();
      // what was loaded ahead has landed (after an abort some was never awaited)
      for (int k = max(0, ahead - nslots); k < ahead; ++k)
        mbar_wait_bounded(e_bar + k % nslots, (k / nslots) & 1, g.status, 100000000ull);
    }
  }
  tc_fence_before();
  __syncthreads();
  __syncwarp();
  if (CTAS == 2) cluster_sync();  // neither leaves before the other's last use of it
  if (warp == kMmaWarp) {
    tc_fence_after();
    if (CTAS == 2) tmem_dealloc_pair(tmem, kCols);
    else tmem_dealloc(tmem, kCols);
  }
}

// ---------------------------------------------------------------------------
// Norms, packing, and the end of the gradient
// ---------------------------------------------------------------------------
constexpr int kSumThreads = 256;

// partial[l][block] = sum of squares of a slice of matrix l; also clears the call's
// status word, before every kernel that may write it.
template <typename T>
__global__ void __launch_bounds__(kSumThreads)
    square_sums(const T* __restrict__ x, float* __restrict__ partial, size_t elems, int* status) {
  __shared__ float sm[kSumThreads / 32];
  let_next_start();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *status = 0;
  x += (size_t)blockIdx.y * elems;
  const size_t per = (elems + gridDim.x - 1) / gridDim.x;
  const size_t first = blockIdx.x * per, last = min(elems, first + per);
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  size_t i = first + threadIdx.x;
  for (; i + 3 * kSumThreads < last; i += 4 * kSumThreads) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float v = to_f32<T>(x[i + u * kSumThreads]);
      s[u] = fmaf(v, v, s[u]);
    }
  }
  for (; i < last; i += kSumThreads) {
    const float v = to_f32<T>(x[i]);
    s[0] = fmaf(v, v, s[0]);
  }
  const float w = warp_sum((s[0] + s[1]) + (s[2] + s[3]));
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = w;
  __syncthreads();
  if (threadIdx.x == 0) {
    float t = 0.f;
    for (int k = 0; k < kSumThreads / 32; ++k) t += sm[k];
    partial[(size_t)blockIdx.y * gridDim.x + blockIdx.x] = t;
  }
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

struct PackArgs {
  const void* x;       // [count][m][n]
  const float* sums;   // [count][parts] squares
  int parts;
  __half *hi, *lo;     // [count][p][ld]
  int p, q, ld, tall;
  float eps;
  int target;
  // forward: the matrices' scales; backward (info null): their exponents and square sums
  MatInfo* info;
  int* exp_out;
  float* sums_out;
};

constexpr int kPack = 64;  // rows and columns of a block's tile

// x times a power of two, in fp16 terms, the shorter side first.
template <typename T>
__global__ void __launch_bounds__(kSumThreads) pack(PackArgs a) {
  __shared__ float sm[kSumThreads / 32];
  __shared__ float tile[kPack][kPack + 1];
  const int l = blockIdx.z;
  let_next_start();
  after_previous();
  const float nu2 = parts_sum(a.sums + (size_t)l * a.parts, a.parts, sm);
  const bool writer = blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0;
  float factor;
  if (a.info) {
    MatInfo r;
    r.norm = sqrtf(nu2);
    r.s = 1.f / (r.norm + a.eps);
    if (r.s > 0.f && r.s < 3.0e38f) {
      int e;
      r.f = 2.f * frexpf(r.s, &e);  // s = f 2^(e - 1)
      r.k = e - 1;
      factor = ldexpf(1.f, r.k + a.target);
    } else {  // an infinite or NaN norm, or 0 and eps = 0: zeros and NaN as s G gives them
      r.f = 1.f;
      r.k = 0;
      factor = r.s;
    }
    if (writer) a.info[l] = r;
  } else {
    const int e = rescaling(nu2, a.target);
    factor = ldexpf(1.f, e);
    if (writer) {
      a.exp_out[l] = e;
      a.sums_out[l] = nu2 * factor * factor;
    }
  }
  const T* x = static_cast<const T*>(a.x) + (size_t)l * a.p * a.q;
  const size_t base = (size_t)l * a.p * a.ld;
  const int r0 = blockIdx.y * kPack, c0 = blockIdx.x * kPack;  // of the packed matrix
  if (a.tall) {
    for (int i = threadIdx.x; i < kPack * kPack; i += kSumThreads) {
      const int c = i / kPack, r = i % kPack;  // x is [q][p]
      if (c0 + c < a.q && r0 + r < a.p) tile[r][c] = to_f32<T>(x[(size_t)(c0 + c) * a.p + r0 + r]);
    }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < kPack * kPack; i += kSumThreads) {
    const int r = i / kPack, c = i % kPack;
    if (r0 + r >= a.p || c0 + c >= a.q) continue;
    const float v = (a.tall ? tile[r][c] : to_f32<T>(x[(size_t)(r0 + r) * a.q + c0 + c])) * factor;
    __half hi, lo;
    split(v, hi, lo);
    a.hi[base + (size_t)(r0 + r) * a.ld + c0 + c] = hi;
    if (a.lo) a.lo[base + (size_t)(r0 + r) * a.ld + c0 + c] = lo;
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
    float h[8] = {}, x[8] = {};
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (a.h[t]) {
        const uint4 v = *reinterpret_cast<const uint4*>(a.h[t] + at);
        const __half* w = reinterpret_cast<const __half*>(&v);
#pragma unroll
        for (int k = 0; k < 8; ++k) h[k] += __half2float(w[k]);
      }
      if (a.x[t]) {
        const uint4 v = *reinterpret_cast<const uint4*>(a.x[t] + at);
        const __half* w = reinterpret_cast<const __half*>(&v);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] += __half2float(w[k]);
      }
    }
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

// dG = s (H_0 - G <H_0, G> s / norm)
template <typename T>
__global__ void __launch_bounds__(kSumThreads) end_gradient(EndArgs a) {
  __shared__ float sm[kSumThreads / 32];
  __shared__ float tile[kPack][kPack + 1];
  const int l = blockIdx.z;
  after_previous();
  const MatInfo r = a.info[l];
  const float dot = parts_sum(a.dots + (size_t)l * a.parts, a.parts, sm);
  // <h, G> = dot 2^-(k + x_exp); a zero matrix has no direction to take off
  const double along = r.norm > 0.f ? ldexp((double)dot, -(r.k + a.x_exp)) * r.s / r.norm : 0.0;
  const double scale = ldexp((double)r.s, -a.exp[l]);
  const float by_h = (float)scale, by_g = (float)(scale * along);
  const size_t n = (size_t)l * a.p * a.q;
  const int r0 = blockIdx.y * kPack, c0 = blockIdx.x * kPack;  // of h
  const size_t base = (size_t)l * a.p * a.ld;
  const T* g = static_cast<const T*>(a.g) + n;
  T* dg = static_cast<T*>(a.dg) + n;
  auto value = [&](int rr, int c) {
    const size_t at = base + (size_t)(r0 + rr) * a.ld + c0 + c;
    return __half2float(a.h[0][at]) + (a.h[1] ? __half2float(a.h[1][at]) : 0.f);
  };
  if (a.tall) {
    for (int i = threadIdx.x; i < kPack * kPack; i += kSumThreads) {
      const int rr = i / kPack, c = i % kPack;
      if (r0 + rr < a.p && c0 + c < a.q) tile[rr][c] = value(rr, c);
    }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < kPack * kPack; i += kSumThreads) {
    const int rr = a.tall ? i % kPack : i / kPack, c = a.tall ? i / kPack : i % kPack;
    if (r0 + rr >= a.p || c0 + c >= a.q) continue;
    const size_t at = a.tall ? (size_t)(c0 + c) * a.p + r0 + rr : (size_t)(r0 + rr) * a.q + c0 + c;
    const float v = a.tall ? tile[rr][c] : value(rr, c);
    dg[at] = from_f32<T>(fmaf(-by_g, to_f32<T>(g[at]), by_h * v));
  }
}

// ---------------------------------------------------------------------------
// Host: scales, workspace, launches
// ---------------------------------------------------------------------------
constexpr int kMaxSteps = 16;

struct Plan {
  int L, m, n, p, q, ldq, ldp, steps, bf16, keep, tall;
  float eps;
  float a[kMaxSteps], b[kMaxSteps], c[kMaxSteps];
  int xe[kMaxSteps], ae[kMaxSteps], be[kMaxSteps];  // exponents of X, A, B as stored
  int xt[kMaxSteps];                                // terms of X
  double M[kMaxSteps + 1];                          // bound on X's singular values
  int square_parts;
};

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
  double M = 1.0;
  p.M[0] = M;
  for (int i = 0; i < p.steps; ++i) {
    const double a = o->coefficients[3 * i], b = o->coefficients[3 * i + 1], c = o->coefficients[3 * i + 2];
    if (!(fabs(a) < 1e6 && fabs(b) < 1e6 && fabs(c) < 1e6)) return FBOB_ERR_INVALID_ARG;
    p.a[i] = (float)a; p.b[i] = (float)b; p.c[i] = (float)c;
    p.xe[i] = store_exp(M);
    p.ae[i] = store_exp(M * M);
    p.be[i] = store_exp(fabs(b) * M * M + fabs(c) * M * M * M * M);
    double most = 0;  // of the polynomial up to M, which rounding may pass a little
    for (int k = 0; k <= 1024; ++k) {
      const double x = 1.01 * M * k / 1024, y = fabs(x * (a + x * x * (b + x * x * c)));
      if (y > most) most = y;
    }
    M = 1.01 * most;
    if (!(M < 64.0)) return FBOB_ERR_INVALID_ARG;  // singular values that run away
    p.M[i + 1] = M;
  }
  // terms of X: the growth of a rounding error by the steps that follow
  double growth = 1;
  for (int i = p.steps - 1; i >= 0; --i) {
    growth *= fabs(p.a[i]) > 1 ? fabs(p.a[i]) : 1;
    // (a bf16 G is one fp16 term, times a power of two)
    p.xt[i] = !p.bf16 || (growth > 16 && i > 0) ? 2 : 1;
  }
  const long long elems = (long long)p.p * p.q;
  const long long parts = (elems + 8191) / 8192;
  p.square_parts = (int)(parts < 1024 ? parts : 1024);
  *out = p;
  return FBOB_OK;
}

// A map of [count][rows][ld] elements, cols of each row; a box: 128 bytes of box_rows rows.
bool make_tile_map(CUtensorMap* m, CUtensorMapDataType type, int size, const void* ptr, int L, int rows,
                   int cols, long long ld, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)L};
  cuuint64_t strides[2] = {(cuuint64_t)ld * size, (cuuint64_t)rows * ld * size};
  cuuint32_t box[3] = {(cuuint32_t)(128 / size), (cuuint32_t)box_rows, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return fn(m, type, 3, const_cast<void*>(ptr), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Carver {
  char* base;
  size_t off;
  bool ok;
  void* take(size_t bytes) {
    void* r = base ? base + off : nullptr;
    off += align_up(bytes);
    return r;
  }
  Terms terms(const Plan& p, int cols, int ld, int n) {
    Terms t;
    const size_t one = (size_t)p.L * p.p * ld * sizeof(__half);
    t.hi = static_cast<__half*>(take(one));
    t.lo = n == 2 ? static_cast<__half*>(take(one)) : nullptr;
    t.rows = p.p; t.cols = cols; t.ld = ld;
    for (int i = 0; base && i < n; ++i) {
      const __half* at = i ? t.lo : t.hi;
      const auto half = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
      ok = ok && make_tile_map(&t.tile[i], half, 2, at, p.L, p.p, cols, ld, kTile);
      ok = ok && make_tile_map(&t.step[i], half, 2, at, p.L, p.p, cols, ld, kDepth);
    }
    return t;
  }
};

// CTAs that share a tile of a rows x cols product.
int product_ctas(const Plan& p, int rows, int cols, bool sym) {
  return getenv("ORTH_CTAS") ? atoi(getenv("ORTH_CTAS")) : 2;
}
int product_tiles(int rows, int cols, bool sym, int ctas) {  // of one matrix
  const int side = kTile * ctas, tm = (rows + side - 1) / side, tn = (cols + side - 1) / side;
  return sym ? tm * (tm + 1) / 2 : tm * tn;
}
int product_parts(const Plan& p) {  // sums of a [p, q] product
  const int ctas = product_ctas(p, p.p, p.q, false);
  return product_tiles(p.p, p.q, false, ctas) * ctas * kEpiWarps;
}

// Forward: [status][info][square sums], then X, A and B of each step (kept), or of two
// and one (X in turn).
struct Forward {
  int* status;
  MatInfo* info;
  float* sums;
  Terms X[kMaxSteps], A[kMaxSteps], B[kMaxSteps];
  bool ok;
  size_t bytes;
};
Forward carve_forward(const Plan& p, char* base) {
  Forward w;
  Carver c{base, 0, true};
  w.status = static_cast<int*>(c.take(sizeof(int)));
  w.info = static_cast<MatInfo*>(c.take(sizeof(MatInfo) * p.L));
  w.sums = static_cast<float*>(c.take(sizeof(float) * p.L * p.square_parts));
  const int small = p.bf16 ? 1 : 2;
  Terms turn[2];  // without keep: room for every step that shares one
  for (int i = 0; !p.keep && i < 2; ++i) {
    int t = 1;
    for (int k = i; k < p.steps; k += 2) t = p.xt[k] > t ? p.xt[k] : t;
    turn[i] = c.terms(p, p.q, p.ldq, t);
  }
  for (int i = 0; i < p.steps; ++i) {
    w.X[i] = p.keep ? c.terms(p, p.q, p.ldq, p.xt[i]) : turn[i & 1];
    if (p.xt[i] == 1) w.X[i].lo = nullptr;
    if (p.keep || i == 0) {
      w.A[i] = c.terms(p, p.p, p.ldp, small);
      w.B[i] = c.terms(p, p.p, p.ldp, small);
    } else {
      w.A[i] = w.A[0];
      w.B[i] = w.B[0];
    }
  }
  w.ok = c.ok;
  w.bytes = c.off;
  return w;
}

// Backward: [status][square sums of dY][exponents: steps + 1][sums of the steps'
// results: two in turn], H in turn, S, T.
struct Backward {
  int* status;
  float *sums, *first, *step_sums[2];
  int* exp[kMaxSteps + 1];
  Terms H[2], S, T;
  bool ok;
  size_t bytes;
};
Backward carve_backward(const Plan& p, char* base) {
  Backward w;
  Carver c{base, 0, true};
  const int t = p.bf16 ? 1 : 2;
  w.status = static_cast<int*>(c.take(sizeof(int)));
  w.sums = static_cast<float*>(c.take(sizeof(float) * p.L * p.square_parts));
  w.first = static_cast<float*>(c.take(sizeof(float) * p.L));
  for (float*& s : w.step_sums) s = static_cast<float*>(c.take(sizeof(float) * p.L * product_parts(p)));
  for (int i = 0; i <= p.steps; ++i) w.exp[i] = static_cast<int*>(c.take(sizeof(int) * p.L));
  for (Terms& h : w.H) h = c.terms(p, p.q, p.ldq, t);
  w.S = c.terms(p, p.p, p.ldp, t);
  w.T = c.terms(p, p.p, p.ldp, t);
  w.ok = c.ok;
  w.bytes = c.off;
  return w;
}

// Launches a kernel that may start while the one before it in the stream ends.
template <typename... P, typename... A>
cudaError_t launch_next(void (*kernel)(P...), dim3 grid, int threads, size_t smem, int cluster,
                        LaunchLog& log, A... args) {
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

// Builds and launches one product.
struct Product {
  ProductArgs g;
  int na = 0, nb = 0, high_a[2], high_b[2], highs = 0, ctas;
  bool nn;
  Product(const Plan& p, const Terms& out, int depth, bool nn_, bool sym, int* status) : nn(nn_) {
    memset(&g, 0, sizeof g);
    ctas = product_ctas(p, out.rows, out.cols, sym);
    g.rows = out.rows;
    g.cols = out.cols;
    g.depth = depth;
    g.count = p.L;
    g.sym = sym;
    g.status = status;
    g.wait_ns = wait_limit_ns();
  }
  // acc += P Q^T (or P Q): every pair of terms but the two low ones
  void add(const Terms& P, const Terms& Q) {
    const int a0 = na, b0 = nb;
    g.a[na++] = P.tile[0];
    if (P.lo) g.a[na++] = P.tile[1];
    g.b[nb++] = nn ? Q.step[0] : Q.tile[0];
    if (Q.lo) g.b[nb++] = nn ? Q.step[1] : Q.tile[1];
    if (Q.lo) pair(a0, b0 + 1);
    if (P.lo) pair(a0 + 1, b0);
    high_a[highs] = a0;
    high_b[highs++] = b0;
  }
  void pair(int a, int b) {
    g.seg_a[g.nseg] = (unsigned char)a;
    g.seg_b[g.nseg++] = (unsigned char)b;
  }
  void plus(const Terms& E) {
    g.ep.e_terms = E.lo ? 2 : 1;
    g.e[0] = E.tile[0];
    g.e[1] = E.tile[1];
  }
  void to(const Terms& O) {
    g.ep.o_terms = O.lo ? 2 : 1;
    g.o[0] = O.tile[0];
    g.o[1] = O.lo ? O.tile[1] : O.step[0];  // one term: mirrored in boxes of 64 rows
    g.ep.o[0] = O.hi;
    g.ep.o[1] = O.lo;
    g.ep.old = O.ld;
  }
  // the caller's tensor, by rows (its map where one can be made) or transposed
  void to_caller(const Plan& p, void* y) {
    const int size = p.bf16 ? 2 : 4;
    g.ep.y = y;
    g.ep.y_bf16 = p.bf16;
    g.ep.y_transposed = p.tall;
    g.ep.y_mapped = !p.tall && (reinterpret_cast<uintptr_t>(y) & 15u) == 0 && p.q * size % 16 == 0 &&
                    make_tile_map(&g.o[0], p.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                  : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                                  size, y, p.L, p.p, p.q, p.q, kTile);
  }
  cudaError_t launch(LaunchLog& log) {
    // The products of high terms come last: the tensor cores cut every addition off to the
    // accumulator's 24 bits, which costs nothing while it holds the small ones only.
    for (int i = 0; i < highs; ++i) pair(high_a[i], high_b[i]);
    const long long tiles = (long long)g.count * product_tiles(g.rows, g.cols, g.sym, ctas);
    const long long most = kSms / ctas;
    const int grid = (int)(tiles < most ? tiles : most) * ctas;
    auto kernel = ctas == 2 ? (nn ? product<2, true> : product<2, false>)
                            : (nn ? product<1, true> : product<1, false>);
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    return launch_next(kernel, dim3((unsigned)grid), kThreads, kSmem, ctas, log, g);
  }
};

cudaError_t squares_and_pack(const Plan& p, const void* x, float* sums, int* status, PackArgs a,
                             LaunchLog& log) {
  const size_t elems = (size_t)p.p * p.q;
  const dim3 grid((unsigned)p.square_parts, (unsigned)p.L);
  if (p.bf16)
    square_sums<<<grid, kSumThreads, 0, log.stream>>>(static_cast<const __nv_bfloat16*>(x), sums, elems, status);
  else
    square_sums<<<grid, kSumThreads, 0, log.stream>>>(static_cast<const float*>(x), sums, elems, status);
  cudaError_t e = cudaGetLastError();
  log.mark();
  if (e != cudaSuccess) return e;
  a.x = x;
  a.sums = sums;
  a.parts = p.square_parts;
  a.p = p.p; a.q = p.q; a.ld = p.ldq; a.tall = p.tall;
  a.eps = p.eps;
  const dim3 tiles((unsigned)((p.q + kPack - 1) / kPack), (unsigned)((p.p + kPack - 1) / kPack), (unsigned)p.L);
  return launch_next(p.bf16 ? pack<__nv_bfloat16> : pack<float>, tiles, kSumThreads, 0, 1, log, a);
}

float pow2(int e) { return ldexpf(1.f, e); }

cudaError_t forward(const Plan& p, const void* G, void* Y, const Forward& w, LaunchLog& log) {
  PackArgs a = {};
  a.hi = w.X[0].hi;
  a.lo = w.X[0].lo;
  a.target = p.xe[0];
  a.info = w.info;
  cudaError_t e = squares_and_pack(p, G, w.sums, w.status, a, log);
  for (int i = 0; e == cudaSuccess && i < p.steps; ++i) {
    const Terms &X = w.X[i], &A = w.A[i], &B = w.B[i];
    Terms Xm = X;  // as it is multiplied
    if (p.bf16) Xm.lo = nullptr;
    {
      Product g(p, A, p.q, false, true, w.status);
      g.add(Xm, Xm);
      g.g.ep.alpha = pow2(p.ae[i] - 2 * p.xe[i]);
      if (i == 0) {
        g.g.ep.info = w.info;
        g.g.ep.fpow = 2;
      }
      g.to(A);
      e = g.launch(log);
    }
    if (e != cudaSuccess) break;
    {
      Product g(p, B, p.p, false, true, w.status);
      g.add(A, A);
      g.plus(A);
      g.g.ep.alpha = p.c[i] * pow2(p.be[i] - 2 * p.ae[i]);
      g.g.ep.beta = p.b[i] * pow2(p.be[i] - p.ae[i]);
      g.to(B);
      e = g.launch(log);
    }
    if (e != cudaSuccess) break;
    const bool last = i + 1 == p.steps;
    Product g(p, X, p.p, true, false, w.status);
    g.add(B, Xm);
    g.plus(X);
    const int out = last ? 0 : p.xe[i + 1];
    g.g.ep.alpha = pow2(out - p.be[i] - p.xe[i]);
    g.g.ep.beta = p.a[i] * pow2(out - p.xe[i]);
    if (i == 0) {
      g.g.ep.info = w.info;
      g.g.ep.fpow = 1;
    }
    if (last) {
      g.to_caller(p, Y);
    } else {
      g.to(w.X[i + 1]);
    }
    e = g.launch(log);
  }
  return e;
}

cudaError_t backward(const Plan& p, const void* G, const void* dY, void* dG, const Forward& f,
                     const Backward& w, LaunchLog& log) {
  // H's norm is brought to 2^target: every entry of H, S, T and of the next H stays below
  // 2^15 whatever their directions
  int target[kMaxSteps], se[kMaxSteps];
  for (int i = 0; i < p.steps; ++i) {
    const double M = p.M[i], a = fabs(p.a[i]), b = fabs(p.b[i]), c = fabs(p.c[i]);
    const double growth = a + 3 * b * M * M + 5 * c * M * M * M * M;
    const double t = (b + 2 * c * M * M) * 2 * M;
    double most = 15 - log2(growth > 1 ? growth : 1);
    const double by_t = 15 - log2(t > 1e-30 ? t : 1e-30) - (p.be[i] - p.xe[i]);
    if (by_t < most) most = by_t;
    target[i] = (int)floor(most) < 12 ? (int)floor(most) : 12;
    se[i] = store_exp(pow2(target[i]) * 2 * M);
  }
  const int top = p.steps - 1;
  PackArgs a = {};
  a.hi = w.H[0].hi;
  a.lo = w.H[0].lo;
  a.target = target[top];
  a.exp_out = w.exp[p.steps];
  a.sums_out = w.first;
  cudaError_t e = squares_and_pack(p, dY, w.sums, w.status, a, log);
  const float* sums = w.first;
  int parts = 1, turn = 0;
  for (int i = top; e == cudaSuccess && i >= 0; --i, turn ^= 1) {
    const Terms &H = w.H[turn], &A = f.A[i], &B = f.B[i];
    Terms X = f.X[i];
    if (p.bf16) X.lo = nullptr;
    {
      Product g(p, w.S, p.q, false, true, w.status);
      g.add(H, X);
      g.add(X, H);
      g.g.ep.alpha = pow2(se[i] - p.xe[i]);
      if (i == 0) {
        g.g.ep.info = f.info;
        g.g.ep.fpow = 1;
      }
      g.to(w.S);
      e = g.launch(log);
    }
    if (e != cudaSuccess) break;
    const int te = p.be[i] - p.xe[i];  // T X and B H share an accumulator
    {
      Product g(p, w.T, p.p, false, true, w.status);
      g.add(A, w.S);
      g.add(w.S, A);
      g.plus(w.S);
      g.g.ep.alpha = p.c[i] * pow2(te - p.ae[i] - se[i]);
      g.g.ep.beta = p.b[i] * pow2(te - se[i]);
      if (i == 0) {  // X_0 is f times what is stored
        g.g.ep.info = f.info;
        g.g.ep.fpow = 1;
      }
      g.to(w.T);
      e = g.launch(log);
    }
    if (e != cudaSuccess) break;
    Product g(p, H, p.p, true, false, w.status);
    g.add(B, H);
    g.add(w.T, X);
    g.plus(H);
    g.g.ep.alpha = pow2(-p.be[i]);
    g.g.ep.beta = p.a[i];
    g.g.ep.sums = i > 0 ? w.step_sums[turn] : nullptr;
    g.g.ep.scale_sums = sums;
    g.g.ep.scale_parts = parts;
    g.g.ep.target = i > 0 ? target[i - 1] : 12;
    g.g.ep.exp_in = w.exp[i + 1];
    g.g.ep.exp_out = w.exp[i];
    g.to(w.H[turn ^ 1]);
    sums = w.step_sums[turn];
    parts = product_parts(p);
    e = g.launch(log);
  }
  if (e != cudaSuccess) return e;
  const Terms &H0 = w.H[turn], &X0 = f.X[0];
  DotArgs d = {};
  d.h[0] = H0.hi;
  d.h[1] = H0.lo;
  d.x[0] = X0.hi;
  d.x[1] = X0.lo;
  d.partial = w.sums;
  d.p = p.p; d.q = p.q; d.ld = p.ldq;
  e = launch_next(term_dots, dim3((unsigned)p.square_parts, (unsigned)p.L), kSumThreads, 0, 1, log, d);
  if (e != cudaSuccess) return e;
  EndArgs n = {};
  n.g = G;
  n.dg = dG;
  n.h[0] = H0.hi;
  n.h[1] = H0.lo;
  n.dots = w.sums;
  n.parts = p.square_parts;
  n.p = p.p; n.q = p.q; n.ld = p.ldq; n.tall = p.tall; n.x_exp = p.xe[0];
  n.info = f.info;
  n.exp = w.exp[0];
  const dim3 tiles((unsigned)((p.q + kPack - 1) / kPack), (unsigned)((p.p + kPack - 1) / kPack), (unsigned)p.L);
  return launch_next(p.bf16 ? end_gradient<__nv_bfloat16> : end_gradient<float>, tiles, kSumThreads, 0, 1,
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
  const Forward w = carve_forward(p, static_cast<char*>(ws));
  if (!w.ok) return FBOB_ERR_CUDA;
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
  const Forward f = carve_forward(p, const_cast<char*>(static_cast<const char*>(kept)));
  const Backward w = carve_backward(p, static_cast<char*>(ws));
  if (!f.ok || !w.ok) return FBOB_ERR_CUDA;
  LaunchLog log{static_cast<cudaStream_t>(stream)};
  begin_call(log);
  const cudaError_t e = backward(p, g, dy, dg, f, w, log);
  end_call(log);
  return e == cudaSuccess ? FBOB_OK : FBOB_ERR_CUDA;
}

}  // extern "C"
