// Differential attention on the tensor cores (tcgen05 / TMEM / TMA), bf16, d and
// dv multiples of 8 up to 128.  The kernels are built for widths D and DV of 64
// and 128; narrower rows arrive with zeros behind them (the copies fill in what
// is past a row's end, and leave it out when they store).  Per head, with
// m = 1, 2 (code: 0, 1) and c the scale,
//   S^m = c Q^m K^mT, P^m = softmax(S^m), O = P^1 V - lam P^2 V;
//   dP = dO V^T, D^m = dO . O^m, dS^1 = P^1*(dP - D^1),
//   dS^2 = -lam P^2*(dP - D^2), dQ^m = c dS^m K^m, dK^m = c dS^mT Q^m,
//   dV = (P^1 - lam P^2)^T dO, dlam_i = -sum_j P^2_ij dP_ij.
//
// The two maps are two score streams over one stream of values: scores of map m
// have a TMEM buffer of their own, so the tensor pipe works on one map while the
// elementwise warps work on the other.
//
// forward (128 query rows per CTA, 128-key tiles): online softmax of both
//   maps, O^1 and O^2 in TMEM, the difference taken once in the epilogue in
//   fp32.  V is loaded once for both products.
// row pass (128 query rows, key tiles of 128 at d = 64 and 64 at d = 128): dQ of
//   both maps.  dP is computed once per tile and stays in registers for the
//   second map.
// column pass (128 key rows, 64-query tiles): dK of both maps and dV, whose
//   two products are one: W = P^1 - lam P^2 is formed in fp32 and multiplied
//   with dO once.  A CTA loops over the query heads that share its key head, or
//   over a part of their queries (col_parts).
// The row and the column pass recompute the scores rather than exchange dQ
// through atomics: every output is accumulated by one CTA in a fixed order, or by
// one per part, with the parts added in their order.
//
// Probabilities, W and dS are rounded to bf16 as operands of the second
// products, the precision of the tensors they are multiplied with; scores,
// softmax statistics, row scalars and every accumulator are fp32.
//
// Warp roles: elementwise warps (warp w: TMEM lane quadrant w % 4; 16 of them in
// the backward passes, each thread a quarter of a row; 8 in the forward, each
// thread a row of one map), one TMA producer, one MMA issuer.  Every wait is
// bounded, and every warp-collective operation sits in warp-uniform control
// flow.
//
// What bounds the passes (B = 1, H = 8, N = 16384, causal, dv = 128; time, and
// what the products they run come to as a share of the measured matmul rate of
// 1917 TFLOP/s):
//            forward        row pass        column pass
//   d = 64   582 us, 74%    572 us, 75%     960 us, 60%
//   d = 128  645 us, 89%    949 us, 76%     1371 us, 63%
// (of which the producers' look at the abort flag is 6 us of the forward at d = 64
// and 15 us of the column pass at d = 128).
// The chain scores -> exponentials -> product within a tile: the accumulators
// leave TMEM for one or two buffers per map, so pipe and elementwise warps wait
// for each other, and each hand-over costs 100 to 250 cycles on either side.  At
// d = 64 a tile of the forward takes 2335 cycles against 1536 of products, one
// of the row pass 2150 against 1536, and a 64-query tile of the column pass 2095
// against 1255.  In the column pass the products and the scalars' loads together
// keep shared memory 75% busy; without any elementwise arithmetic it would take
// 833 us.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <float.h>
#include <math.h>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "ops.h"
#include "sm103.cuh"
#include "tc_common.cuh"

namespace fbob {

using namespace sm103;
using namespace tc;

namespace {

constexpr int kWarps = 16;                 // elementwise warps
constexpr int kConsumers = kWarps * 32;
constexpr int kProducerWarp = kWarps;
constexpr int kMmaWarp = kWarps + 1;
constexpr int kThreads = (kWarps + 2) * 32;
constexpr int kRowSlices = kWarps / 4;     // column slices per row
// Forward: 4 softmax warps per map, one thread per row of 128 scores (no
// exchange between threads), a producer and an MMA warp, so that a thread has
// 168 registers.  16 warps of 96 registers, which exchanged each row's maximum,
// took 733 us at N = 16384 where this then took 605.
constexpr int kSoftmax = 8 * 32;
constexpr int kFwdProducer = 8, kFwdMma = 9, kFwdThreads = 10 * 32;
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint64_t kDrainNs = 100000000ull;  // limit of the waits after an abort
constexpr uint32_t kMinusInf = 0xff800000u;

struct Common {
  int* status;
  unsigned long long wait_ns;  // limit of one bounded wait
  int N, causal;
  int H, G;        // query heads, and those per key head
  int units, group;  // CTA grid: heads, heads per group (cta_coord)
  float scale;
  bool narrow_d, narrow_v;  // d < D, dv < DV (kernels with NARROW: a test of
                            // these in all cost the others 1%)
  LamArg lam;
};

__device__ __forceinline__ float lam_value(const LamArg& l, size_t i) {
  return l.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(l.p)[i])
                : static_cast<const float*>(l.p)[i];
}
// lam of row n of head bh = b H + h
__device__ __forceinline__ float lam_row(const LamArg& l, int bh, int H, int N, int n) {
  return lam_value(l, l.kind == FBOB_LAM_ONE ? 0 : l.kind == FBOB_LAM_HEAD ? (size_t)(bh % H)
                                                                           : (size_t)bh * N + n);
}

// Bounded wait.  It sleeps on the barrier before it looks at the clock: almost
// every wait ends in that sleep, and a read of the global timer costs more than
// most of them last.  A wait that runs out records the timeout and sets the
// CTA's abort flag; it returns all the same, and so do all later waits at
// once.  So control flow stays the same in every lane without a vote (which
// cost 3% to 4% of each kernel), the roles run to their ends on whatever the
// buffers hold, and only the producers stop: the call's outputs are undefined,
// every access stays in bounds, and the CTA drains its copies and MMAs and
// frees its TMEM as ever.
__device__ __forceinline__ void await(uint64_t* bar, uint32_t parity, Abort* ab, int* status) {
  if (mbar_try_wait(bar, parity) || ab->flag) return;
  const uint64_t limit = ab->limit_ns;
  if (mbar_try_wait_sleep(bar, parity, limit < kPollSleepNs ? (uint32_t)limit : kPollSleepNs)) return;
  wait_bar(bar, parity, ab, status);
}

// The producers' wait for a free stage.  Behind the abort flag the MMA warp's
// commits free stages whose copies have not landed yet, and another copy would
// arrive on their barrier once more than it counts (which ends the context): the
// flag is up before such a commit, so it is looked at behind the wait.
__device__ __forceinline__ bool stage_free(uint64_t* bar, uint32_t parity, Abort* ab, int* status) {
  return wait_bar(bar, parity, ab, status) && !ab->flag;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// One arrival for the whole warp: its lanes' earlier writes (shared memory, or
// TMEM behind tc_fence_before) are ordered before it.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// Row scalars of the backward, in blocks of 64 rows so that a query tile's are
// one copy: [B H][ceil(N / 64)][5][64] fp32 of
//   -LSE^1 log2 e, -LSE^2 log2 e, -D^1, -lam, lam D^2   (rows past N: zero)
// P^m = 2^(S^m c log2 e - LSE^m log2 e), dS^1 = P^1 (dP - D^1) and
// dS^2 = P^2 (-lam dP + lam D^2) take them as they are.
__host__ __device__ __forceinline__ size_t scal_offset(int bh, int N, int n) {
  return (((size_t)bh * ((N + 63) / 64) + n / 64) * 5) * 64 + n % 64;
}

// Untiled copy global -> shared (16-byte aligned, a multiple of 16 bytes),
// counted on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// [rows][W] tile of rows row.. of head bh, as [rows][64] blocks with 128-byte
// swizzle: one box where the tensor's rows are W wide, else one per block, with
// zeros past the row's end.  Either way the barrier counts rows x W elements.
template <int W, int ROWS>
__device__ __forceinline__ void load_rows(uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int row,
                                          int bh, bool narrow) {
  load_tile(dst, map, bar, row, bh);
  if (W == 128 && narrow) tma_load_4d(dst + ROWS * 128, map, bar, 64, row, 0, bh);
}

__device__ __forceinline__ void store_box(const CUtensorMap* map, const void* src, int x, int row, int r,
                                          int bh) {
  asm volatile(
      "cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(smem_u32(src)), "r"(x), "r"(row), "r"(r), "r"(bh)
      : "memory");
}
// The tile of load_rows back: rows past N, and elements past a row's end, are
// left as they are.  r: third coordinate of the map.  The caller
// fences its writes (fence_async_smem) and ends with stores_done.
template <int W, int ROWS>
__device__ __forceinline__ void store_rows(const CUtensorMap* map, const uint8_t* src, int row, int bh,
                                           bool narrow, int r = 0) {
  store_box(map, src, 0, row, r, bh);
  if (W == 128 && narrow) store_box(map, src + ROWS * 128, 64, row, r, bh);
}
// The stores of this thread have read their shared memory.
__device__ __forceinline__ void stores_done() {
  bulk_commit_group();
  bulk_wait_read_all();
}
// 8 packed words (16 features) of a row into the tile, from 16-byte chunk c on.
__device__ __forceinline__ void put16(uint32_t tile, int row, int c, const uint32_t (&v)[8]) {
  st_shared_v4(tile + sw128_offset(row, c), v[0], v[1], v[2], v[3]);
  st_shared_v4(tile + sw128_offset(row, c + 1), v[4], v[5], v[6], v[7]);
}

// 32 fp32 values, scaled, as 32 bf16 features of a row, from chunk c on.
__device__ __forceinline__ void put32(uint32_t tile, int row, int c, const uint32_t (&v)[32], float mul) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = pack_bf16(__uint_as_float(v[8 * q + 2 * e]) * mul,
                       __uint_as_float(v[8 * q + 2 * e + 1]) * mul);
    st_shared_v4(tile + sw128_offset(row, c + q), w[0], w[1], w[2], w[3]);
  }
}

// 32 fp32 values to 128 bytes of one row (16-byte aligned)
__device__ __forceinline__ void put32_global(float* dst, const uint32_t (&v)[32]) {
#pragma unroll
  for (int q = 0; q < 8; ++q)
    reinterpret_cast<uint4*>(dst)[q] = make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
}

// ===========================================================================
// Forward
// ===========================================================================
template <int D, int DV>
struct Fwd {
  static constexpr int BM = 128, BN = 128;
  static constexpr uint32_t QB = BM * D * 2;       // Q or K of one map
  static constexpr uint32_t VB = BN * DV * 2;
  // d = 64: stages of a whole key tile (K^1, K^2, V) on one barrier.  d = 128:
  // K and V do not fit three times; a ring of three K^m and one of two V
  static constexpr bool ONE = D == 64;
  static constexpr int KS = ONE ? 6 : 3, VS = ONE ? 3 : 2;
  static constexpr uint32_t OFF_Q = 0, OFF_K = 2 * QB, OFF_V = OFF_K + KS * QB;
  static constexpr uint32_t OFF_RED = OFF_V + VS * VB;  // [2][128] row sums
  static constexpr uint32_t OFF_MISC = OFF_RED + 2 * 128 * 4;
  static constexpr uint32_t SMEM = OFF_MISC + 512;
  static_assert(SMEM <= 232448, "forward shared memory budget");
  static_assert(4 * BM * DV * 2 <= OFF_RED - OFF_K, "o and rest are staged over the tiles");
  // TMEM columns: two score buffers (map m in buffer m; bf16 P overwrites the
  // first 16 of each thread's 32), O^1, O^2
  static constexpr uint32_t TMEM_COLS = 512;
  __host__ __device__ static constexpr uint32_t T_S(int m) { return 128u * m; }
  __host__ __device__ static constexpr uint32_t T_O(int m) { return 256u + (uint32_t)DV * m; }
  __host__ __device__ static constexpr uint32_t p_col(int k) { return 32u * (k >> 1) + 8u * (k & 1); }
  // The reference maximum (log2 domain) moves only when a tile's maximum
  // exceeds it by more than this, so O is rescaled in TMEM rarely
  static constexpr float kRescale = 8.f;
};

struct FwdParams : Common {
  bool rest;  // whether O^2 and what its and o's rounding left off are wanted (mR)
  float* lse;
};

template <int D, int DV, bool NARROW>
__global__ void __launch_bounds__(kFwdThreads, 1)
    diff_fwd_pass(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mK,
                  const __grid_constant__ CUtensorMap mV, const __grid_constant__ CUtensorMap mO,
                  const __grid_constant__ CUtensorMap mR, FwdParams prm) {
  using C = Fwd<D, DV>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  if (sb & 1023u) {  // 128-byte swizzled tiles need a 1024-byte aligned base
    if (threadIdx.x == 0) report_status(prm.status, FBOB_ERR_CUDA);
    return;
  }
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::OFF_MISC);
  // one barrier per tile stage (v_full, v_empty), or per K^m and per V stage
  uint64_t* v_full = q_full + 1;             // [VS]
  uint64_t* v_empty = v_full + C::VS;        // [VS]: a tile's last products done
  uint64_t* k_full = v_empty + C::VS;        // [KS] (d = 128)
  uint64_t* k_empty = k_full + C::KS;        // [KS] (d = 128)
  uint64_t* s_full = k_empty + C::KS;        // [2]: scores of map m in TMEM
  uint64_t* p_full = s_full + 2;             // [2][2]: half a tile's bf16 P written, O^m rescaled
  uint64_t* o_done = p_full + 4;
  uint64_t* drain = o_done + 1;
  static_assert((1 + 2 * C::VS + 2 * C::KS + 8) * 8 <= 256, "barriers end below the TMEM slot");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC + 256);
  Abort* ab = reinterpret_cast<Abort*>(smem + C::OFF_MISC + 264);
  float* red = reinterpret_cast<float*>(smem + C::OFF_RED);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int N = prm.N;
  const bool nd = NARROW && prm.narrow_d, nv = NARROW && prm.narrow_v;
  const int nblk = (N + C::BM - 1) / C::BM;
  const CtaCoord cc = cta_coord(prm.units, prm.group, nblk);
  const int bh = cc.bh;
  const int kvh = (bh / prm.H) * (prm.H / prm.G) + (bh % prm.H) / prm.G;
  const int blk = prm.causal ? nblk - 1 - cc.blk : cc.blk;  // long rows first
  const int i0 = blk * C::BM;
  const int T = ((prm.causal ? min(N, i0 + C::BM) : N) + C::BN - 1) / C::BN;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int s = 0; s < C::VS; ++s) {
      mbar_init(v_full + s, 1);
      mbar_init(v_empty + s, 1);
    }
    for (int s = 0; s < C::KS; ++s) {
      mbar_init(k_full + s, 1);
      mbar_init(k_empty + s, 1);
    }
    for (int m = 0; m < 2; ++m) {
      mbar_init(s_full + m, 1);
      mbar_init(p_full + 2 * m, 4);
      mbar_init(p_full + 2 * m + 1, 4);
    }
    mbar_init(o_done, 1);
    mbar_init(drain, 1);
    ab->flag = 0;
    ab->limit_ns = prm.wait_ns;
    fence_mbar_init();
  }
  if (warp == kFwdMma) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // K^m of tile t is subtile u = 2 t + m of its ring
  auto k_at = [&](int u) { return C::OFF_K + (uint32_t)(u % C::KS) * C::QB; };
  auto v_at = [&](int t) { return C::OFF_V + (uint32_t)(t % C::VS) * C::VB; };

  if (warp == kFwdProducer) {
    if (lane == 0) {
      mbar_arrive_expect_tx(q_full, 2 * C::QB);
      load_rows<D, C::BM>(smem + C::OFF_Q, &mQ, q_full, i0, 2 * bh, nd);
      load_rows<D, C::BM>(smem + C::OFF_Q + C::QB, &mQ, q_full, i0, 2 * bh + 1, nd);
      int k_issued = 0, v_issued = 0;
      for (int t = 0; t < T; ++t) {
        if (!C::ONE) {
          for (; k_issued < 2 * t + 2; ++k_issued) {
            const int u = k_issued, ks = u % C::KS;
            if (u >= C::KS && !stage_free(k_empty + ks, ((u / C::KS) - 1) & 1, ab, prm.status)) break;
            mbar_arrive_expect_tx(k_full + ks, C::QB);
            load_rows<D, C::BN>(smem + k_at(u), &mK, k_full + ks, t * C::BN, 2 * kvh + (u & 1), nd);
          }
          if (k_issued < 2 * t + 2) break;
        }
        const int vs = t % C::VS;
        if (t >= C::VS && !stage_free(v_empty + vs, ((t / C::VS) - 1) & 1, ab, prm.status)) break;
        mbar_arrive_expect_tx(v_full + vs, C::VB + (C::ONE ? 2 * C::QB : 0));
        if (C::ONE) {
          load_rows<D, C::BN>(smem + k_at(2 * t), &mK, v_full + vs, t * C::BN, 2 * kvh, nd);
          load_rows<D, C::BN>(smem + k_at(2 * t + 1), &mK, v_full + vs, t * C::BN, 2 * kvh + 1, nd);
        }
        load_rows<DV, C::BN>(smem + v_at(t), &mV, v_full + vs, t * C::BN, kvh, nv);
        ++v_issued;
      }
      // every load this thread issued has landed before the CTA exits (after an
      // abort some were never awaited); on the normal path these return at once
      mbar_wait_bounded(q_full, 0, prm.status, kDrainNs);
      for (int u = max(0, k_issued - C::KS); u < k_issued; ++u)
        mbar_wait_bounded(k_full + (u % C::KS), (u / C::KS) & 1, prm.status, kDrainNs);
      for (int t = max(0, v_issued - C::VS); t < v_issued; ++t)
        mbar_wait_bounded(v_full + (t % C::VS), (t / C::VS) & 1, prm.status, kDrainNs);
    }
  } else if (warp == kFwdMma) {
    constexpr uint32_t id_s = idesc_bf16(128, C::BN, false, false);  // S = Q K^T
    constexpr uint32_t id_o = idesc_bf16(128, DV, false, true);      // O += P V: B MN-major
    // A wait of this warp costs a few hundred cycles of a busy pipe and a commit
    // some tens.  So only what someone waits for is committed, and the loads of
    // a tile are awaited by a softmax warp, before its arrival for the tile
    // before (only the first tile's here).
    auto issue_s = [&](int t, int m) {
      const int u = 2 * t + m;
      const uint32_t q_lo = opaque(lo_kmajor(sb + C::OFF_Q + m * C::QB));
      const uint32_t k_lo = opaque(lo_kmajor(sb + k_at(u)));
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        mma_ss_w(tmem + C::T_S(m), q_lo + kslice_off(C::BM, k), k_lo + kslice_off(C::BN, k), id_s,
                 k > 0 ? 1u : 0u);
      mma_commit_w(s_full + m);
      if (!C::ONE) mma_commit_w(k_empty + u % C::KS);
    };
    await(q_full, 0, ab, prm.status);
    if (C::ONE) {
      await(v_full, 0, ab, prm.status);
    } else {
      await(k_full, 0, ab, prm.status);
      await(k_full + 1, 0, ab, prm.status);
    }
    tc_fence_after();
    issue_s(0, 0);
    issue_s(0, 1);
    for (int t = 0; t < T; ++t) {
      const bool more = t + 1 < T;
      const uint32_t v_mn = opaque(lo_mnmajor(sb + v_at(t), C::BN * 128));
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        // O^m += P^m V, A = bf16 P from TMEM, in two halves of 64 keys; then
        // the next tile's scores over P.  Their commit covers the product, so
        // whoever sees S^m of a tile may rescale O^m.
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          await(p_full + 2 * m + h, t & 1, ab, prm.status);
          tc_fence_after();
#pragma unroll
          for (int k = 4 * h; k < 4 * h + 4; ++k)
            mma_ts_w(tmem + C::T_O(m), tmem + C::T_S(m) + C::p_col(k), v_mn + kstep_off(k), id_o,
                     (t > 0 || k > 0) ? 1u : 0u);
        }
        if (m == 1) mma_commit_w(v_empty + t % C::VS);
        if (more) issue_s(t + 1, m);
      }
    }
    mma_commit_w(o_done);
    // every MMA this thread issued has completed before TMEM is released
    mma_commit_w(drain);
    mbar_wait_bounded(drain, 0, prm.status, kDrainNs);
  } else {
    // ---------------- softmax warps: thread = query row of one map ----------
    const int quad = warp & 3, m = warp >> 2;
    const int row = 32 * quad + lane;
    const int i = i0 + row;
    const float sc2 = prm.scale * kLog2e;
    const f2 sc2_2 = {sc2, sc2};
    const uint32_t lane_off = (uint32_t)(32 * quad) << 16;
    const uint32_t ts = tmem + lane_off + C::T_S(m);
    // the row's reference maximum (log2 domain) and sum of 2^(S c log2 e - max)
    float mx = -INFINITY, l = 0.f;
    for (int t = 0; t < T; ++t) {
      const int j0 = t * C::BN;
      // for the MMA warp: the next tile has landed
      if (C::ONE && warp == 0 && t + 1 < T)
        await(v_full + (t + 1) % C::VS, ((t + 1) / C::VS) & 1, ab, prm.status);
      await(s_full + m, t & 1, ab, prm.status);
      tc_fence_after();
      uint32_t s[4][32];
      tmem_ld32x4(ts, ts + 32, ts + 64, ts + 96, s[0], s[1], s[2], s[3]);
      // masked entries become -inf, so they give 2^-inf = 0 below
      if (j0 + C::BN > N || (prm.causal && j0 + C::BN - 1 > i0 + 32 * quad)) {
        const int end = prm.causal ? min(N, i + 1) : N;  // keys visible to this row
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (j0 + 32 * c + e >= end) s[c][e] = kMinusInf;
      }
      // the row's maximum over the tile (c log2 e > 0 keeps the order)
      float top[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        top[c] = __uint_as_float(s[c][0]);
#pragma unroll
        for (int e = 1; e < 31; e += 2)
          top[c] = max3(top[c], __uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1]));
        top[c] = fmaxf(top[c], __uint_as_float(s[c][31]));
      }
      const float mt = fmaxf(max3(top[0], top[1], top[2]), top[3]) * sc2;
      const bool move = mt > mx + C::kRescale;
      if (t == 0) {
        // key 0 is visible to every row, but infinite features can make every
        // score of the tile -inf, and -inf - -inf would reach the later tiles
        mx = fmaxf(mt, -FLT_MAX);
      } else if (__any_sync(0xffffffffu, move)) {
        // O^m holds the sums of the earlier tiles, whose products were committed
        // with these scores: rescale the row (rows that did not move by 1)
        const float alpha = move ? ex2_approx(mx - mt) : 1.f;
#pragma unroll 1
        for (int c = 0; c < DV; c += 16) {
          uint32_t v[16];
          const uint32_t ta = tmem + lane_off + C::T_O(m) + c;
          tmem_ld16(ta, v);
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
          tmem_st16(ta, v);
        }
        if (move) mx = mt;
        l *= alpha;
      }
      const f2 nm = {-mx, -mx};
      f2 acc = {0.f, 0.f};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t pw[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const f2 x = fma2({__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1])}, sc2_2, nm);
          const f2 p = {ex2_approx(x.x), ex2_approx(x.y)};
          acc = add2(acc, p);
          pw[e >> 1] = pack_bf16(p.x, p.y);
        }
        // bf16 P over the first 16 of the chunk's 32 columns; the product with
        // the first half starts while the second one is computed
        tmem_st16(ts + 32 * c, pw);
        if (c & 1) {
          // for the MMA warp, at d = 128: V of this tile and K^m of the next have
          // landed.  Behind the scores, no earlier: they tell that the slot's load
          // before this one has landed (its products were issued before them).
          // One phase short of the awaited one the parity reads as if that were
          // over, and the products would take keys that are still on their way.
          if (!C::ONE && quad == 0) {
            const int u = 2 * (t + 1) + m;
            if (c == 1 && m == 0) await(v_full + t % C::VS, (t / C::VS) & 1, ab, prm.status);
            if (c == 3 && t + 1 < T) await(k_full + u % C::KS, (u / C::KS) & 1, ab, prm.status);
          }
          tc_fence_before();
          warp_arrive(p_full + 2 * m + (c >> 1));
        }
      }
      l += acc.x + acc.y;
    }
    // ---- epilogue: O = O^1 / l^1 - lam O^2 / l^2, and LSE (natural log) ----
    red[m * 128 + row] = l;
    named_sync<kSoftmax>(1);
    const float L[2] = {red[row], red[128 + row]};
    await(o_done, 0, ab, prm.status);
    tc_fence_after();
    constexpr int PART = DV / 2;  // features per thread
    const int f0 = PART * m;
    const bool in = i < N;
    const float inv1 = 1.f / L[0], inv2 = 1.f / L[1];
    const float w = in ? lam_row(prm.lam, bh, prm.H, N, i) : 0.f;
    // through shared memory (the tiles' stages are free) into whole lines: from
    // the threads, each in a row of its own, the stores took 9000 cycles
    const uint32_t so = sb + C::OFF_K, sr = so + C::BM * DV * 2;  // o; rest's three parts
#pragma unroll
    for (int c = 0; c < PART; c += 16) {
      uint32_t a[16], b[16];
      tmem_ld16x2(tmem + lane_off + C::T_O(0) + f0 + c, tmem + lane_off + C::T_O(1) + f0 + c, a, b);
      auto left = [](uint32_t w, float x, float y) {  // what the rounding to w left off
        const float2 back = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
        return pack_bf16(x - back.x, y - back.y);
      };
      uint32_t wo[8], w2[8], l2[8], wl[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x2 = __uint_as_float(b[2 * e]) * inv2, y2 = __uint_as_float(b[2 * e + 1]) * inv2;
        const float x = fmaf(-w, x2, __uint_as_float(a[2 * e]) * inv1);
        const float y = fmaf(-w, y2, __uint_as_float(a[2 * e + 1]) * inv1);
        wo[e] = pack_bf16(x, y);
        w2[e] = pack_bf16(x2, y2);
        l2[e] = left(w2[e], x2, y2);
        wl[e] = left(wo[e], x, y);
      }
      const uint32_t blk = (uint32_t)((f0 + c) / 64) * C::BM * 128;  // 64-feature block
      const int chunk = (f0 + c) % 64 / 8;
      put16(so + blk, row, chunk, wo);
      if (prm.rest) {
        put16(sr + blk, row, chunk, w2);
        put16(sr + C::BM * DV * 2 + blk, row, chunk, l2);
        put16(sr + 2 * C::BM * DV * 2 + blk, row, chunk, wl);
      }
    }
    fence_async_smem();
    named_sync<kSoftmax>(1);
    if (threadIdx.x == 0) {
      store_rows<DV, C::BM>(&mO, smem + C::OFF_K, i0, bh, nv);
      if (prm.rest) {
        const uint8_t* src = smem + C::OFF_K + C::BM * DV * 2;
        for (int r = 0; r < 3; ++r)  // a wide row's 64-feature blocks follow one another
          store_rows<DV, C::BM>(&mR, src + r * C::BM * DV * 2, i0, bh, nv, nv ? r : r * (DV / 64));
      }
      stores_done();
    }
    if (in)
      prm.lse[((size_t)bh * 2 + m) * N + i] = (mx + log2f(m == 0 ? L[0] : L[1])) * kLn2;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kFwdMma) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// ===========================================================================
// Row scalars: D^2 = dO . O^2, D^1 = dO . O + lam D^2 (O = O^1 - lam O^2; both
// with what their rounding left off)
// ===========================================================================
// acc + the dot product of 8 bf16 pairs, in fp32
__device__ __forceinline__ float dot8(const uint4& a, const uint4& b, float acc) {
  const __nv_bfloat162* x = reinterpret_cast<const __nv_bfloat162*>(&a);
  const __nv_bfloat162* y = reinterpret_cast<const __nv_bfloat162*>(&b);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 u = __bfloat1622float2(x[e]), v = __bfloat1622float2(y[e]);
    acc = fmaf(u.x, v.x, fmaf(u.y, v.y, acc));
  }
  return acc;
}

// DV/8 lanes per row, 16 bytes of each tensor per lane (vecs = dv/8 of them); a
// block takes 64 rows of one head.  Bound: memory (O, rest and dO read once).
template <int DV>
__global__ void __launch_bounds__(256, 4)
    diff_tc_scalars(const uint4* __restrict__ o, const uint4* __restrict__ rest,
                    const uint4* __restrict__ dO, const float* __restrict__ lse, LamArg lam,
                    float* __restrict__ scal, int H, int N, int vecs) {
  constexpr int L = DV / 8, ROWS = 256 / L, STEPS = 64 / ROWS;
  __shared__ float dots[2][64];
  const int nb = (N + 63) / 64;
  const int bh = blockIdx.x / nb, n0 = (blockIdx.x % nb) * 64;
  const int sub = threadIdx.x / L, c = threadIdx.x % L;
  // thread e < 64 writes the scalars of row n0 + e: fetched ahead
  const int n = n0 + threadIdx.x;
  float l1 = 0.f, l2 = 0.f, w = 0.f;
  if (threadIdx.x < 64 && n < N) {
    l1 = lse[(size_t)bh * 2 * N + n];
    l2 = lse[((size_t)bh * 2 + 1) * N + n];
    w = lam_row(lam, bh, H, N, n);
  }
  float s1[STEPS], s2[STEPS];
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int r = i * ROWS + sub;
    s1[i] = s2[i] = 0.f;
    if (n0 + r < N && c < vecs) {
      const size_t row = (size_t)bh * N + n0 + r;
      const uint4 g = dO[row * vecs + c];
      s1[i] = dot8(o[row * vecs + c], g, dot8(rest[(3 * row + 2) * vecs + c], g, 0.f));
      s2[i] = dot8(rest[3 * row * vecs + c], g, dot8(rest[(3 * row + 1) * vecs + c], g, 0.f));
    }
  }
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
#pragma unroll
    for (int x = L / 2; x > 0; x >>= 1) {
      s1[i] += __shfl_xor_sync(0xffffffffu, s1[i], x);
      s2[i] += __shfl_xor_sync(0xffffffffu, s2[i], x);
    }
    if (c == 0) {
      dots[0][i * ROWS + sub] = s1[i];
      dots[1][i * ROWS + sub] = s2[i];
    }
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    float* dst = scal + scal_offset(bh, N, n0) + threadIdx.x;
    const float d1 = dots[0][threadIdx.x], d2 = dots[1][threadIdx.x];
    dst[0 * 64] = -l1 * kLog2e;
    dst[1 * 64] = -l2 * kLog2e;
    dst[2 * 64] = -fmaf(w, d2, d1);
    dst[3 * 64] = -w;
    dst[4 * 64] = w * d2;
  }
}

// ===========================================================================
// Row pass: dQ of both maps, and each row's sum_j P^2 dP
// ===========================================================================
template <int D, int DV>
struct Row {
  // d = 128: dQ^1 and dQ^2 take half of TMEM, so the key tiles are halved
  static constexpr int BM = 128, BN = D == 64 ? 128 : 64;
  static constexpr int NC = BN / kRowSlices;   // key columns per thread
  static constexpr int KS = 3, VS = 2;         // stages of K^1 and K^2, and of V
  static constexpr uint32_t QB = BM * D * 2, OB = BM * DV * 2;  // Q of one map, dO
  static constexpr uint32_t KB = BN * D * 2, VB = BN * DV * 2;  // K of one map, V
  static constexpr uint32_t OFF_Q = 0, OFF_DO = 2 * QB, OFF_K = OFF_DO + OB;
  static constexpr uint32_t OFF_V = OFF_K + KS * 2 * KB;
  static constexpr uint32_t OFF_RED = OFF_V + VS * VB;  // [slices][128]
  static constexpr uint32_t OFF_MISC = OFF_RED + kRowSlices * 128 * 4;
  static constexpr uint32_t SMEM = OFF_MISC + 512;
  static_assert(SMEM <= 232448, "row pass shared memory budget");
  static_assert(2 * QB <= KS * 2 * KB, "dQ is staged over the K ring");
  // TMEM columns: two score buffers (bf16 dS over the first half of each
  // thread's columns), dP, dQ^1, dQ^2
  static constexpr uint32_t TMEM_COLS = 512, T_DP = 2 * BN;
  __host__ __device__ static constexpr uint32_t T_S(int m) { return (uint32_t)BN * m; }
  __host__ __device__ static constexpr uint32_t T_DQ(int m) { return 3u * BN + (uint32_t)D * m; }
  __host__ __device__ static constexpr uint32_t a_col(int k) {
    return NC == 32 ? 32u * (k >> 1) + 8u * (k & 1) : 16u * k;
  }
  static_assert(3 * BN + 2 * D <= TMEM_COLS, "row pass TMEM budget");
};

struct RowParams : Common {
  const float* scal;  // row scalars (diff_tc_scalars)
  float* d2;          // [B, H, N]: sum_j P^2_ij dP_ij
};

template <int D, int DV, bool NARROW>
__global__ void __launch_bounds__(kThreads, 1)
    diff_row_pass(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mK,
                  const __grid_constant__ CUtensorMap mV, const __grid_constant__ CUtensorMap mDO,
                  const __grid_constant__ CUtensorMap mDQ, RowParams prm) {
  using C = Row<D, DV>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  if (sb & 1023u) {
    if (threadIdx.x == 0) report_status(prm.status, FBOB_ERR_CUDA);
    return;
  }
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::OFF_MISC);  // Q^1, Q^2, dO
  uint64_t* full = q_full + 1;             // [KS]: K^1, K^2 and V of a tile landed
  uint64_t* k_empty = full + C::KS;        // [KS]
  uint64_t* v_empty = k_empty + C::KS;     // [VS]
  uint64_t* s_full = v_empty + C::VS;      // [2]: scores of map m in TMEM, for map 0 dP too
  uint64_t* dp_read = s_full + 2;          // every thread holds its dP
  uint64_t* ds_full = dp_read + 1;         // [2]: bf16 dS written over the scores
  uint64_t* acc_done = ds_full + 2;
  uint64_t* drain = acc_done + 1;
  static_assert((1 + 2 * C::KS + C::VS + 7) * 8 <= 256, "barriers end below the TMEM slot");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC + 256);
  Abort* ab = reinterpret_cast<Abort*>(smem + C::OFF_MISC + 264);
  float* red = reinterpret_cast<float*>(smem + C::OFF_RED);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int N = prm.N;
  const bool nd = NARROW && prm.narrow_d, nv = NARROW && prm.narrow_v;
  const int nblk = (N + C::BM - 1) / C::BM;
  const CtaCoord cc = cta_coord(prm.units, prm.group, nblk);
  const int bh = cc.bh;
  const int kvh = (bh / prm.H) * (prm.H / prm.G) + (bh % prm.H) / prm.G;
  const int blk = prm.causal ? nblk - 1 - cc.blk : cc.blk;
  const int i0 = blk * C::BM;
  const int T = ((prm.causal ? min(N, i0 + C::BM) : N) + C::BN - 1) / C::BN;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int s = 0; s < C::KS; ++s) {
      mbar_init(full + s, 1);
      mbar_init(k_empty + s, 1);
    }
    for (int s = 0; s < C::VS; ++s) mbar_init(v_empty + s, 1);
    for (int m = 0; m < 2; ++m) {
      mbar_init(s_full + m, 1);
      mbar_init(ds_full + m, kWarps);
    }
    mbar_init(dp_read, kWarps);
    mbar_init(acc_done, 1);
    mbar_init(drain, 1);
    ab->flag = 0;
    ab->limit_ns = prm.wait_ns;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == kProducerWarp) {
    if (lane == 0) {
      mbar_arrive_expect_tx(q_full, 2 * C::QB + C::OB);
      load_rows<DV, C::BM>(smem + C::OFF_DO, &mDO, q_full, i0, bh, nv);
      load_rows<D, C::BM>(smem + C::OFF_Q, &mQ, q_full, i0, 2 * bh, nd);
      load_rows<D, C::BM>(smem + C::OFF_Q + C::QB, &mQ, q_full, i0, 2 * bh + 1, nd);
      int issued = 0;
      for (int t = 0; t < T; ++t) {
        const int ks = t % C::KS, vs = t % C::VS;
        if (t >= C::VS && !stage_free(v_empty + vs, ((t / C::VS) - 1) & 1, ab, prm.status)) break;
        if (t >= C::KS && !stage_free(k_empty + ks, ((t / C::KS) - 1) & 1, ab, prm.status)) break;
        uint8_t* dst = smem + C::OFF_K + ks * 2 * C::KB;
        mbar_arrive_expect_tx(full + ks, 2 * C::KB + C::VB);
        load_rows<DV, C::BN>(smem + C::OFF_V + vs * C::VB, &mV, full + ks, t * C::BN, kvh, nv);
        load_rows<D, C::BN>(dst, &mK, full + ks, t * C::BN, 2 * kvh, nd);
        load_rows<D, C::BN>(dst + C::KB, &mK, full + ks, t * C::BN, 2 * kvh + 1, nd);
        ++issued;
      }
      mbar_wait_bounded(q_full, 0, prm.status, kDrainNs);
      for (int t = max(0, issued - C::KS); t < issued; ++t)
        mbar_wait_bounded(full + (t % C::KS), (t / C::KS) & 1, prm.status, kDrainNs);
    }
  } else if (warp == kMmaWarp) {
    constexpr uint32_t id_s = idesc_bf16(128, C::BN, false, false);  // S and dP
    constexpr uint32_t id_q = idesc_bf16(128, D, false, true);       // dQ += dS K: B MN-major
    auto k_tile = [&](int t, int m) { return sb + C::OFF_K + (uint32_t)(2 * (t % C::KS) + m) * C::KB; };
    auto issue_s = [&](int t, int m) {
      const uint32_t q_lo = opaque(lo_kmajor(sb + C::OFF_Q + m * C::QB));
      const uint32_t k_lo = opaque(lo_kmajor(k_tile(t, m)));
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        mma_ss_w(tmem + C::T_S(m), q_lo + kslice_off(C::BM, k), k_lo + kslice_off(C::BN, k), id_s,
                 k > 0 ? 1u : 0u);
    };
    auto issue_dp = [&](int t) {
      const uint32_t do_lo = opaque(lo_kmajor(sb + C::OFF_DO));
      const uint32_t v_lo = opaque(lo_kmajor(sb + C::OFF_V + (t % C::VS) * C::VB));
#pragma unroll
      for (int k = 0; k < DV / 16; ++k)
        mma_ss_w(tmem + C::T_DP, do_lo + kslice_off(C::BM, k), v_lo + kslice_off(C::BN, k), id_s,
                 k > 0 ? 1u : 0u);
      mma_commit_w(v_empty + t % C::VS);
    };
    // dQ^m += dS^m K^m
    auto issue_dq = [&](int t, int m) {
      const uint32_t k_mn = opaque(lo_mnmajor(k_tile(t, m), C::BN * 128));
#pragma unroll
      for (int k = 0; k < C::BN / 16; ++k)
        mma_ts_w(tmem + C::T_DQ(m), tmem + C::T_S(m) + C::a_col(k), k_mn + kstep_off(k), id_q,
                 (t > 0 || k > 0) ? 1u : 0u);
    };
    // (the loads of later tiles are awaited by an elementwise warp)
    await(q_full, 0, ab, prm.status);
    await(full, 0, ab, prm.status);
    tc_fence_after();
    issue_dp(0);
    issue_s(0, 0);
    mma_commit_w(s_full);  // covers dP, issued before
    for (int t = 0; t < T; ++t) {
      const bool more = t + 1 < T;
      // scores go over the dS of the tile before, whose dQ product is issued;
      // the next dP over this one, as soon as every thread has read it
      issue_s(t, 1);
      mma_commit_w(s_full + 1);
      if (more) {
        await(dp_read, t & 1, ab, prm.status);
        tc_fence_after();
        issue_dp(t + 1);
      }
      await(ds_full, t & 1, ab, prm.status);
      tc_fence_after();
      issue_dq(t, 0);
      if (more) {
        issue_s(t + 1, 0);
        mma_commit_w(s_full);
      }
      await(ds_full + 1, t & 1, ab, prm.status);
      tc_fence_after();
      issue_dq(t, 1);
      mma_commit_w(k_empty + t % C::KS);
    }
    mma_commit_w(acc_done);
    mma_commit_w(drain);
    mbar_wait_bounded(drain, 0, prm.status, kDrainNs);
  } else {
    // ---------------- elementwise warps: thread = query row ----------------
    constexpr int NC = C::NC;
    const int quad = warp & 3, slice = warp >> 2;
    const int row = 32 * quad + lane;
    const int i = i0 + row;
    const bool in = i < N;
    const uint32_t lane_off = (uint32_t)(32 * quad) << 16;
    const float sc2 = prm.scale * kLog2e;
    const f2 sc2_2 = {sc2, sc2};
    // dS^1 = P^1 (dP - D^1), dS^2 = P^2 (-lam dP + lam D^2): a factor and a
    // summand per map; rows past the end have Q = dO = 0 and stay zero
    const float* sc = prm.scal + scal_offset(bh, N, in ? i : 0);
    const float nl[2] = {in ? sc[0] : 0.f, in ? sc[64] : 0.f};
    const float mul[2] = {1.f, in ? sc[3 * 64] : 0.f};
    const float add[2] = {in ? sc[2 * 64] : 0.f, in ? sc[4 * 64] : 0.f};
    f2 d2 = {0.f, 0.f};
    for (int t = 0; t < T; ++t) {
      const int j0 = t * C::BN + NC * slice;
      const bool need_mask = (j0 + NC > N) || (prm.causal && j0 + NC - 1 > i0 + 32 * quad);
      // for the MMA warp: the next tile has landed
      if (warp == 0 && t + 1 < T) await(full + (t + 1) % C::KS, ((t + 1) / C::KS) & 1, ab, prm.status);
      uint32_t dp[NC];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        await(s_full + m, t & 1, ab, prm.status);
        tc_fence_after();
        const uint32_t ts = tmem + lane_off + C::T_S(m) + NC * slice;
        uint32_t sr[NC];
        if (m == 0) {
          const uint32_t tp = tmem + lane_off + C::T_DP + NC * slice;
          if constexpr (NC == 32) tmem_ld32x2(ts, tp, sr, dp);
          else tmem_ld16x2(ts, tp, sr, dp);
          tc_fence_before();
          warp_arrive(dp_read);
        } else {
          if constexpr (NC == 32) tmem_ld32(ts, sr);
          else tmem_ld16(ts, sr);
        }
        const f2 nl2 = {nl[m], nl[m]}, mul2_ = {mul[m], mul[m]}, add2_ = {add[m], add[m]};
        uint32_t dsw[NC / 2];
        auto body = [&](auto masked) {
#pragma unroll
          for (int c = 0; c < NC; c += 2) {
            const f2 x = fma2({__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])}, sc2_2, nl2);
            f2 p = {ex2_approx(x.x), ex2_approx(x.y)};
            if (decltype(masked)::value) {
              const int j = j0 + c;
              p.x = (j < N && (!prm.causal || j <= i)) ? p.x : 0.f;
              p.y = (j + 1 < N && (!prm.causal || j + 1 <= i)) ? p.y : 0.f;
            }
            const f2 g = {__uint_as_float(dp[c]), __uint_as_float(dp[c + 1])};
            if (m == 1) d2 = fma2(p, g, d2);
            const f2 ds = mul2(p, fma2(g, mul2_, add2_));
            dsw[c >> 1] = pack_bf16(ds.x, ds.y);
          }
        };
        if (need_mask) body(std::true_type{});
        else body(std::false_type{});
        if constexpr (NC == 32) tmem_st16(ts, dsw);
        else tmem_st8(ts, dsw);
        tc_fence_before();
        warp_arrive(ds_full + m);
      }
    }
    // ---- epilogue: dQ (scaled): half the features of one map per thread ----
    red[slice * 128 + row] = d2.x + d2.y;
    await(acc_done, 0, ab, prm.status);
    tc_fence_after();
    const int m = slice >> 1;
#pragma unroll
    for (int x = 0; x < D / 64; ++x) {
      const int f = D / 2 * (slice & 1) + 32 * x;
      uint32_t v[32];
      tmem_ld32(tmem + lane_off + C::T_DQ(0) + D * m + f, v);
      put32(sb + C::OFF_K + m * C::QB + f / 64 * C::BM * 128, row, f % 64 / 8, v, prm.scale);
    }
    fence_async_smem();
    named_sync<kConsumers>(1);
    if (threadIdx.x == 0) {
      store_rows<D, C::BM>(&mDQ, smem + C::OFF_K, i0, 2 * bh, nd);
      store_rows<D, C::BM>(&mDQ, smem + C::OFF_K + C::QB, i0, 2 * bh + 1, nd);
      stores_done();
    }
    if (slice == 0 && in) {
      float s = 0.f;
#pragma unroll
      for (int u = 0; u < kRowSlices; ++u) s += red[u * 128 + row];
      prm.d2[(size_t)bh * N + i] = s;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// ===========================================================================
// Column pass: dK of both maps and dV
// ===========================================================================
template <int D, int DV>
struct Col {
  static constexpr int BM = 128, BN = 64;
  static constexpr int ST = D == 64 ? 4 : 2;      // query tile stages: Q^1, Q^2, dO
  static constexpr uint32_t KB = BM * D * 2;     // stationary K of one map
  static constexpr uint32_t VB = BM * DV * 2;
  static constexpr uint32_t QB = BN * D * 2;     // streamed Q of one map
  static constexpr uint32_t OB = BN * DV * 2;     // streamed dO
  static constexpr uint32_t STB = 2 * QB + OB;
  static constexpr uint32_t OFF_K = 0, OFF_V = 2 * KB, OFF_T = OFF_V + VB;
  static constexpr uint32_t SCB = 5 * BN * 4;     // its row scalars (diff_tc_scalars)
  static constexpr uint32_t OFF_SC = OFF_T + ST * STB;
  static constexpr uint32_t OFF_MISC = OFF_SC + ST * SCB;
  static constexpr uint32_t SMEM = OFF_MISC + 512;
  static_assert(SMEM <= 232448, "column pass shared memory budget");
  static_assert(2 * KB + VB <= ST * STB, "dK and dV are staged over the tiles");
  // TMEM columns.  d = 64: S^T of map 1, two buffers for that of map 2, dP^T,
  // dK^1, dK^2, dV.  Each thread's 16 columns then hold bf16 dS^T in the last 8
  // and, for map 2, W^T in the first 8.  With the second buffer a tile's three
  // score blocks are all computed while the elementwise warps are on map 2 of
  // the tile before.  d = 128: the accumulators leave two blocks: S^T of map 1,
  // and dP^T, over which S^T of map 2 goes once dP^T has been read.
  static constexpr bool WIDE = D == 128;
  static constexpr uint32_t TMEM_COLS = 512, T_S1 = 0, T_DP = WIDE ? 64 : 192, T_DV = 384;
  static constexpr int S2 = WIDE ? 1 : 2;  // buffers of S^T of map 2
  // that of tile a, and the parity of the phase of its barriers
  __host__ __device__ static constexpr int buf(int a) { return a & (S2 - 1); }
  __host__ __device__ static constexpr uint32_t phase(int a) { return (uint32_t)(a >> (S2 - 1)) & 1u; }
  __host__ __device__ static constexpr uint32_t T_S2(int b) { return 64u + 64u * b; }
  __host__ __device__ static constexpr uint32_t T_DK(int m) {
    return (WIDE ? 128u : 256u) + (uint32_t)D * m;
  }
};

struct ColParams : Common {
  const float* scal;  // row scalars (diff_tc_scalars)
  float* parts;       // [gridDim.y][B Hk][N][2 D + DV]: partial dK^1, dK^2, dV
};

// PARTS: gridDim.y CTAs share a key block (the branches of one kernel for both
// cost the whole blocks 1%)
template <int D, int DV, bool NARROW, bool PARTS>
__global__ void __launch_bounds__(kThreads, 1)
    diff_col_pass(const __grid_constant__ CUtensorMap mK, const __grid_constant__ CUtensorMap mV,
                  const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mDO,
                  const __grid_constant__ CUtensorMap mDK, const __grid_constant__ CUtensorMap mDV,
                  ColParams prm) {
  using C = Col<D, DV>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  if (sb & 1023u) {
    if (threadIdx.x == 0) report_status(prm.status, FBOB_ERR_CUDA);
    return;
  }
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(smem + C::OFF_MISC);
  uint64_t* full = kv_full + 1;            // [ST]: Q^1, Q^2, dO landed, scalars written
  uint64_t* empty = full + C::ST;          // [ST]: the tile's last products done
  // S^T of map 2 is a tile ahead of the warps where it has two TMEM buffers
  // (!WIDE).  Each then has a barrier of its own, for the scores and for the
  // operands over them, so that none runs two phases ahead of a waiter and no
  // warp's arrival for the next tile counts for this one: a buffer's next scores
  // are committed behind the wait for its operands.
  uint64_t* s_full = empty + C::ST;        // S^T of map 1 and dP^T in TMEM
  uint64_t* s2_full = s_full + 1;          // [S2]: S^T of map 2
  uint64_t* dp_read = s2_full + C::S2;     // every thread holds its dP
  uint64_t* ds_full = dp_read + 1;         // bf16 dS^T of map 1 written over the scores
  uint64_t* ds2_full = ds_full + 1;        // [S2]: bf16 operands of map 2
  uint64_t* acc_done = ds2_full + C::S2;
  uint64_t* drain = acc_done + 1;
  static_assert((1 + 2 * C::ST + 5 + 2 * C::S2) * 8 <= 256, "barriers end below the TMEM slot");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC + 256);
  Abort* ab = reinterpret_cast<Abort*>(smem + C::OFF_MISC + 264);
  float* scal = reinterpret_cast<float*>(smem + C::OFF_SC);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int N = prm.N;
  const bool nd = NARROW && prm.narrow_d, nv = NARROW && prm.narrow_v;
  const CtaCoord cc = cta_coord(prm.units, prm.group, (N + C::BM - 1) / C::BM);
  const int kvh = cc.bh, Hk = prm.H / prm.G;
  const int bh0 = (kvh / Hk) * prm.H + (kvh % Hk) * prm.G;  // first query head
  const int j0 = cc.blk * C::BM;
  const int qstart = prm.causal ? j0 : 0;  // j0 is a multiple of BN
  const int Tq = (N - qstart + C::BN - 1) / C::BN;
  // query tiles of all the query heads; this CTA's: a0 .. a0 + T - 1
  const int all = Tq * prm.G, part = blockIdx.y, split = gridDim.y;
  const int a0 = PARTS ? (int)((long long)all * part / split) : 0;
  const int T = PARTS ? (int)((long long)all * (part + 1) / split) - a0 : all;
  float* part_rows = prm.parts + ((size_t)part * prm.units + kvh) * N * (2 * D + DV);
  if (PARTS && T == 0) {  // the mask leaves this part nothing
    const int rows = min(C::BM, N - j0);
    for (int e = threadIdx.x; e < rows * (2 * D + DV); e += kThreads)
      part_rows[(size_t)j0 * (2 * D + DV) + e] = 0.f;
    return;
  }

  if (threadIdx.x == 0) {
    mbar_init(kv_full, 1);
    for (int s = 0; s < C::ST; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    mbar_init(s_full, 1);
    mbar_init(ds_full, kWarps);
    for (int s = 0; s < C::S2; ++s) {
      mbar_init(s2_full + s, 1);
      mbar_init(ds2_full + s, kWarps);
    }
    mbar_init(dp_read, kWarps);
    mbar_init(acc_done, 1);
    mbar_init(drain, 1);
    ab->flag = 0;
    ab->limit_ns = prm.wait_ns;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == kProducerWarp) {
    if (lane == 0) {
      mbar_arrive_expect_tx(kv_full, 2 * C::KB + C::VB);
      load_rows<DV, C::BM>(smem + C::OFF_V, &mV, kv_full, j0, kvh, nv);
      load_rows<D, C::BM>(smem + C::OFF_K, &mK, kv_full, j0, 2 * kvh, nd);
      load_rows<D, C::BM>(smem + C::OFF_K + C::KB, &mK, kv_full, j0, 2 * kvh + 1, nd);
    }
    if (lane == 0) {
      int g = PARTS ? a0 / Tq : 0, t = PARTS ? a0 % Tq : 0, issued = 0;  // tile t within head g
      for (int a = 0; a < T; ++a) {
        const int st = a % C::ST, q0 = qstart + t * C::BN, bh = bh0 + g;
        if (a >= C::ST && !stage_free(empty + st, ((a / C::ST) - 1) & 1, ab, prm.status)) break;
        uint8_t* dst = smem + C::OFF_T + st * C::STB;
        mbar_arrive_expect_tx(full + st, C::STB + C::SCB);
        load_rows<D, C::BN>(dst, &mQ, full + st, q0, 2 * bh, nd);
        load_rows<D, C::BN>(dst + C::QB, &mQ, full + st, q0, 2 * bh + 1, nd);
        load_rows<DV, C::BN>(dst + 2 * C::QB, &mDO, full + st, q0, bh, nv);
        bulk_load(smem + C::OFF_SC + st * C::SCB, prm.scal + scal_offset(bh, N, q0), C::SCB, full + st);
        ++issued;
        if (++t == Tq) {
          t = 0;
          ++g;
        }
      }
      mbar_wait_bounded(kv_full, 0, prm.status, kDrainNs);
      for (int a = max(0, issued - C::ST); a < issued; ++a)
        mbar_wait_bounded(full + (a % C::ST), (a / C::ST) & 1, prm.status, kDrainNs);
    }
  } else if (warp == kMmaWarp) {
    constexpr uint32_t id_s = idesc_bf16(128, C::BN, false, false);  // S^T and dP^T
    constexpr uint32_t id_k = idesc_bf16(128, D, false, true);       // dK += dS^T Q
    constexpr uint32_t id_v = idesc_bf16(128, DV, false, true);      // dV += W^T dO
    auto tile = [&](int a) { return sb + C::OFF_T + (uint32_t)(a % C::ST) * C::STB; };
    auto s_cols = [&](int a, int m) { return tmem + (m == 0 ? C::T_S1 : C::T_S2(C::buf(a))); };
    auto issue_s = [&](int a, int m) {
      const uint32_t k_lo = opaque(lo_kmajor(sb + C::OFF_K + m * C::KB));
      const uint32_t q_lo = opaque(lo_kmajor(tile(a) + m * C::QB));
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        mma_ss_w(s_cols(a, m), k_lo + kslice_off(C::BM, k), q_lo + kslice_off(C::BN, k), id_s,
                 k > 0 ? 1u : 0u);
    };
    auto issue_dp = [&](int a) {
      const uint32_t v_lo = opaque(lo_kmajor(sb + C::OFF_V));
      const uint32_t do_lo = opaque(lo_kmajor(tile(a) + 2 * C::QB));
#pragma unroll
      for (int k = 0; k < DV / 16; ++k)
        mma_ss_w(tmem + C::T_DP, v_lo + kslice_off(C::BM, k), do_lo + kslice_off(C::BN, k), id_s,
                 k > 0 ? 1u : 0u);
    };
    // S^T of both maps (the first commit covers dP^T, issued before)
    auto issue_scores = [&](int a) {
      issue_s(a, 0);
      mma_commit_w(s_full);
      issue_s(a, 1);
      mma_commit_w(s2_full + C::buf(a));
    };
    // dK^m += dS^m^T Q^m
    auto issue_dk = [&](int a, int m) {
      const uint32_t t_a = s_cols(a, m);
      const uint32_t q_mn = opaque(lo_mnmajor(tile(a) + m * C::QB, C::BN * 128));
#pragma unroll
      for (int k = 0; k < C::BN / 16; ++k)
        mma_ts_w(tmem + C::T_DK(m), t_a + 16 * k + 8, q_mn + kstep_off(k), id_k, (a > 0 || k > 0) ? 1u : 0u);
    };
    // dV += W^T dO
    auto issue_dv = [&](int a) {
      const uint32_t do_mn = opaque(lo_mnmajor(tile(a) + 2 * C::QB, C::BN * 128));
#pragma unroll
      for (int k = 0; k < C::BN / 16; ++k)
        mma_ts_w(tmem + C::T_DV, s_cols(a, 1) + 16 * k, do_mn + kstep_off(k), id_v,
                 (a > 0 || k > 0) ? 1u : 0u);
    };
    await(kv_full, 0, ab, prm.status);
    await(full, 0, ab, prm.status);
    tc_fence_after();
    if (C::WIDE) {
      issue_s(0, 0);
      issue_dp(0);
      mma_commit_w(s_full);
      for (int a = 0; a < T; ++a) {
        const bool more = a + 1 < T;
        // S^T of map 2 over dP^T, once every thread has read it
        await(dp_read, a & 1, ab, prm.status);
        tc_fence_after();
        issue_s(a, 1);
        mma_commit_w(s2_full + C::buf(a));
        // dK^1, then the next tile's S^T of map 1 over the dS^T it read
        if (more) await(full + (a + 1) % C::ST, ((a + 1) / C::ST) & 1, ab, prm.status);
        await(ds_full, a & 1, ab, prm.status);
        tc_fence_after();
        issue_dk(a, 0);
        if (more) issue_s(a + 1, 0);
        // dK^2 and dV, then the next dP^T over their operands
        await(ds2_full + C::buf(a), C::phase(a), ab, prm.status);
        tc_fence_after();
        issue_dk(a, 1);
        issue_dv(a);
        mma_commit_w(empty + a % C::ST);
        if (more) {
          issue_dp(a + 1);
          mma_commit_w(s_full);
        }
      }
    }
    if (!C::WIDE) {  // (the loads of later tiles are awaited by the elementwise warps)
      issue_dp(0);
      issue_scores(0);
    }
    for (int a = 0; !C::WIDE && a < T; ++a) {
      const bool more = a + 1 < T;
      // the next dP^T over this one, as soon as every thread has read it
      if (more) {
        await(dp_read, a & 1, ab, prm.status);
        tc_fence_after();
        issue_dp(a + 1);
      }
      await(ds_full, a & 1, ab, prm.status);
      tc_fence_after();
      // dK^1, then the next tile's scores: S^T of map 1 over the dS^T that
      // product read, that of map 2 over the operands of tile a - 1
      issue_dk(a, 0);
      if (more) issue_scores(a + 1);
      await(ds2_full + C::buf(a), C::phase(a), ab, prm.status);
      tc_fence_after();
      issue_dk(a, 1);
      issue_dv(a);
      mma_commit_w(empty + a % C::ST);
    }
    mma_commit_w(acc_done);
    mma_commit_w(drain);
    mbar_wait_bounded(drain, 0, prm.status, kDrainNs);
  } else {
    // ---------------- elementwise warps: thread = key row ------------------
    constexpr int NC = C::BN / kRowSlices;  // query columns per thread: 16
    const int quad = warp & 3, slice = warp >> 2;
    const int row = 32 * quad + lane;
    const int j = j0 + row;
    const uint32_t lane_off = (uint32_t)(32 * quad) << 16;
    const float sc2 = prm.scale * kLog2e;
    const f2 sc2_2 = {sc2, sc2};
    int t = PARTS ? a0 % Tq : 0;
    for (int a = 0; a < T; ++a) {
      const int st = a % C::ST;
      const int qa = qstart + t * C::BN + NC * slice;
      if (++t == Tq) t = 0;
      const bool need_mask = (qa + NC > N) || (prm.causal && qa < j0 + 32 * quad + 31);
      const float4* sc4 = reinterpret_cast<const float4*>(scal + st * 5 * C::BN + NC * slice);
      // this tile's scalars (already there), and for the MMA warp the next tile
      if (a == 0 || C::WIDE) await(full + st, (a / C::ST) & 1, ab, prm.status);
      if (!C::WIDE && a + 1 < T)
        await(full + (a + 1) % C::ST, ((a + 1) / C::ST) & 1, ab, prm.status);
      uint32_t dp[NC];
      float p1[NC];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        if (m == 0) await(s_full, a & 1, ab, prm.status);
        else await(s2_full + C::buf(a), C::phase(a), ab, prm.status);
        tc_fence_after();
        const uint32_t ts = tmem + lane_off + (m == 0 ? C::T_S1 : C::T_S2(C::buf(a))) + NC * slice;
        uint32_t sr[NC];
        if (m == 0) {
          tmem_ld16x2(ts, tmem + lane_off + C::T_DP + NC * slice, sr, dp);
          tc_fence_before();
          warp_arrive(dp_read);
        } else {
          tmem_ld16(ts, sr);
        }
        uint32_t dsw[NC / 2], ww[NC / 2];
        auto body = [&](auto masked) {
#pragma unroll
          for (int c4 = 0; c4 < NC / 4; ++c4) {  // 4 query columns per step
            const float4 L = sc4[m * (C::BN / 4) + c4];
            const float4 A = sc4[(m == 0 ? 2 : 4) * (C::BN / 4) + c4];  // -D^1, or lam D^2
            const float4 W = m == 0 ? make_float4(1.f, 1.f, 1.f, 1.f) : sc4[3 * (C::BN / 4) + c4];
            const f2 nl[2] = {{L.x, L.y}, {L.z, L.w}}, ad[2] = {{A.x, A.y}, {A.z, A.w}};
            const f2 nw[2] = {{W.x, W.y}, {W.z, W.w}};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int c = 4 * c4 + 2 * h;
              const f2 x = fma2({__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])}, sc2_2, nl[h]);
              f2 p = {ex2_approx(x.x), ex2_approx(x.y)};
              if (decltype(masked)::value) {
                const int q = qa + c;
                p.x = (q < N && (!prm.causal || q >= j)) ? p.x : 0.f;
                p.y = (q + 1 < N && (!prm.causal || q + 1 >= j)) ? p.y : 0.f;
              }
              const f2 gdp = {__uint_as_float(dp[c]), __uint_as_float(dp[c + 1])};
              f2 ds;
              if (m == 0) {
                p1[c] = p.x;
                p1[c + 1] = p.y;
                ds = mul2(p, add2(gdp, ad[h]));
              } else {
                const f2 wt = fma2(p, nw[h], {p1[c], p1[c + 1]});  // W = P^1 - lam P^2
                ww[c >> 1] = pack_bf16(wt.x, wt.y);
                ds = mul2(p, fma2(gdp, nw[h], ad[h]));
              }
              dsw[c >> 1] = pack_bf16(ds.x, ds.y);
            }
          }
        };
        if (need_mask) body(std::true_type{});
        else body(std::false_type{});
        if (m == 0) tmem_st8(ts + 8, dsw);
        else tmem_st8x2(ts, ww, ts + 8, dsw);
        tc_fence_before();
        warp_arrive(m == 0 ? ds_full : ds2_full + C::buf(a));
      }
    }
    // ---- epilogue: dK (scaled), half the features of one map per thread, and dV ----
    await(acc_done, 0, ab, prm.status);
    tc_fence_after();
    const int m = slice >> 1;
    uint32_t v[32];
    // a part's sums go out in fp32, for diff_col_join
    float* mine = part_rows + (size_t)j * (2 * D + DV);
#pragma unroll
    for (int x = 0; x < D / 64; ++x) {
      const int f = D / 2 * (slice & 1) + 32 * x;
      tmem_ld32(tmem + lane_off + C::T_DK(0) + D * m + f, v);
      if (!PARTS)
        put32(sb + C::OFF_T + m * C::KB + f / 64 * C::BM * 128, row, f % 64 / 8, v, prm.scale);
      else if (j < N)
        put32_global(mine + D * m + f, v);
    }
    if (DV == 128 || slice < 2) {
      tmem_ld32(tmem + lane_off + C::T_DV + 32 * slice, v);
      if (!PARTS)
        put32(sb + C::OFF_T + 2 * C::KB + m * C::BM * 128, row, 32 * (slice & 1) / 8, v, 1.f);
      else if (j < N)
        put32_global(mine + 2 * D + 32 * slice, v);
    }
    fence_async_smem();
    named_sync<kConsumers>(1);
    if (!PARTS && threadIdx.x == 0) {
      store_rows<D, C::BM>(&mDK, smem + C::OFF_T, j0, 2 * kvh, nd);
      store_rows<D, C::BM>(&mDK, smem + C::OFF_T + C::KB, j0, 2 * kvh + 1, nd);
      store_rows<DV, C::BM>(&mDV, smem + C::OFF_T + 2 * C::KB, j0, kvh, nv);
      stores_done();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// dK (scaled) and dV from the column pass's parts, added in their order: a
// thread per 4 features of a key row.
template <int D, int DV>
__global__ void __launch_bounds__(256)
    diff_col_join(const float4* __restrict__ parts, uint2* __restrict__ dk, uint2* __restrict__ dv,
                  int split, int N, size_t rows, int d, int dv_, float scale) {
  constexpr int W = (2 * D + DV) / 4;
  const size_t e = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= rows * W) return;
  float4 x = parts[e];
  for (int s = 1; s < split; ++s) {
    const float4 y = parts[(size_t)s * rows * W + e];
    x.x += y.x;
    x.y += y.y;
    x.z += y.z;
    x.w += y.w;
  }
  const size_t row = e / W, kvh = row / N, j = row - kvh * N;
  const int f = (int)(e - row * W);
  if (f < 2 * D / 4) {
    const int m = f / (D / 4), c = f % (D / 4);
    if (4 * c < d)
      dk[((2 * kvh + m) * N + j) * (d / 4) + c] =
          make_uint2(pack_bf16(x.x * scale, x.y * scale), pack_bf16(x.z * scale, x.w * scale));
  } else {
    const int c = f - 2 * D / 4;
    if (4 * c < dv_) dv[row * (dv_ / 4) + c] = make_uint2(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w));
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// Parts of the column pass: with few key heads or keys its blocks leave SMs
// idle, while each walks over the queries of every head of its group.  So it is
// cut into as many parts as the SMs take, of 8 or more 64-query tiles each, and
// their sums are joined.  dK and dV at d = 64, dv = 128, causal, in one part and
// cut: 2 key heads of 16 heads, 2048 tokens 276 -> 82 + 4 us; 1 of 8, 512 tokens
// 77 -> 24 + 4; 2 of 2, 2048 tokens 43 -> 24 + 4; but with 16 tiles to cut (8 of
// 8 heads, 1024 tokens) 26 -> 25 + 4, so fewer than 24 stay whole.
int col_parts(const DiffProblem& p) {
  constexpr long long kTiles = 8;
  const long long blocks = (long long)((p.N + 127) / 128) * p.B * p.Hk;
  const long long tiles = (long long)((p.N + 63) / 64) * p.G();
  return tiles < 3 * kTiles ? 1 : (int)max(1ll, min((long long)kSms / blocks, tiles / kTiles));
}

// The kernels' width for rows of `width`
int built(int width) { return width <= 64 ? 64 : 128; }

Common common(const DiffProblem& p, const DiffTensors& t, const DiffWorkspace& ws, int units) {
  Common c{};
  c.status = ws.status;
  c.wait_ns = wait_limit_ns();
  c.N = p.N;
  c.causal = p.causal;
  c.H = p.H;
  c.G = p.G();
  c.units = units;
  c.group = cta_group_heads(units, (p.N + 127) / 128, kSms);
  c.scale = p.scale;
  c.narrow_d = p.d != built(p.d);
  c.narrow_v = p.dv != built(p.dv);
  c.lam = t.lam;
  return c;
}

// [B, heads, N, parts, width] as boxes of `rows` rows of one part: all 64-feature
// blocks where a row is as wide as the kernel (then the third coordinate counts
// blocks), else one block (it counts parts)
bool tiles(CUtensorMap* m, const void* ptr, const DiffProblem& p, int heads, int width, int rows,
           int parts = 1) {
  const bool wide = width == built(width);
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t blocks = wide ? width / 64 : 1, w = width / blocks, n = p.N, r = parts * blocks;
  const cuuint64_t dims[4] = {w, n, r, (cuuint64_t)p.B * heads};
  const cuuint64_t strides[3] = {r * w * 2, w * 2, n * r * w * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)rows, (cuuint32_t)blocks, 1}, es[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename K, typename P, typename... M>
cudaError_t run(K kernel, int units, int parts, int N, int threads, uint32_t smem, LaunchLog& log,
                const P& prm, const M&... maps) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kernel<<<dim3(((N + 127) / 128) * units, parts), threads, smem, log.stream>>>(maps..., prm);
  e = cudaGetLastError();
  log.mark();
  return e;
}

template <int D, int DV>
cudaError_t forward_d(const DiffProblem& p, const DiffTensors& t, const DiffWorkspace& ws,
                      LaunchLog& log) {
  CUtensorMap mQ, mK, mV, mO, mR;  // without rest mR is a placeholder
  if (!tiles(&mQ, t.q, p, 2 * p.H, p.d, 128) || !tiles(&mK, t.k, p, 2 * p.Hk, p.d, 128) ||
      !tiles(&mV, t.v, p, p.Hk, p.dv, 128) || !tiles(&mO, t.o, p, p.H, p.dv, 128) ||
      !tiles(&mR, t.rest ? t.rest : t.o, p, p.H, p.dv, 128, t.rest ? 3 : 1))
    return cudaErrorInvalidValue;
  FwdParams f;
  static_cast<Common&>(f) = common(p, t, ws, p.B * p.H);
  f.rest = t.rest != nullptr;
  f.lse = t.lse;
  const auto kernel = f.narrow_d || f.narrow_v ? diff_fwd_pass<D, DV, true> : diff_fwd_pass<D, DV, false>;
  return run(kernel, f.units, 1, p.N, kFwdThreads, Fwd<D, DV>::SMEM, log, f, mQ, mK, mV, mO, mR);
}

template <int D, int DV>
cudaError_t backward_d(const DiffProblem& p, const DiffTensors& t, const DiffWorkspace& ws,
                       LaunchLog& log) {
  using Rw = Row<D, DV>;
  using Cl = Col<D, DV>;
  // r: the row pass's, c: the column pass's
  CUtensorMap rQ, rK, rV, rDO, rDQ, cK, cV, cQ, cDO, cDK, cDV;
  if (!tiles(&rQ, t.q, p, 2 * p.H, p.d, Rw::BM) || !tiles(&rK, t.k, p, 2 * p.Hk, p.d, Rw::BN) ||
      !tiles(&rV, t.v, p, p.Hk, p.dv, Rw::BN) || !tiles(&rDO, t.dO, p, p.H, p.dv, Rw::BM) ||
      !tiles(&rDQ, t.dq, p, 2 * p.H, p.d, Rw::BM) || !tiles(&cK, t.k, p, 2 * p.Hk, p.d, Cl::BM) ||
      !tiles(&cV, t.v, p, p.Hk, p.dv, Cl::BM) || !tiles(&cQ, t.q, p, 2 * p.H, p.d, Cl::BN) ||
      !tiles(&cDO, t.dO, p, p.H, p.dv, Cl::BN) || !tiles(&cDK, t.dk, p, 2 * p.Hk, p.d, Cl::BM) ||
      !tiles(&cDV, t.dv, p, p.Hk, p.dv, Cl::BM))
    return cudaErrorInvalidValue;
  const int blocks = (p.N + 63) / 64 * p.B * p.H;
  diff_tc_scalars<DV><<<blocks, 256, 0, log.stream>>>(
      static_cast<const uint4*>(t.o), static_cast<const uint4*>(t.rest),
      static_cast<const uint4*>(t.dO), t.lse, t.lam, ws.scal, p.H, p.N, p.dv / 8);
  cudaError_t e = cudaGetLastError();
  log.mark();
  if (e != cudaSuccess) return e;
  RowParams r;
  static_cast<Common&>(r) = common(p, t, ws, p.B * p.H);
  r.scal = ws.scal;
  r.d2 = ws.d2;
  const bool narrow = r.narrow_d || r.narrow_v;
  e = run(narrow ? diff_row_pass<D, DV, true> : diff_row_pass<D, DV, false>, r.units, 1, p.N,
          kThreads, Rw::SMEM, log, r, rQ, rK, rV, rDO, rDQ);
  if (e != cudaSuccess) return e;
  ColParams c;
  static_cast<Common&>(c) = common(p, t, ws, p.B * p.Hk);
  c.scal = ws.scal;
  c.parts = ws.parts;
  const int parts = col_parts(p);
  if (parts == 1)
    return run(narrow ? diff_col_pass<D, DV, true, false> : diff_col_pass<D, DV, false, false>,
               c.units, 1, p.N, kThreads, Cl::SMEM, log, c, cK, cV, cQ, cDO, cDK, cDV);
  e = run(narrow ? diff_col_pass<D, DV, true, true> : diff_col_pass<D, DV, false, true>, c.units,
          parts, p.N, kThreads, Cl::SMEM, log, c, cK, cV, cQ, cDO, cDK, cDV);
  if (e != cudaSuccess) return e;
  const size_t rows = (size_t)c.units * p.N, quads = rows * ((2 * D + DV) / 4);
  diff_col_join<D, DV><<<(unsigned)((quads + 255) / 256), 256, 0, log.stream>>>(
      reinterpret_cast<const float4*>(ws.parts), static_cast<uint2*>(t.dk),
      static_cast<uint2*>(t.dv), parts, p.N, rows, p.d, p.dv, p.scale);
  e = cudaGetLastError();
  log.mark();
  return e;
}

}  // namespace

size_t diff_tc_scalar_count(const DiffProblem& p) {
  return (size_t)p.B * p.H * ((p.N + 63) / 64) * 5 * 64;
}

size_t diff_tc_part_count(const DiffProblem& p) {
  const int parts = col_parts(p);
  return parts == 1 ? 0 : (size_t)parts * p.B * p.Hk * p.N * (2 * built(p.d) + built(p.dv));
}

bool diff_tc_supported(const DiffProblem& p) {
  return p.bf16 && p.d % 8 == 0 && p.dv % 8 == 0 && p.d <= 128 && p.dv <= 128;
}

cudaError_t diff_tc_forward(const DiffProblem& p, const DiffTensors& t, const DiffWorkspace& ws,
                            LaunchLog& log) {
  if (p.d <= 64)
    return p.dv <= 64 ? forward_d<64, 64>(p, t, ws, log) : forward_d<64, 128>(p, t, ws, log);
  return p.dv <= 64 ? forward_d<128, 64>(p, t, ws, log) : forward_d<128, 128>(p, t, ws, log);
}

cudaError_t diff_tc_backward(const DiffProblem& p, const DiffTensors& t, const DiffWorkspace& ws,
                             LaunchLog& log) {
  if (p.d <= 64)
    return p.dv <= 64 ? backward_d<64, 64>(p, t, ws, log) : backward_d<64, 128>(p, t, ws, log);
  return p.dv <= 64 ? backward_d<128, 64>(p, t, ws, log) : backward_d<128, 128>(p, t, ws, log);
}

}  // namespace fbob
