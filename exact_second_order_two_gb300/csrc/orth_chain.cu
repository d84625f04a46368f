// The products of an orthogonalisation as one kernel.
//
// Every step is a few products that depend on one another, matrix by matrix.  The blocks
// stay and take items (a tile of a product) in order, products of a stack's matrices
// side by side; an item whose operands are still being written waits for them: each
// product counts the parts of its tiles that are in memory.  So a product's last tiles
// and the next one's first run together (separate launches left 11 us between two products:
// 4 x 2048 x 2048 took 643 us).  Items are handed out by a counter, and an item waits for
// earlier ones only: those that hold earlier ones run, so that every wait ends, whatever
// else occupies the GPU.
//
// Warps: 8 finish tiles, one loads operands, one multiplies, one moves what is added in and
// results out, one takes items and waits for what they read; two accumulators, so that
// a tile is finished while the next is multiplied, and items taken ahead, so that the next
// tile's loads follow at once.  (With the waits in the loading and finishing warps a tile
// of 256 x 256 x 2048 took 15 us, 10.5 of them its MMAs.)
//
// A pair of CTAs multiplies a tile of 256 rows and 256 or 128 columns, each loading its
// 128 rows of P and half of the columns of Q, CTA 0 issuing for both: at 256 columns 64
// bytes a clock of shared memory and of L2 for each SM.  (Single CTAs with tiles of
// 128 x 128 need 128, which is what an SM has: 4 x 2048 x 2048 took 1.5 times as long.)
// 128 columns where 256 leave pairs idle.
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

using namespace tc;

constexpr int kStages = 5;
constexpr uint32_t kStageBytes = 2 * kTileBytes;
constexpr int kProducerWarp = 8, kMmaWarp = 9, kMoverWarp = 10, kSchedulerWarp = 11, kThreads = 384;
constexpr int kRing = 4;  // items on their way through the roles
// The two groups finish 64 columns at a time, each through two slots of 128 rows x 64
// columns: what is added comes in by TMA, the result is written in its place and leaves by
// TMA.  Values of two terms take both slots; of one term, where the result is symmetric, the
// second holds the tile transposed.  (Mirrored by stores from registers a tile of 128 x 64
// took 4 us, with a box more to store 2.)
constexpr uint32_t kOffSlots = kStages * kStageBytes;
constexpr uint32_t kOffMisc = kOffSlots + kGroups * 2 * kTileBytes;
constexpr uint32_t kSmem = kOffMisc + 512;
static_assert(kSmem <= 232448, "shared memory budget");

struct TileAt {
  int l, i, j, index;  // matrix, tile row and column, its number within the matrix
  bool below;          // the diagonal's square: its mirror is no tile
};
__device__ __forceinline__ TileAt tile_at(const Phase& p, int rows, int item) {
  const int t = item - p.first;
  TileAt r;
  r.l = t / p.tiles;
  r.index = t - r.l * p.tiles;
  if (p.sym) {  // rows of w, 2 w, 3 w .. tiles, of which the last w hold the diagonal
    const int w = kHigh / p.wide;
    int i = (int)((sqrtf(8.f * (r.index / w) + 1.f) - 1.f) * 0.5f);
    while (w * i * (i + 1) / 2 > r.index) --i;
    while (w * (i + 1) * (i + 2) / 2 <= r.index) ++i;
    r.i = i;
    r.j = r.index - w * i * (i + 1) / 2;
    r.below = r.j < w * i;
  } else {  // a column of tiles after the other: its operand tile is shared
    const int tm = (rows + kHigh - 1) / kHigh;
    r.j = r.index / tm;
    r.i = r.index - r.j * tm;
    r.below = false;
  }
  return r;
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
                                             const Phase& p, size_t base, int row, int col, int rows,
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
      const size_t at = base + (size_t)c * p.ld + pair;
      *reinterpret_cast<uint32_t*>(p.mirror[0] + at) = h;
      *reinterpret_cast<uint32_t*>(p.mirror[1] + at) = l;
    }
  }
}

// 32 values of a row straight to the caller's tensor, where no map can take them.
__device__ __forceinline__ void put_caller(const f2 (&v)[16], const ChainArgs& g, int l, int row, int col) {
  if (row >= g.rows) return;
  const size_t first = (size_t)l * g.rows * g.cols +
                       (g.y_transposed ? (size_t)col * g.rows + row : (size_t)row * g.cols + col);
  const size_t step = g.y_transposed ? g.rows : 1;
#pragma unroll
  for (int c = 0; c < 32; ++c)
    if (col + c < g.cols) {
      const float x = c & 1 ? v[c / 2].y : v[c / 2].x;
      if (g.y_bf16) static_cast<__nv_bfloat16*>(g.y)[first + c * step] = __float2bfloat16_rn(x);
      else static_cast<float*>(g.y)[first + c * step] = x;
    }
}

__device__ __forceinline__ void fence_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

// Waits until `count` reaches `target`, as wait_bar does; what was counted is then visible
// to this thread.
__device__ __forceinline__ bool wait_count(const int* count, int target, Abort* ab, int* status) {
  uint64_t t0 = 0;
  for (uint32_t it = 0;; ++it) {
    int n;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(n) : "l"(count) : "memory");
    if (n >= target) break;
    if (ab->flag) return false;
    if (it == 0) t0 = global_ns();
    else if ((it & 63u) == 0 && global_ns() - t0 > ab->limit_ns) {
      report_status(status, FBOB_ERR_TIMEOUT);
      ab->flag = 1;
      return false;
    }
    __nanosleep(64);
  }
  return true;
}

// mbarrier wait with what the other CTA of the pair wrote before its arrival.
__device__ __forceinline__ bool try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ void st_cluster(uint32_t addr, int v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ void sleep_10ms() {  // what an abort leaves in flight lands
  const uint64_t t0 = global_ns();
  while (global_ns() - t0 < 10000000ull) __nanosleep(10000);
}

// Slots that a group has in turn: one where values, or a tile and its mirror, take both.
__device__ __forceinline__ int slots_of(const Phase& p, const ChainArgs& g) {
  return p.sym || p.e_terms == 2 || p.o_terms == 2 || (p.o_terms == 0 && !g.y_bf16) ? 1 : 2;
}

// SPLIT.  The tensor cores cut each addition off to the accumulator's 24 bits, always
// towards zero, which over a long contraction would be the largest error by far (a
// steep polynomial of a result near 1 enlarges it ten times: 512 x 2048, fp32, was 5.6e-6 off
// with sums of 256 elements, the same in fp32 torch 2.8e-6).  So the accumulator takes
// g.part stages at a time, and the finishing warps add these sums up, rounded: for two-term
// operands 64 elements (more above 2^18), the products with low terms first; for one term
// 4096, where there are more than 65536 (1 x 2^22 was 3.5% off in one sum).
template <bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1) chain(const __grid_constant__ ChainArgs g) {
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
  uint64_t* written = e_full + 2 * kGroups;                       // [kGroups][2]
  uint64_t* r_full = written + 2 * kGroups;                       // [kRing]
  uint64_t* r_empty = r_full + kRing;                             // [kRing]
  uint64_t* go = r_empty + kRing;                                 // [kRing]
  uint64_t* started = go + kRing;
  uint64_t* drain = started + 1;
  static_assert((2 * kStages + 4 + 4 * kGroups + 3 * kRing + 2) * 8 <= 320, "barriers end below the rest");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc + 320);
  Abort* ab = reinterpret_cast<Abort*>(smem + kOffMisc + 328);
  volatile int* ring = reinterpret_cast<volatile int*>(smem + kOffMisc + 352);  // [kRing]: items, -1: none left
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  constexpr uint32_t kCols = 2 * kWide;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(t_full + b, 1);
      mbar_init(t_empty + b, 2 * kEpiWarps);
    }
    for (int i = 0; i < 2 * kGroups; ++i) {
      mbar_init(e_full + i, 1);
      mbar_init(written + i, kEpiWarps / kGroups);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(r_full + i, 1);
      mbar_init(go + i, 1);
      // the multiplying warp, and each CTA's finishing, loading and moving ones
      mbar_init(r_empty + i, 1 + 2 * (kEpiWarps + 2));
    }
    mbar_init(started, 1);
    mbar_init(drain, 1);
    ab->flag = 0;
    ab->limit_ns = g.wait_ns;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc_pair(tmem_slot, kCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the other's barriers are there
  tc_fence_after();
  after_previous();
  const uint32_t tmem = *tmem_slot;

  // waits for the n-th phase of a ring of barriers that the scheduler arrives on; false
  // after an abort
  auto await_ring = [&](uint64_t* bars, int n) -> bool {
    uint64_t* bar = bars + n % kRing;
    const uint32_t parity = (n / kRing) & 1;
    if (!try_wait_cluster(bar, parity)) {
      const uint64_t t0 = global_ns();
      while (!try_wait_cluster(bar, parity)) {
        if (ab->flag) return false;
        if (global_ns() - t0 > ab->limit_ns) {
          report_status(g.status, FBOB_ERR_TIMEOUT);
          ab->flag = 1;
          return false;
        }
      }
    }
    return true;
  };
  // the n-th item, for one who reads the ring
  auto next_item = [&](int n, int& item) -> bool {
    if (!await_ring(r_full, n)) return false;
    item = ring[n % kRing];
    return true;
  };
  auto item_read = [&](int n) {
    mbar_arrive_cluster(cluster_addr(r_empty + n % kRing, 0));
  };
  // the phase of an item (items come in order)
  auto phase_of = [&](int ph, int item) {
    while (ph + 1 < g.phases && item >= g.phase[ph + 1].first) ++ph;
    return ph;
  };
  if (warp == kSchedulerWarp) {
    if (lane == 0 && rank == 0) {
      int ph = 0;
      for (int n = 0;; ++n) {
        // one ahead: an item taken earlier would be missing where a block is idle
        if (n >= 1 && !wait_bar(started, (n - 1) & 1, ab, g.status)) break;
        int item = atomicAdd(g.ticket, 1);
        if (item >= g.items) item = -1;
        // The others learn of it at once, and see to what it needs of the arguments (maps, that
        // are far when first used); they load when what the phase reads of this matrix is
        // written.
        if (n >= kRing && !wait_bar(r_empty + n % kRing, ((n / kRing) - 1) & 1, ab, g.status)) break;
        ring[n % kRing] = item;
        mbar_arrive(r_full + n % kRing);
        st_cluster(cluster_addr(const_cast<int*>(ring + n % kRing), 1), item);
        mbar_arrive_cluster(cluster_addr(r_full + n % kRing, 1));
        if (item < 0) break;
        ph = phase_of(ph, item);
        const Phase& p = g.phase[ph];
        const int l = (item - p.first) / p.tiles;
        if (ph > 0 && !wait_count(g.done + (size_t)(ph - 1) * g.count + l, 2 * g.phase[ph - 1].tiles, ab,
                                  g.status))
          break;
        mbar_arrive(go + n % kRing);
        mbar_arrive_cluster(cluster_addr(go + n % kRing, 1));
      }
    }
  } else if (warp == kProducerWarp) {
    // The whole warp, with operands that are the same in all lanes; one lane issues.  What this
    // loop does for a stage bounds the rate: a look at the abort flag in it (which the
    // waits do when they have to wait) made 4096 x 16384 5% slower.
    {
      int it = 0, ph = 0;
      bool ok = true;
      for (int n = 0; ok; ++n) {
        int item = -1;
        if (!__all_sync(0xffffffffu, next_item(n, item))) break;
        if (lane == 0) item_read(n);
        item = __reduce_max_sync(0xffffffffu, item);
        if (item < 0) break;
        ph = phase_of(ph, item);
        const Phase& p = g.phase[ph];
        const TileAt at = tile_at(p, g.rows, item);
        const int half = p.wide / 2;  // of the tile's columns, this CTA's part of Q
        const int row = at.i * kHigh + rank * kTile, col = at.j * p.wide + rank * half;
        const int blocks = (p.depth + kDepth - 1) / kDepth;
        const bool nn = p.nn;
        if (lane < p.nseg) {
          tma_prefetch_desc(&g.maps[p.seg_a[lane]]);
          tma_prefetch_desc(&g.maps[p.seg_b[lane]]);
        }
        if (!__all_sync(0xffffffffu, await_ring(go, n))) break;
        fence_async_all();  // the loads see what the scheduler saw written
        // a segment after the other; SPLIT: every pair of terms of one stretch of the
        // contraction together
        const int outer = SPLIT ? blocks : p.nseg, inner = SPLIT ? p.nseg : blocks;
        for (int o = 0; ok && o < outer; ++o) {
          const CUtensorMap *ma = &g.maps[p.seg_a[SPLIT ? 0 : o]], *mb = &g.maps[p.seg_b[SPLIT ? 0 : o]];
          int la = p.at_a[SPLIT ? 0 : o] + at.l, lb = p.at_b[SPLIT ? 0 : o] + at.l;
          for (int i = 0; i < inner; ++i, ++it) {
            const int s = it % kStages, k = SPLIT ? o : i;
            if (it >= kStages && !warp_wait(empty + s, ((it / kStages) - 1) & 1, ab, g.status)) {
              ok = false;
              break;
            }
            if (lane != 0) continue;
            if (SPLIT) {
              ma = &g.maps[p.seg_a[i]];
              mb = &g.maps[p.seg_b[i]];
              la = p.at_a[i] + at.l;
              lb = p.at_b[i] + at.l;
            }
            uint8_t *pa = smem + s * kStageBytes, *pb = pa + kTileBytes;
            if (rank == 0) mbar_arrive_expect_tx(full + s, 2 * (kTileBytes + half * 128));
            const uint32_t bar = cluster_addr(full + s, 0);
            tma_load_3d_pair(pa, ma, bar, k * kDepth, row, la);
            if (nn) {
              tma_load_3d_pair(pb, mb, bar, col, k * kDepth, lb);
              if (half > 64) tma_load_3d_pair(pb + kTileBytes / 2, mb, bar, col + 64, k * kDepth, lb);
            } else {
              tma_load_3d_pair(pb, mb, bar, k * kDepth, col, lb);
            }
          }
        }
      }
      __syncwarp();
      // every load issued has landed before the block exits: CTA 0 sees the barriers
      // that count both CTAs' loads; what an abort leaves uncounted gets a fixed time
      if (rank == 0 && lane == 0)
        for (int u = max(0, it - kStages); u < it; ++u)
          mbar_wait_bounded(full + u % kStages, (u / kStages) & 1, g.status, 100000000ull);
      if (ab->flag) sleep_10ms();
    }
  } else if (warp == kMmaWarp) {
    if (rank == 0) {
      int it = 0, nb = 0, ph = 0;  // stages, accumulators taken
      bool ok = true;
      for (int n = 0; ok; ++n) {
        int item = -1;
        if (!__all_sync(0xffffffffu, next_item(n, item))) break;
        if (lane == 0) item_read(n);
        item = __reduce_max_sync(0xffffffffu, item);  // in a uniform register, as what follows from it
        if (item < 0) break;
        ph = phase_of(ph, item);
        const Phase& p = g.phase[ph];
        const bool nn = p.nn;
        const uint32_t id = idesc_f16(kHigh, p.wide, nn);
        const int total = p.nseg * ((p.depth + kDepth - 1) / kDepth);
        const int part = SPLIT ? g.part : total;
        for (int k0 = 0; ok && k0 < total; k0 += part, ++nb) {
          const uint32_t d = tmem + (nb & 1) * kWide;
          if (nb >= 2 && !warp_wait(t_empty + (nb & 1), ((nb >> 1) - 1) & 1, ab, g.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const int k1 = min(total, k0 + part);
          for (int k = k0; k < k1; ++k, ++it) {
            const int s = it % kStages;
            if (!warp_wait(full + s, (it / kStages) & 1, ab, g.status)) {
              ok = false;
              break;
            }
            tc_fence_after();
            if (k == 0 && lane == 0) mbar_arrive(started);
            const uint32_t a_lo = opaque(lo_kmajor(sb + s * kStageBytes));
            const uint32_t b_at = sb + s * kStageBytes + kTileBytes;
            const uint32_t b_lo = opaque(nn ? lo_mnmajor(b_at, kTileBytes / 2) : lo_kmajor(b_at));
            const uint32_t b_step = nn ? kstep_off(1) : 2;
#pragma unroll
            for (int u = 0; u < kDepth / 16; ++u)
              mma_ss_pair_w(d, a_lo + 2 * u, b_lo + b_step * u, id, k - k0 + u > 0 ? 1u : 0u);
            mma_commit_pair_w(empty + s, 3);
          }
          if (ok) mma_commit_pair_w(t_full + (nb & 1), 3);
        }
      }
      // every MMA this warp issued has completed before TMEM is released
      mma_commit_pair_w(drain, 1);
      mbar_wait_bounded(drain, 0, g.status, 100000000ull);
    }
  } else if (warp == kMoverWarp) {
    if (lane == 0) {
      uint32_t uses = 0;  // parity of each group's slots: bit 2 group + slot
      int ph = 0;
      bool ok = true;
      for (int n = 0; ok; ++n) {
        int item;
        if (!next_item(n, item)) break;
        item_read(n);
        if (item < 0) break;
        ph = phase_of(ph, item);
        const Phase& p = g.phase[ph];
        const TileAt at = tile_at(p, g.rows, item);
        const int row0 = at.i * kHigh + rank * kTile;
        const bool to_caller = p.o_terms == 0, mapped = !to_caller || g.y_mapped;
        const bool mirror = p.sym && at.below;
        const int nslots = slots_of(p, g), chunks = p.wide / (64 * kGroups);
        // what is added to chunk c of a group comes into its slot
        auto prepare = [&](int group, int c) {
          const int s = 2 * group + c % nslots, col = at.j * p.wide + (group + c * kGroups) * 64;
          uint8_t* const slot = smem + kOffSlots + s * kTileBytes;
          if (p.e_terms) {
            mbar_arrive_expect_tx(e_full + s, p.e_terms * kTileBytes);
            tma_load_3d(slot, &g.maps[p.e_map[0]], e_full + s, col, row0, p.e_at + at.l);
            if (p.e_terms == 2)
              tma_load_3d(slot + kTileBytes, &g.maps[p.e_map[1]], e_full + s, col, row0, p.e_at + at.l);
          } else {
            mbar_arrive(e_full + s);
          }
        };
        if (p.e_terms) {
          if (!await_ring(go, n)) break;
          fence_async_all();
        }
        if (ab->flag) break;
        for (int group = 0; group < kGroups; ++group)
          for (int c = 0; c < nslots && c < chunks; ++c) prepare(group, c);
        for (int c = 0; ok && c < chunks; ++c)
          for (int group = 0; ok && group < kGroups; ++group) {
            const int s = 2 * group + c % nslots, col0 = at.j * p.wide + (group + c * kGroups) * 64;
            uint8_t* const slot = smem + kOffSlots + s * kTileBytes;
            if (!wait_bar(written + s, (uses >> s) & 1, ab, g.status) || ab->flag) {
              ok = false;
              break;
            }
            uses ^= 1u << s;
            if (mapped && row0 < g.rows && col0 < p.cols) {
              const CUtensorMap *m0 = &g.maps[p.o_map[0]], *m1 = &g.maps[p.o_map[1]];
              const int l = p.o_at + at.l;
              tma_store_3d(m0, slot, col0, row0, l);
              if (p.o_terms == 2) {
                tma_store_3d(m1, slot + kTileBytes, col0, row0, l);
              } else if (mirror) {
                tma_store_3d(m1, slot + kTileBytes, row0, col0, l);
                if (row0 + 64 < g.rows)
                  tma_store_3d(m1, slot + kTileBytes + kTileBytes / 2, row0 + 64, col0, l);
              } else if (to_caller && !g.y_bf16 && col0 + 32 < p.cols) {
                tma_store_3d(m0, slot + kTileBytes, col0 + 32, row0, l);
              }
              bulk_commit_group();
            }
            if (c + nslots < chunks) {
              bulk_wait_read_all();
              prepare(group, c + nslots);
            }
          }
        if (!ok) break;
        // the tile is in memory: its stores, and what the finishing warps wrote themselves
        bulk_wait_all();
        asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(g.done + (size_t)ph * g.count + at.l)
                     : "memory");
      }
      bulk_wait_all();
      if (ab->flag) sleep_10ms();
    }
  } else {
    const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
    const int group = warp >> 2, r = 32 * (warp & 3) + lane;
    uint32_t uses = 0;
    int ph = 0, nb = 0, scaled = -1, scaled_ph = -1, shift = 0;
    bool ok = true;
    for (int n = 0; ok; ++n) {
      int item = -1;
      if (!__all_sync(0xffffffffu, next_item(n, item))) break;
      if (lane == 0) item_read(n);
      if (item < 0) break;
      ph = phase_of(ph, item);
      const Phase& p = g.phase[ph];
      const TileAt at = tile_at(p, g.rows, item);
      const int row0 = at.i * kHigh + rank * kTile, row = row0 + r;
      const bool to_caller = p.o_terms == 0, mapped = !to_caller || g.y_mapped;
      const bool mirror = p.sym && at.below;
      const int nslots = slots_of(p, g), chunks = p.wide / (64 * kGroups);  // chunks for each group
      float alpha = p.alpha, beta = p.beta;
      if (p.fpow) {
        const float f = g.info[at.l].f, ff = p.fpow == 2 ? f * f : f;
        alpha *= ff;
        beta *= ff;
      }
      int by_alpha = 0, by_beta = 0;  // powers of two
      if (p.step >= 0) {
        const int e0 = g.info[at.l].e[p.step], e1 = g.info[at.l].e[p.step + 1];
        by_alpha = p.e_alpha[0] * e0 + p.e_alpha[1] * e1;
        by_beta = p.e_beta[0] * e0 + p.e_beta[1] * e1;
      }
      if (p.scale_sums) {
        if (!__all_sync(0xffffffffu, await_ring(go, n))) break;
        if (scaled != at.l || scaled_ph != ph) {
          const float* q = p.scale_sums + (size_t)at.l * p.scale_parts;
          float nu2 = 0.f;
          for (int i = lane; i < p.scale_parts; i += 32) nu2 += __ldcg(q + i);
          shift = rescaling(Squares{warp_sum(nu2), 0}, p.target);
          scaled = at.l;
          scaled_ph = ph;
        }
        by_alpha += shift;
        by_beta += shift;
        if (at.index == 0 && threadIdx.x == 0 && rank == 0) p.exp_out[at.l] = __ldcg(p.exp_in + at.l) + shift;
      }
      if (by_alpha | by_beta) {
        alpha = ldexpf(alpha, by_alpha);
        beta = ldexpf(beta, by_beta);
      }
      f2 total[SPLIT ? 32 : 1];  // of the thread's 64 columns
      if (SPLIT) {
#pragma unroll
        for (int k = 0; k < 32; ++k) total[SPLIT ? k : 0] = f2{0.f, 0.f};
        const int stages = p.nseg * ((p.depth + kDepth - 1) / kDepth);
        for (int k0 = 0; ok && k0 < stages; k0 += g.part, ++nb) {
          if (!warp_wait(t_full + (nb & 1), (nb >> 1) & 1, ab, g.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t acc[32];
            tmem_ld32(tmem + lane_off + (nb & 1) * kWide + group * 64 + 32 * h, acc);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              f2& t = total[SPLIT ? 16 * h + k : 0];
              t = add2(t, f2{__uint_as_float(acc[2 * k]), __uint_as_float(acc[2 * k + 1])});
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(cluster_addr(t_empty + (nb & 1), 0));
        }
        if (!ok) break;
      } else {
        if (!warp_wait(t_full + (n & 1), (n >> 1) & 1, ab, g.status)) break;
        tc_fence_after();
      }
      float sum = 0.f;
#pragma unroll 1
      for (int c = 0; c < chunks; ++c) {
        const int in_tile = (group + c * kGroups) * 64, col0 = at.j * p.wide + in_tile;
        const int s = 2 * group + c % nslots;
        uint8_t* const slot = smem + kOffSlots + s * kTileBytes;
        if (!warp_wait(e_full + s, (uses >> s) & 1, ab, g.status)) {
          ok = false;
          break;
        }
        uses ^= 1u << s;
#pragma unroll(SPLIT ? 2 : 1)
        for (int h = 0; h < 2; ++h) {
          const int col = col0 + 32 * h;
          f2 v[16];
          if (SPLIT) {
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = mul2(f2{alpha, alpha}, total[SPLIT ? 16 * h + k : 0]);
          } else {
            uint32_t acc[32];
            tmem_ld32(tmem + lane_off + (n & 1) * kWide + in_tile + 32 * h, acc);
#pragma unroll
            for (int k = 0; k < 16; ++k)
              v[k] = mul2(f2{alpha, alpha}, f2{__uint_as_float(acc[2 * k]), __uint_as_float(acc[2 * k + 1])});
          }
          if (p.e_terms) add_slot(v, slot, r, h, beta);
          if (p.e_terms == 2) add_slot(v, slot + kTileBytes, r, h, beta);
          if (p.sums) {  // (what lies outside is zero)
#pragma unroll
            for (int k = 0; k < 16; ++k) sum = fmaf(v[k].x, v[k].x, fmaf(v[k].y, v[k].y, sum));
          }
          uint32_t w[16];
          if (!to_caller) {
#pragma unroll
            for (int k = 0; k < 16; ++k) w[k] = to_halves(v[k]);
            put_slot(w, slot, r, h);
            if (p.o_terms == 2) {
              uint32_t lo[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) lo[k] = to_halves(fma2(f2{-1.f, -1.f}, halves(w[k]), v[k]));
              put_slot(lo, slot + kTileBytes, r, h);
              if (mirror) {
                put_mirrored(w, lo, p, (size_t)(p.o_at + at.l) * g.rows * p.ld, row, col, g.rows, p.cols);
                fence_async_all();  // (they are read by TMA)
                __threadfence();
              }
            } else if (mirror) {
              put_slot_transposed(w, slot + kTileBytes, r, h);
            }
          } else if (!mapped) {
            put_caller(v, g, at.l, row, col);
          } else if (g.y_bf16) {
#pragma unroll
            for (int k = 0; k < 16; ++k) w[k] = pack_bf16(v[k].x, v[k].y);
            put_slot(w, slot, r, h);
          } else if (h == 0) {  // 32 fp32 columns fill a slot's row: kept in both until all is read
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
        if (c == chunks - 1) {
          tc_fence_before();
          if (p.sums) {
            sum = warp_sum(sum);
            if (lane == 0) {
              p.sums[((size_t)at.l * p.tiles + at.index) * (2 * kEpiWarps) + rank * kEpiWarps + warp] = sum;
              __threadfence();
            }
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(written + s);
          if (!SPLIT && c == chunks - 1) mbar_arrive_cluster(cluster_addr(t_empty + (n & 1), 0));
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  __syncwarp();
  cluster_sync();  // neither leaves before the other's last use of it
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kCols);
  }
}

}  // namespace

cudaError_t launch_chain(const ChainArgs& g, bool split, LaunchLog& log) {
  auto kernel = split ? chain<true> : chain<false>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  const int grid = 2 * (g.items < kPairs ? g.items : kPairs);
  return launch_next(kernel, dim3((unsigned)grid), kThreads, kSmem, 2, log, g);
}

}  // namespace orth
}  // namespace fbob
