// Norms of queries and keys for each head, with the rotary positions in the
// same pass.  A row x of d features at position p becomes
//   y = R (w . n),   n = r x,   r = (<x, x> / d + eps)^(-1/2),
// with R the rotation of its feature pairs by p (times the magnitude; features
// that are not turned stay).  With g = R^T dy and h = w . g, the gradients are
//   dx = r (h - n <h, n> / d),   dw = sum over rows of g . n,
// and for cotangents a of dx and c of dw, with t = r (a - n <a, n> / d) and
// u = c . g - (r / d) (<a, n> h + <h, n> a), those of x, w and dy are
//   gx = r (u - n <u, n> / d) - (r / d) <h, t> n,   gw = sum over rows of g . t,
//   gdy = R (w . t + c . n).
// Every inner product is one with x, times a power of r, or <h, a>: all of a row's
// sums are made in one exchange, before r is known, and each row is read once.
//
// Bound: memory.  A group of lanes holds a row (two runs of P elements a lane, as
// the rotation pairs them) and walks over heads of one position, so that a sine and
// cosine serve them all; queries and keys are one launch.  The sums over rows
// are carried in registers by blocks that stay (a few per SM), added up in the block
// through shared memory, and over the blocks by a second launch: every sum in a
// fixed order.  norm_rows takes chunks of 16 or 8 features, where they tile the turned and
// the other part; norm_kernel what is left, a feature at a time: odd widths, odd addresses, and
// aligned heads of which as many are turned as no chunk tiles (20 of 40, 12 of 64).  8 + 8
// heads x 26214 x 40, bf16, forward, backward and second derivative: 44, 81 and 116 us with 20
// turned, 30, 46 and 75 in chunks with all turned; x 16384 x 64 with 12 turned 36, 56 and 85,
// with all 21, 31 and 46.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "ops.h"
#include "rotary.cuh"

namespace fbob {
namespace {

using namespace rope;

constexpr int kThreads = 128;
constexpr int kMaxDim = 256;

// One tensor's part of a call, as the kernels read it.
struct Side {
  const void *x, *w, *dy, *a, *c;
  void *y, *ddy;
  long long xs[3], dys[3], as[3], ys[3], ddys[3];  // over batch, head, position, in elements
  int H, heads, groups;  // heads per unit, units per block of positions
  int blocks;            // thread blocks that work on it
  long long units;
  bool sums;             // the gradient of w is wanted
};

struct NormArgs {
  Side side[2];
  const double* inv_freq;
  const long long* positions;  // null: offset + n
  long long pos_sb, offset;
  float* partial;              // [blocks with sums][d]
  int B, N, d, half;           // half = rotary_dim / 2 pairs
  int lanes;                   // lanes of a row: a power of two
  int w_bf16;
  float eps, inv_d, magnitude;
};

// A lane's features of a row: C chunks of two runs of P.
template <int P, int C>
struct Row {
  float u[C][P], v[C][P];
};

// Which features a lane holds.
template <int P, int C>
struct Place {
  int e0[C], e1[C];
  bool one[C], two[C], turned[C];
  __device__ __forceinline__ Place(const NormArgs& a, int lane, bool interleaved) {
    const int chunks = a.d / (2 * P) + (P == 1 ? (a.d & 1) : 0), rot = a.half / P;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int c = lane + j * a.lanes;
      one[j] = c < chunks;
      turned[j] = c < rot;
      if (turned[j]) {
        e0[j] = interleaved ? 2 * P * c : P * c;
        e1[j] = interleaved ? e0[j] + P : e0[j] + a.half;
      } else {
        e0[j] = 2 * a.half + (c - rot) * 2 * P;
        e1[j] = e0[j] + P;
      }
      two[j] = one[j] && e1[j] < a.d;  // not for an odd width's last feature
    }
  }
};

template <typename T, int P, int C>
struct Raw {
  Vec<T, P> u[C], v[C];
  __device__ __forceinline__ void load(const T* p, const Place<P, C>& at) {
#pragma unroll
    for (int j = 0; j < C; ++j) {
      if (at.one[j]) u[j].load(p + at.e0[j]);
      if (at.two[j]) v[j].load(p + at.e1[j]);
    }
  }
  __device__ __forceinline__ void get(Row<P, C>& r, const Place<P, C>& at) const {
#pragma unroll
    for (int j = 0; j < C; ++j) {
#pragma unroll
      for (int i = 0; i < P; ++i) r.u[j][i] = r.v[j][i] = 0.f;
      if (at.one[j]) u[j].get(r.u[j]);
      if (at.two[j]) v[j].get(r.v[j]);
    }
  }
};

template <typename T, int P, int C>
__device__ __forceinline__ void put(T* p, const Row<P, C>& r, const Place<P, C>& at) {
#pragma unroll
  for (int j = 0; j < C; ++j) {
    Vec<T, P> t;
    if (at.one[j]) {
      t.set(r.u[j]);
      t.store(p + at.e0[j]);
    }
    if (at.two[j]) {
      t.set(r.v[j]);
      t.store(p + at.e1[j]);
    }
  }
}

// f of each of the lane's features, with its index i in the run
#define FBOB_EACH(j, i) \
  _Pragma("unroll") for (int j = 0; j < C; ++j) _Pragma("unroll") for (int i = 0; i < P; ++i)

template <int P, int C>
__device__ __forceinline__ float dot(const Row<P, C>& a, const Row<P, C>& b) {
  float s = 0.f;
  FBOB_EACH(j, i) s = fmaf(a.u[j][i], b.u[j][i], fmaf(a.v[j][i], b.v[j][i], s));
  return s;
}

// Sums over the lanes of a row, every lane its own copy.
template <int K>
__device__ __forceinline__ void row_sums(float (&s)[K], int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) {
#pragma unroll
    for (int k = 0; k < K; ++k) s[k] += __shfl_xor_sync(0xffffffffu, s[k], o);
  }
}

// The turning of a row at one position: cosines and sines (with the magnitude).
template <int P, int C>
struct Angles {
  float cs[C][P], sn[C][P];
  __device__ __forceinline__ void at(long long p, const unsigned long long* turns, int lane, int lanes,
                                     const Place<P, C>& place, float magnitude) {
#pragma unroll
    for (int j = 0; j < C; ++j) {
      if (!place.turned[j]) continue;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const unsigned long long t =
            (unsigned long long)p * turns[(lane + j * lanes) * P + i];
        float s, c;
        sincos_turns((uint32_t)((t + 0x80000000ull) >> 32), s, c);
        cs[j][i] = c * magnitude;
        sn[j][i] = s * magnitude;
      }
    }
  }
  template <bool INTERLEAVED, bool INVERSE>
  __device__ __forceinline__ void apply(Row<P, C>& r, const Place<P, C>& place) const {
#pragma unroll
    for (int j = 0; j < C; ++j) {
      if (!place.turned[j]) continue;
      if (INVERSE) {
        float back[P];
#pragma unroll
        for (int i = 0; i < P; ++i) back[i] = -sn[j][i];
        turn<P, INTERLEAVED>(r.u[j], r.v[j], cs[j], back);
      } else {
        turn<P, INTERLEAVED>(r.u[j], r.v[j], cs[j], sn[j]);
      }
    }
  }
};

__device__ __forceinline__ float vector_at(const void* p, int bf16, int i) {
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i])
              : static_cast<const float*>(p)[i];
}

// A [d] vector from shared memory, at the lane's features.
template <int P, int C>
__device__ __forceinline__ void from_shared(Row<P, C>& r, const float* v, const Place<P, C>& at) {
  FBOB_EACH(j, i) {
    r.u[j][i] = at.one[j] ? v[at.e0[j] + i] : 0.f;
    r.v[j][i] = at.two[j] ? v[at.e1[j] + i] : 0.f;
  }
}

enum { kForward, kBackward, kSecond };

// A block's sums over rows, from those of its groups of lanes.
__device__ __forceinline__ void block_partial(const float* red, const NormArgs& a, bool second_side, int block,
                                              int per_block) {
  __syncthreads();
  float* const out = a.partial + ((size_t)(second_side && a.side[0].sums ? a.side[0].blocks : 0) + block) * a.d;
  for (int i = threadIdx.x; i < a.d; i += kThreads) {
    float t = 0.f;
    for (int k = 0; k < per_block; ++k) t += red[k * a.d + i];
    out[i] = t;
  }
}

// Rows whose loads are in flight together.
template <int OP, int C>
constexpr int kRows = C > 1 || OP != kForward ? 1 : 2;

// Shared memory: [half] angles of one position, [d] w, [d] c; then, for the sums
// at the end, [rows of a block][d].
template <int OP, typename TI, typename TO, int P, int C, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) norm_kernel(const __grid_constant__ NormArgs a) {
  extern __shared__ unsigned long long turns[];
  float* const sw = reinterpret_cast<float*>(turns + a.half);
  float* const sc = sw + a.d;
  constexpr int U = kRows<OP, C>;
  if (OP != kForward) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // norm_sums
  const bool second_side = blockIdx.x >= (unsigned)a.side[0].blocks;
  const Side& s = a.side[second_side];
  const int block = blockIdx.x - (second_side ? a.side[0].blocks : 0);
  const int lane = threadIdx.x & (a.lanes - 1), group = threadIdx.x / a.lanes;
  const int per_block = kThreads / a.lanes;  // positions of a unit
  const Place<P, C> place(a, lane, INTERLEAVED);

  turns_table<kThreads>(turns, a.inv_freq, a.half);
  for (int i = threadIdx.x; i < a.d; i += kThreads) {
    sw[i] = s.w ? vector_at(s.w, a.w_bf16, i) : 1.f;
    if (OP == kSecond) sc[i] = s.c ? vector_at(s.c, a.w_bf16, i) : 0.f;
  }
  __syncthreads();
  Row<P, C> w, c, acc;
  from_shared(w, sw, place);
  if (OP == kSecond) from_shared(c, sc, place);
  FBOB_EACH(j, i) acc.u[j][i] = acc.v[j][i] = 0.f;

  const long long items = (long long)a.B * a.N;
  for (long long unit = block; unit < s.units; unit += s.blocks) {
    const long long ib = unit / s.groups;
    const int h0 = (int)(unit - ib * s.groups) * s.heads, h1 = min(s.H, h0 + s.heads);
    const long long item = ib * per_block + group;
    const bool active = item < items;  // the other groups' lanes only take part in exchanges
    const long long b = active ? item / a.N : 0, n = active ? item - b * a.N : 0;
    const TI* __restrict__ x = static_cast<const TI*>(s.x) + b * s.xs[0] + n * s.xs[2];
    const TO* __restrict__ dy = static_cast<const TO*>(s.dy) + b * s.dys[0] + n * s.dys[2];
    const TI* __restrict__ ca = static_cast<const TI*>(s.a) + b * s.as[0] + n * s.as[2];
    Angles<P, C> angles;
    const long long pos = !active ? 0 : a.positions ? a.positions[b * a.pos_sb + n] : a.offset + n;
    for (int hb = h0; hb < h1; hb += U) {
      Raw<TI, P, C> rx[U], ra[U];
      Raw<TO, P, C> rdy[U];
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (active && hb + i < h1) {
          rx[i].load(x + (hb + i) * s.xs[1], place);
          if (OP != kForward) rdy[i].load(dy + (hb + i) * s.dys[1], place);
          if (OP == kSecond && s.a) ra[i].load(ca + (hb + i) * s.as[1], place);
        }
      if (hb == h0) angles.at(pos, turns, lane, a.lanes, place, a.magnitude);
#pragma unroll
      for (int k = 0; k < U; ++k) {
        if (hb + k >= h1) break;  // the same for the whole block
        Row<P, C> xv, g, av;
        if (active) {
          rx[k].get(xv, place);
          if (OP != kForward) rdy[k].get(g, place);
        } else {
          FBOB_EACH(j, i) xv.u[j][i] = xv.v[j][i] = g.u[j][i] = g.v[j][i] = 0.f;
        }
        if (OP == kForward) {
          float sum[1] = {dot(xv, xv)};
          row_sums(sum, a.lanes);
          const float r = rsqrtf(fmaf(sum[0], a.inv_d, a.eps));
          FBOB_EACH(j, i) {
            xv.u[j][i] *= r * w.u[j][i];
            xv.v[j][i] *= r * w.v[j][i];
          }
          angles.template apply<INTERLEAVED, false>(xv, place);
          if (active)
            put<TO, P, C>(static_cast<TO*>(s.y) + b * s.ys[0] + (hb + k) * s.ys[1] + n * s.ys[2], xv,
                          place);
        } else if (OP == kBackward) {
          angles.template apply<INTERLEAVED, true>(g, place);
          float sum[2] = {dot(xv, xv), 0.f};
          FBOB_EACH(j, i) sum[1] = fmaf(w.u[j][i] * g.u[j][i], xv.u[j][i],
                                        fmaf(w.v[j][i] * g.v[j][i], xv.v[j][i], sum[1]));
          row_sums(sum, a.lanes);
          // (0 where there is no row: without eps it would be an infinity times the zeros)
          const float r = active ? rsqrtf(fmaf(sum[0], a.inv_d, a.eps)) : 0.f;
          const float back = r * r * sum[1] * a.inv_d;  // dx = r (h - back x)
          FBOB_EACH(j, i) {
            acc.u[j][i] = fmaf(g.u[j][i], r * xv.u[j][i], acc.u[j][i]);
            acc.v[j][i] = fmaf(g.v[j][i], r * xv.v[j][i], acc.v[j][i]);
            xv.u[j][i] = r * fmaf(-back, xv.u[j][i], w.u[j][i] * g.u[j][i]);
            xv.v[j][i] = r * fmaf(-back, xv.v[j][i], w.v[j][i] * g.v[j][i]);
          }
          if (active)
            put<TI, P, C>(static_cast<TI*>(s.y) + b * s.ys[0] + (hb + k) * s.ys[1] + n * s.ys[2], xv,
                          place);
        } else {
          if (active && s.a) {
            ra[k].get(av, place);
          } else {
            FBOB_EACH(j, i) av.u[j][i] = av.v[j][i] = 0.f;
          }
          angles.template apply<INTERLEAVED, true>(g, place);
          // <x, x>, <h, x>, <a, x>, <h, a>, <c . g, x>
          float sum[5] = {dot(xv, xv), 0.f, dot(av, xv), 0.f, 0.f};
          FBOB_EACH(j, i) {
            const float hu = w.u[j][i] * g.u[j][i], hv = w.v[j][i] * g.v[j][i];
            sum[1] = fmaf(hu, xv.u[j][i], fmaf(hv, xv.v[j][i], sum[1]));
            sum[3] = fmaf(hu, av.u[j][i], fmaf(hv, av.v[j][i], sum[3]));
            sum[4] = fmaf(c.u[j][i] * g.u[j][i], xv.u[j][i],
                          fmaf(c.v[j][i] * g.v[j][i], xv.v[j][i], sum[4]));
          }
          row_sums(sum, a.lanes);
          // (0 where there is no row: without eps it would be an infinity times the zeros)
          const float r = active ? rsqrtf(fmaf(sum[0], a.inv_d, a.eps)) : 0.f;
          const float hn = r * sum[1] * a.inv_d, an = r * sum[2] * a.inv_d;  // <h, n> / d, <a, n> / d
          const float ht = r * (sum[3] - r * sum[1] * an);                   // <h, t>
          const float un = r * a.inv_d * sum[4] - 2.f * r * an * hn;         // <u, n> / d
          // gx = r (u - back x), t = r (a - at x)
          const float back = r * (un + ht * a.inv_d), at = an * r;
          FBOB_EACH(j, i) {
            const float xu = xv.u[j][i], xw = xv.v[j][i], au = av.u[j][i], aw = av.v[j][i];
            const float gu = g.u[j][i], gw = g.v[j][i];
            const float tu = r * fmaf(-at, xu, au), tw = r * fmaf(-at, xw, aw);
            acc.u[j][i] = fmaf(gu, tu, acc.u[j][i]);
            acc.v[j][i] = fmaf(gw, tw, acc.v[j][i]);
            const float uu = c.u[j][i] * gu - r * (an * (w.u[j][i] * gu) + hn * au);
            const float uw = c.v[j][i] * gw - r * (an * (w.v[j][i] * gw) + hn * aw);
            g.u[j][i] = fmaf(w.u[j][i], tu, c.u[j][i] * (r * xu));
            g.v[j][i] = fmaf(w.v[j][i], tw, c.v[j][i] * (r * xw));
            xv.u[j][i] = r * fmaf(-back, xu, uu);
            xv.v[j][i] = r * fmaf(-back, xw, uw);
          }
          angles.template apply<INTERLEAVED, false>(g, place);
          if (active) {
            put<TI, P, C>(static_cast<TI*>(s.y) + b * s.ys[0] + (hb + k) * s.ys[1] + n * s.ys[2], xv,
                          place);
            put<TO, P, C>(
                static_cast<TO*>(s.ddy) + b * s.ddys[0] + (hb + k) * s.ddys[1] + n * s.ddys[2], g,
                place);
          }
        }
      }
    }
  }
  if (OP == kForward || !s.sums) return;
  float* const red = sc + (OP == kSecond ? a.d : 0);  // [per_block][d]
  FBOB_EACH(j, i) {
    if (place.one[j]) red[group * a.d + place.e0[j] + i] = acc.u[j][i];
    if (place.two[j]) red[group * a.d + place.e1[j] + i] = acc.v[j][i];
  }
  block_partial(red, a, second_side, block, per_block);
}


// ---------------------------------------------------------------------------
// Rows in chunks of 16 or 8 features, aligned.  Arithmetic is in pairs of
// features; rows come through shared memory, a row ahead of the one that is worked on, and
// weights are read from there where a row needs them.  32 heads x 8192 x 128, bf16, with the
// sums over rows: 33 us forward, 48 backward and 73 for the second derivative (4.0 to 4.6
// TB/s).  With rows loaded into registers 33, 62 and 93; with everything in registers, one
// feature at a time, 39, 59 and 127.
// ---------------------------------------------------------------------------
using f2 = float2;
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ f2 mul2(f2 a, f2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ f2 both(float a) { return f2{a, a}; }

template <int P>
struct Run {  // P features
  f2 p[P / 2];
};
template <int P>
struct Runs {  // the two runs of a chunk
  Run<P> u, v;
};
template <int P>
__device__ __forceinline__ void clear(Runs<P>& r) {
#pragma unroll
  for (int i = 0; i < P / 2; ++i) r.u.p[i] = r.v.p[i] = both(0.f);
}

// A lane's two runs of a row, on their way through shared memory: each thread copies its
// own pieces, as many rows ahead as the ring holds, and no other reads them.  Pieces are 16
// bytes, or a whole run of 8.
template <typename T, int P>
constexpr int kPiece = P * (int)sizeof(T) < 16 ? P * (int)sizeof(T) : 16;
template <typename T, int P>
constexpr int kRowBytes = 2 * P * (int)sizeof(T) * kThreads;  // of a block's threads

template <int BYTES>
__device__ __forceinline__ void copy_piece(uint32_t to, const void* from, bool whole) {
  // fp32 runs are pieces of half a sector each, runs of 8 bytes less: through L1, where one
  // finds what another brought
  if (BYTES == 16 && whole) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"(BYTES) : "memory");
}
template <typename T, int P>
__device__ __forceinline__ void copy_row(uint32_t to, const T* p, int e0, int e1) {
  constexpr int B = kPiece<T, P>, N = P * (int)sizeof(T) / B;  // pieces of a run
  to += threadIdx.x * B;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    copy_piece<B>(to + i * kThreads * B, p + e0 + i * B / (int)sizeof(T), N == 1);
    copy_piece<B>(to + (i + N) * kThreads * B, p + e1 + i * B / (int)sizeof(T), N == 1);
  }
}
template <int P>
__device__ __forceinline__ void get_row(Runs<P>& r, const uint8_t* from, const __nv_bfloat16*) {
  from += threadIdx.x * kPiece<__nv_bfloat16, P>;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t w[P / 2];
    const uint8_t* at = from + k * kThreads * kPiece<__nv_bfloat16, P>;
    if (P == 8) {
      const uint4 x = *reinterpret_cast<const uint4*>(at);
      w[0] = x.x; w[1] = x.y; w[P / 2 - 2] = x.z; w[P / 2 - 1] = x.w;
    } else {
      const uint2 x = *reinterpret_cast<const uint2*>(at);
      w[0] = x.x; w[1] = x.y;
    }
    Run<P>& h = k ? r.v : r.u;
#pragma unroll
    for (int i = 0; i < P / 2; ++i)
      h.p[i] = f2{__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u)};
  }
}
template <int P>
__device__ __forceinline__ void get_row(Runs<P>& r, const uint8_t* from, const float*) {
  from += threadIdx.x * 16;
#pragma unroll
  for (int k = 0; k < P / 2; ++k) {
    const float4 x = *reinterpret_cast<const float4*>(from + k * kThreads * 16);
    Run<P>& h = k < P / 4 ? r.u : r.v;
    h.p[2 * (k % (P / 4))] = f2{x.x, x.y};
    h.p[2 * (k % (P / 4)) + 1] = f2{x.z, x.w};
  }
}
template <int P>
__device__ __forceinline__ void put_run(__nv_bfloat16* p, const Run<P>& h) {
  __nv_bfloat162 t[P / 2];
#pragma unroll
  for (int i = 0; i < P / 2; ++i) t[i] = __floats2bfloat162_rn(h.p[i].x, h.p[i].y);
  if (P == 8) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(t);
  else *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(t);
}
template <int P>
__device__ __forceinline__ void put_run(float* p, const Run<P>& h) {
#pragma unroll
  for (int i = 0; i < P / 4; ++i)
    reinterpret_cast<float4*>(p)[i] = make_float4(h.p[2 * i].x, h.p[2 * i].y, h.p[2 * i + 1].x, h.p[2 * i + 1].y);
}
template <int P>
__device__ __forceinline__ Run<P> shared_run(const float* p) {
  Run<P> h;
#pragma unroll
  for (int i = 0; i < P / 4; ++i) {
    const float4 t = reinterpret_cast<const float4*>(p)[i];
    h.p[2 * i] = f2{t.x, t.y};
    h.p[2 * i + 1] = f2{t.z, t.w};
  }
  return h;
}

template <int P>
__device__ __forceinline__ float dot(const Runs<P>& a, const Runs<P>& b) {
  f2 s = mul2(a.u.p[0], b.u.p[0]), t = mul2(a.v.p[0], b.v.p[0]);
#pragma unroll
  for (int i = 1; i < P / 2; ++i) {
    s = fma2(a.u.p[i], b.u.p[i], s);
    t = fma2(a.v.p[i], b.v.p[i], t);
  }
  return (s.x + t.x) + (s.y + t.y);
}

// Cosines and sines of a chunk's P pairs; a chunk that is not turned has 1 and 0.
template <int P>
struct TurnRuns {
  float cs[P], sn[P];
  // r turned: half layout pairs u[i] with v[i], interleaved neighbours in a run
  template <bool INTERLEAVED, bool INVERSE>
  __device__ __forceinline__ void apply(Runs<P>& r) const {
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      if (INTERLEAVED) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          f2& x = k ? r.v.p[i] : r.u.p[i];
          const float c = cs[P / 2 * k + i], s = INVERSE ? -sn[P / 2 * k + i] : sn[P / 2 * k + i];
          x = f2{fmaf(x.x, c, -x.y * s), fmaf(x.x, s, x.y * c)};
        }
      } else {
        const f2 c = {cs[2 * i], cs[2 * i + 1]}, s = {sn[2 * i], sn[2 * i + 1]};
        const f2 u = r.u.p[i], v = r.v.p[i];
        const f2 uc = mul2(u, c), vc = mul2(v, c);
        if (INVERSE) {
          r.u.p[i] = fma2(v, s, uc);
          r.v.p[i] = f2{fmaf(-u.x, s.x, vc.x), fmaf(-u.y, s.y, vc.y)};
        } else {
          r.u.p[i] = f2{fmaf(-v.x, s.x, uc.x), fmaf(-v.y, s.y, uc.y)};
          r.v.p[i] = fma2(u, s, vc);
        }
      }
    }
  }
};

// Blocks an SM is to hold, bytes of a row of a block's ring, and its rows (four to sixteen
// were no faster than two: what is in flight at 12 to 24 warps is enough then).
template <int OP>
constexpr int kResident = OP == kForward ? 6 : OP == kBackward ? 4 : 3;
template <int OP, typename TI, typename TO, int P>
constexpr int kRingRow = kRowBytes<TI, P> + (OP == kForward ? 0 : kRowBytes<TO, P>) +
                         (OP == kSecond ? kRowBytes<TI, P> : 0);
constexpr int kDeep = 2;

template <int OP, typename TI, typename TO, int P, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, kResident<OP>) norm_rows(const __grid_constant__ NormArgs a) {
  extern __shared__ __align__(16) unsigned long long turns[];
  constexpr int D = kDeep, R = kRingRow<OP, TI, TO, P>;
  uint8_t* const ring = reinterpret_cast<uint8_t*>(turns);  // [D][R]
  unsigned long long* const table = reinterpret_cast<unsigned long long*>(ring + D * R);
  float* const sw = reinterpret_cast<float*>(table + ((a.half + 1) & ~1));
  float* const sc = sw + a.d;
  if (OP != kForward) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // norm_sums
  const bool second_side = blockIdx.x >= (unsigned)a.side[0].blocks;
  const Side& s = a.side[second_side];
  const int block = blockIdx.x - (second_side ? a.side[0].blocks : 0);
  const int lane = threadIdx.x & (a.lanes - 1), group = threadIdx.x / a.lanes;
  const int per_block = kThreads / a.lanes;  // positions of a unit
  const int rot = a.half / P;
  const bool have = lane < a.d / (2 * P), turned = lane < rot;
  const int e0 = turned ? (INTERLEAVED ? 2 * P : P) * lane : 2 * a.half + (lane - rot) * 2 * P;
  const int e1 = turned && !INTERLEAVED ? e0 + a.half : e0 + P;
  const long long items = (long long)a.B * a.N;
  // a unit's first head, the end of its heads, and this thread's row of it, if any
  auto unit_at = [&](long long unit, int& h0, int& h1, int& b, int& n) -> bool {
    const long long ib = s.groups == 1 ? unit : unit / s.groups;
    h0 = (int)(unit - ib * s.groups) * s.heads;
    h1 = min(s.H, h0 + s.heads);
    const long long item = ib * per_block + group;
    const bool active = item < items && have;  // the other lanes only take part in exchanges
    b = active ? (int)(item / a.N) : 0;
    n = active ? (int)(item - (long long)b * a.N) : 0;
    return active;
  };

  // the next row to copy
  long long c_unit = block;
  int c_left = 0, c_slot = 0;
  bool c_active = false;
  const TI *cx = nullptr, *cca = nullptr;
  const TO* cdy = nullptr;
  const uint32_t ring_at = smem_u32(ring);
  auto enter_unit = [&] {
    if (c_unit >= s.units) return;
    int h0, h1, b, n;
    c_active = unit_at(c_unit, h0, h1, b, n);
    c_left = h1 - h0;
    cx = static_cast<const TI*>(s.x) + b * s.xs[0] + n * s.xs[2] + h0 * s.xs[1];
    if (OP != kForward) cdy = static_cast<const TO*>(s.dy) + b * s.dys[0] + n * s.dys[2] + h0 * s.dys[1];
    if (OP == kSecond && s.a) cca = static_cast<const TI*>(s.a) + b * s.as[0] + n * s.as[2] + h0 * s.as[1];
  };
  auto copy_next = [&] {
    if (c_unit < s.units) {
      if (c_active) {
        const uint32_t to = ring_at + c_slot * R;
        copy_row<TI, P>(to, cx, e0, e1);
        if (OP != kForward) copy_row<TO, P>(to + kRowBytes<TI, P>, cdy, e0, e1);
        if (OP == kSecond && s.a) copy_row<TI, P>(to + kRowBytes<TI, P> + kRowBytes<TO, P>, cca, e0, e1);
      }
      cx += s.xs[1];
      if (OP != kForward) cdy += s.dys[1];
      if (OP == kSecond && s.a) cca += s.as[1];
      if (--c_left == 0) {
        c_unit += s.blocks;
        enter_unit();
      }
    }
    c_slot = c_slot + 1 == D ? 0 : c_slot + 1;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  enter_unit();
#pragma unroll 1
  for (int i = 0; i < D; ++i) copy_next();

  turns_table<kThreads>(table, a.inv_freq, a.half);
  for (int i = threadIdx.x; i < a.d; i += kThreads) {
    sw[i] = s.w ? vector_at(s.w, a.w_bf16, i) : 1.f;
    if (OP == kSecond) sc[i] = s.c ? vector_at(s.c, a.w_bf16, i) : 0.f;
  }
  __syncthreads();
  Runs<P> acc;
#pragma unroll
  for (int i = 0; i < P / 2; ++i) acc.u.p[i] = acc.v.p[i] = both(0.f);

  int slot = 0;
  for (long long unit = block; unit < s.units; unit += s.blocks) {
    int h0, h1, b, n;
    const bool active = unit_at(unit, h0, h1, b, n);
    using TY = typename std::conditional<OP == kForward, TO, TI>::type;
    TY* y = static_cast<TY*>(s.y) + b * s.ys[0] + n * s.ys[2] + h0 * s.ys[1];
    TO* ddy = static_cast<TO*>(s.ddy) + b * s.ddys[0] + n * s.ddys[2] + h0 * s.ddys[1];
    TurnRuns<P> t8;
    const long long p = !active ? 0 : a.positions ? a.positions[b * a.pos_sb + n] : a.offset + n;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      float sn = 0.f, cs = 1.f;
      if (turned) {
        sincos_turns((uint32_t)(((unsigned long long)p * table[P * lane + i] + 0x80000000ull) >> 32), sn, cs);
        sn *= a.magnitude;
        cs *= a.magnitude;
      }
      t8.cs[i] = cs;
      t8.sn[i] = sn;
    }
#pragma unroll 1
    for (int head = h0; head < h1; ++head) {
      asm volatile("cp.async.wait_group %0;" ::"n"(D - 1) : "memory");
      const uint8_t* from = ring + slot * R;
      slot = slot + 1 == D ? 0 : slot + 1;
      Runs<P> xv, g, av;
      if (active) {
        get_row(xv, from, static_cast<const TI*>(nullptr));
        if (OP != kForward) get_row(g, from + kRowBytes<TI, P>, static_cast<const TO*>(nullptr));
      } else {
#pragma unroll
        for (int i = 0; i < P / 2; ++i) xv.u.p[i] = xv.v.p[i] = g.u.p[i] = g.v.p[i] = both(0.f);
      }
      if (OP == kSecond) {
        if (active && s.a) {
          get_row(av, from + kRowBytes<TI, P> + kRowBytes<TO, P>, static_cast<const TI*>(nullptr));
        } else {
#pragma unroll
          for (int i = 0; i < P / 2; ++i) av.u.p[i] = av.v.p[i] = both(0.f);
        }
      }
      copy_next();  // into the slot that was just read
      {
        if (OP == kForward) {
          float sum[1] = {dot(xv, xv)};
          row_sums(sum, a.lanes);
          const f2 r = both(rsqrtf(fmaf(sum[0], a.inv_d, a.eps)));
          if (!active) continue;
          const Run<P> wu = shared_run<P>(sw + e0), wv = shared_run<P>(sw + e1);
#pragma unroll
          for (int i = 0; i < P / 2; ++i) {
            xv.u.p[i] = mul2(mul2(r, wu.p[i]), xv.u.p[i]);
            xv.v.p[i] = mul2(mul2(r, wv.p[i]), xv.v.p[i]);
          }
          t8.template apply<INTERLEAVED, false>(xv);
          put_run<P>(y + e0, xv.u);
          put_run<P>(y + e1, xv.v);
          y += s.ys[1];
        } else if (OP == kBackward) {
          t8.template apply<INTERLEAVED, true>(g);
          Runs<P> h;
          if (have) {
            const Run<P> wu = shared_run<P>(sw + e0), wv = shared_run<P>(sw + e1);
#pragma unroll
            for (int i = 0; i < P / 2; ++i) {
              h.u.p[i] = mul2(wu.p[i], g.u.p[i]);
              h.v.p[i] = mul2(wv.p[i], g.v.p[i]);
            }
          } else {
            h = g;
          }
          float sum[2] = {dot(xv, xv), dot(h, xv)};
          row_sums(sum, a.lanes);
          if (!active) continue;
          const float r = rsqrtf(fmaf(sum[0], a.inv_d, a.eps));
          // dx = r h - (r^3 <h, x> / d) x
          const f2 r2 = both(r), back = both(-r * (r * r * sum[1] * a.inv_d));
#pragma unroll
          for (int i = 0; i < P / 2; ++i) {
            acc.u.p[i] = fma2(g.u.p[i], mul2(r2, xv.u.p[i]), acc.u.p[i]);
            acc.v.p[i] = fma2(g.v.p[i], mul2(r2, xv.v.p[i]), acc.v.p[i]);
            xv.u.p[i] = fma2(r2, h.u.p[i], mul2(back, xv.u.p[i]));
            xv.v.p[i] = fma2(r2, h.v.p[i], mul2(back, xv.v.p[i]));
          }
          put_run<P>(y + e0, xv.u);
          put_run<P>(y + e1, xv.v);
          y += s.ys[1];
        } else {
          t8.template apply<INTERLEAVED, true>(g);
          // <x, x>, <h, x>, <a, x>, <h, a>, <c . g, x>
          float sum[5] = {dot(xv, xv), 0.f, dot(av, xv), 0.f, 0.f};
          if (have) {
            f2 hx = both(0.f), ha = both(0.f), cx = both(0.f);
#pragma unroll
            for (int run = 0; run < 2; ++run) {
              const Run<P> w = shared_run<P>(sw + (run ? e1 : e0)), c = shared_run<P>(sc + (run ? e1 : e0));
              const Run<P> &gr = run ? g.v : g.u, &xr = run ? xv.v : xv.u, &ar = run ? av.v : av.u;
#pragma unroll
              for (int i = 0; i < P / 2; ++i) {
                const f2 h = mul2(w.p[i], gr.p[i]);
                hx = fma2(h, xr.p[i], hx);
                ha = fma2(h, ar.p[i], ha);
                cx = fma2(mul2(c.p[i], gr.p[i]), xr.p[i], cx);
              }
            }
            sum[1] = hx.x + hx.y;
            sum[3] = ha.x + ha.y;
            sum[4] = cx.x + cx.y;
          }
          row_sums(sum, a.lanes);
          if (!active) continue;
          const float r = rsqrtf(fmaf(sum[0], a.inv_d, a.eps));
          const float hn = r * sum[1] * a.inv_d, an = r * sum[2] * a.inv_d;  // <h, n> / d, <a, n> / d
          const float ht = r * (sum[3] - r * sum[1] * an);                   // <h, t>
          const float un = r * a.inv_d * sum[4] - 2.f * r * an * hn;         // <u, n> / d
          // gx = r (c . g - r (an h + hn a) - back x),  t = r (a - an r x)
          const f2 r2 = both(r), by_h = both(-r * an), by_a = both(-r * (r * hn)),
                   by_x = both(-r * (r * (un + ht * a.inv_d))), at = both(-r * (an * r));
#pragma unroll
          for (int run = 0; run < 2; ++run) {
            const Run<P> w = shared_run<P>(sw + (run ? e1 : e0)), c = shared_run<P>(sc + (run ? e1 : e0));
            Run<P> &gr = run ? g.v : g.u, &xr = run ? xv.v : xv.u, &ac = run ? acc.v : acc.u;
            const Run<P>& ar = run ? av.v : av.u;
#pragma unroll
            for (int i = 0; i < P / 2; ++i) {
              const f2 t = fma2(r2, ar.p[i], mul2(at, xr.p[i]));
              ac.p[i] = fma2(gr.p[i], t, ac.p[i]);
              const f2 q = mul2(r2, fma2(by_h, w.p[i], c.p[i]));  // what multiplies g in gx
              const f2 out = fma2(w.p[i], t, mul2(c.p[i], mul2(r2, xr.p[i])));
              xr.p[i] = fma2(q, gr.p[i], fma2(by_a, ar.p[i], mul2(by_x, xr.p[i])));
              gr.p[i] = out;
            }
          }
          t8.template apply<INTERLEAVED, false>(g);
          put_run<P>(y + e0, xv.u);
          put_run<P>(y + e1, xv.v);
          put_run<P>(ddy + e0, g.u);
          put_run<P>(ddy + e1, g.v);
          y += s.ys[1];
          ddy += s.ddys[1];
        }
      }
    }
  }
  if (OP == kForward || !s.sums) return;
  __syncthreads();  // every thread is past its last row
  float* const red = reinterpret_cast<float*>(ring);  // [per_block][d]: 8 KB at most
  if (have) {
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      *reinterpret_cast<f2*>(red + group * a.d + e0 + 2 * i) = acc.u.p[i];
      *reinterpret_cast<f2*>(red + group * a.d + e1 + 2 * i) = acc.v.p[i];
    }
  }
  block_partial(red, a, second_side, block, per_block);
}

// dw[i] = sum over the blocks' partial sums: 32 features and 32 parts of the blocks
// to a thread block.
struct SumArgs {
  void* out[2];
  int first[2], blocks[2];
  const float* partial;
  int d, bf16;
};
__global__ void __launch_bounds__(1024) norm_sums(SumArgs a) {
  __shared__ float sm[32][33];
  const int t = blockIdx.y, f = blockIdx.x * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched while the rows' kernel ends
  float s = 0.f;
  if (f < a.d) {
#pragma unroll 8
    for (int b = part; b < a.blocks[t]; b += 32) s += a.partial[((size_t)a.first[t] + b) * a.d + f];
  }
  sm[part][threadIdx.x & 31] = s;
  __syncthreads();
  s = warp_sum(sm[threadIdx.x & 31][part]);
  const int g = blockIdx.x * 32 + part;
  if ((threadIdx.x & 31) == 0 && g < a.d && a.out[t]) {
    if (a.bf16) static_cast<__nv_bfloat16*>(a.out[t])[g] = __float2bfloat16_rn(s);
    else static_cast<float*>(a.out[t])[g] = s;
  }
}

// Blocks per SM of norm_kernel, and as many or more of norm_rows with sums.
constexpr int kBlocksPerSm = 6;

// Lanes of a row, heads of a unit and blocks of each tensor.  A unit takes as
// many heads (up to 16) as leave half a wave of threads, so that few sines are
// computed; one where the call is small and latency counts.  Blocks stay and take units in
// turn, so that the table of angles is made, and sums are carried, a few times an SM.
void plan(NormArgs& a, int P, int C, int per_sm) {
  const int chunks = a.d / (2 * P) + (P == 1 ? (a.d & 1) : 0);
  int lanes = 1;
  while (lanes < 32 && lanes < (chunks + C - 1) / C) lanes *= 2;
  a.lanes = lanes;
  const long long blocks = ((long long)a.B * a.N * lanes + kThreads - 1) / kThreads;
  int heads = 16;
  long long units = 0;
  for (;; heads /= 2) {
    units = 0;
    for (Side& s : a.side) {
      s.heads = heads;
      s.groups = (s.H + heads - 1) / heads;
      s.units = blocks * s.groups;
      units += s.units;
    }
    if (heads == 1 || units * kThreads >= kSms * 1024ll) break;
  }
  // blocks in proportion to the rows of each tensor
  const long long most = kSms * per_sm, rows = a.side[0].H + a.side[1].H;
  for (Side& s : a.side) {
    const long long n = units > most ? most * s.H / rows : s.units;
    s.blocks = (int)(n < s.units ? (n > 0 ? n : 1) : s.units);
  }
}

// norm_rows, or norm_kernel where P = 1.
template <int OP, typename TI, typename TO, int P, int C, bool INTERLEAVED>
cudaError_t launch(NormArgs& a, LaunchLog& log) {
  plan(a, P, C, P > 1 ? kResident<OP> : kBlocksPerSm);
  size_t smem = sizeof(unsigned long long) * ((a.half + 1) & ~1) + sizeof(float) * a.d * (OP == kSecond ? 2 : 1);
  const unsigned grid = (unsigned)(a.side[0].blocks + a.side[1].blocks);
  if constexpr (P > 1) {
    // (the limit belongs to the kernel, which another thread may be about to launch: it is always
    // set to the most that a call takes, kMaxDim features, all turned)
    constexpr size_t ring = kDeep * kRingRow<OP, TI, TO, P>;
    constexpr size_t most = ring + sizeof(unsigned long long) * (kMaxDim / 2) + sizeof(float) * kMaxDim * 2;
    smem += ring;
    const cudaError_t e = cudaFuncSetAttribute(norm_rows<OP, TI, TO, P, INTERLEAVED>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (e != cudaSuccess) return e;
    norm_rows<OP, TI, TO, P, INTERLEAVED><<<grid, kThreads, smem, log.stream>>>(a);
  } else {
    smem += OP == kForward ? 0 : sizeof(float) * a.d * (kThreads / a.lanes);
    norm_kernel<OP, TI, TO, P, C, INTERLEAVED><<<grid, kThreads, smem, log.stream>>>(a);
  }
  const cudaError_t e = cudaGetLastError();
  log.mark();
  return e;
}

template <typename T>
bool aligned_rows(const void* p, const long long (&st)[3], int P) {
  const long long bytes = P * (long long)sizeof(T) < 16 ? P * (long long)sizeof(T) : 16;
  if (!p) return true;
  bool ok = reinterpret_cast<uintptr_t>(p) % bytes == 0;
  for (long long x : st) ok = ok && x * (long long)sizeof(T) % bytes == 0;
  return ok;
}

// Whether chunks of P pairs tile the turned and the other part, and every access is
// aligned (16 bytes, or all P elements where they are fewer).  32 lanes hold a row of
// kMaxDim features at P = 4.
template <int OP, typename TI, typename TO, int P>
bool chunked(const NormArgs& a) {
  bool ok = a.half % P == 0 && (a.d - 2 * a.half) % (2 * P) == 0;
  for (const Side& s : a.side) {
    if (!s.H) continue;
    ok = ok && aligned_rows<TI>(s.x, s.xs, P);
    ok = ok && (OP == kForward ? aligned_rows<TO>(s.y, s.ys, P) : aligned_rows<TI>(s.y, s.ys, P));
    if (OP != kForward) ok = ok && aligned_rows<TO>(s.dy, s.dys, P);
    if (OP == kSecond)
      ok = ok && aligned_rows<TI>(s.a, s.as, P) && aligned_rows<TO>(s.ddy, s.ddys, P);
  }
  return ok;
}

template <int OP, typename TI, typename TO, bool IL>
cudaError_t dispatch(NormArgs& a, LaunchLog& log) {
  if (chunked<OP, TI, TO, 8>(a)) return launch<OP, TI, TO, 8, 1, IL>(a, log);
  if (chunked<OP, TI, TO, 4>(a)) return launch<OP, TI, TO, 4, 1, IL>(a, log);
  return launch<OP, TI, TO, 1, 4, IL>(a, log);
}

template <int OP>
cudaError_t dispatch(NormArgs& a, bool bi, bool bo, bool il, LaunchLog& log) {
  using H = __nv_bfloat16;
  if (bi && bo) return il ? dispatch<OP, H, H, true>(a, log) : dispatch<OP, H, H, false>(a, log);
  if (bi) return il ? dispatch<OP, H, float, true>(a, log) : dispatch<OP, H, float, false>(a, log);
  if (bo) return il ? dispatch<OP, float, H, true>(a, log) : dispatch<OP, float, H, false>(a, log);
  return il ? dispatch<OP, float, float, true>(a, log) : dispatch<OP, float, float, false>(a, log);
}

size_t workspace_bytes(const fbob_qk_norm_t* s) {
  return ((size_t)kSms * kBlocksPerSm + 2) * s->d * sizeof(float);
}

bool off(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

int check(const fbob_qk_norm_t* s) {
  if (!s) return FBOB_ERR_INVALID_ARG;
  if (s->B < 1 || s->N < 1 || s->d < 1 || s->rotary_dim < 0 || s->rotary_dim > s->d ||
      (s->rotary_dim & 1) || (s->interleaved & ~1))
    return FBOB_ERR_INVALID_ARG;
  if (!(s->eps >= 0.f) || !(s->magnitude == s->magnitude)) return FBOB_ERR_INVALID_ARG;
  for (int dt : {s->in_dtype, s->out_dtype, s->weight_dtype})
    if (dt != FBOB_BF16 && dt != FBOB_FP32) return FBOB_ERR_UNSUPPORTED;
  return s->d > kMaxDim ? FBOB_ERR_UNSUPPORTED : FBOB_OK;
}

int call(int op, const fbob_qk_norm_t* s, const fbob_norm_side_t* q, const fbob_norm_side_t* k,
         const double* inv_freq, const long long* positions, void* ws, size_t ws_bytes, void* stream) {
  const int st = check(s);
  if (st != FBOB_OK) return st;
  if (!q || (s->rotary_dim > 0 && !inv_freq) || off(inv_freq, 8) || off(positions, 8))
    return FBOB_ERR_INVALID_ARG;
  const size_t si = s->in_dtype == FBOB_BF16 ? 2 : 4, so = s->out_dtype == FBOB_BF16 ? 2 : 4;
  const size_t sw = s->weight_dtype == FBOB_BF16 ? 2 : 4;
  NormArgs a = {};
  double heads = 0;
  bool sums = false;
  for (int i = 0; i < 2; ++i) {
    const fbob_norm_side_t* f = i ? k : q;
    if (!f) continue;
    Side& t = a.side[i];
    if (f->H < 1 || !f->x || !f->y) return FBOB_ERR_INVALID_ARG;
    if (off(f->x, si) || off(f->y, op == kForward ? so : si) || off(f->weight, sw))
      return FBOB_ERR_INVALID_ARG;
    if (op != kForward && (!f->dy || off(f->dy, so) || off(f->dweight, sw))) return FBOB_ERR_INVALID_ARG;
    if (op == kSecond && (!f->ddy || off(f->ddy, so) || off(f->a, si) || off(f->c, sw)))
      return FBOB_ERR_INVALID_ARG;
    t.H = f->H;
    t.x = f->x; t.w = f->weight; t.y = f->y;
    if (op != kForward) {
      t.dy = f->dy;
      t.sums = f->dweight != nullptr;
    }
    if (op == kSecond) {
      t.a = f->a; t.c = f->c; t.ddy = f->ddy;
    }
    for (int j = 0; j < 3; ++j) {
      t.xs[j] = f->x_strides[j];
      t.dys[j] = f->dy_strides[j];
      t.as[j] = f->a_strides[j];
      t.ys[j] = f->y_strides[j];
      t.ddys[j] = f->ddy_strides[j];
    }
    heads += f->H;
    sums = sums || t.sums;
  }
  if (heads > 65535.0 || heads * s->B * s->N * s->d > (double)(1ll << 38)) return FBOB_ERR_UNSUPPORTED;
  if (sums) {
    if (!ws || off(ws, 16)) return FBOB_ERR_INVALID_ARG;
    if (ws_bytes < workspace_bytes(s)) return FBOB_ERR_WORKSPACE;
  }
  a.inv_freq = inv_freq;
  a.positions = positions;
  a.pos_sb = s->pos_stride;
  a.offset = s->offset;
  a.partial = static_cast<float*>(ws);
  a.B = s->B; a.N = s->N; a.d = s->d;
  a.half = s->rotary_dim / 2;
  a.w_bf16 = s->weight_dtype == FBOB_BF16;
  a.eps = s->eps;
  a.inv_d = 1.f / (float)s->d;
  a.magnitude = s->magnitude;
  LaunchLog log{static_cast<cudaStream_t>(stream)};
  begin_call(log);
  const bool bi = s->in_dtype == FBOB_BF16, bo = s->out_dtype == FBOB_BF16, il = s->interleaved != 0;
  cudaError_t e = op == kForward    ? dispatch<kForward>(a, bi, bo, il, log)
                  : op == kBackward ? dispatch<kBackward>(a, bi, bo, il, log)
                                    : dispatch<kSecond>(a, bi, bo, il, log);
  if (e == cudaSuccess && sums) {
    SumArgs r = {};
    int first = 0;
    for (int i = 0; i < 2; ++i) {
      r.out[i] = a.side[i].sums ? (i ? k : q)->dweight : nullptr;
      r.first[i] = first;
      r.blocks[i] = a.side[i].sums ? a.side[i].blocks : 0;
      first += r.blocks[i];
    }
    r.partial = a.partial;
    r.d = a.d;
    r.bf16 = a.w_bf16;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3((unsigned)(a.d + 31) / 32, 2);
    c.blockDim = dim3(1024);
    c.stream = log.stream;
    cudaLaunchAttribute early;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    c.attrs = &early;
    c.numAttrs = 1;
    e = cudaLaunchKernelEx(&c, norm_sums, r);
    log.mark();
  }
  end_call(log);
  return e == cudaSuccess ? FBOB_OK : FBOB_ERR_CUDA;
}

}  // namespace
}  // namespace fbob

using namespace fbob;

extern "C" {

size_t fbob_qk_norm_workspace_size(const fbob_qk_norm_t* s) {
  return check(s) == FBOB_OK ? workspace_bytes(s) : 0;
}

int fbob_qk_norm_forward(const fbob_qk_norm_t* s, const fbob_norm_side_t* q, const fbob_norm_side_t* k,
                         const double* inv_freq, const long long* positions, void* stream) {
  return call(kForward, s, q, k, inv_freq, positions, nullptr, 0, stream);
}

int fbob_qk_norm_backward(const fbob_qk_norm_t* s, const fbob_norm_side_t* q, const fbob_norm_side_t* k,
                          const double* inv_freq, const long long* positions, void* ws,
                          size_t ws_bytes, void* stream) {
  return call(kBackward, s, q, k, inv_freq, positions, ws, ws_bytes, stream);
}

int fbob_qk_norm_bob(const fbob_qk_norm_t* s, const fbob_norm_side_t* q, const fbob_norm_side_t* k,
                     const double* inv_freq, const long long* positions, void* ws, size_t ws_bytes,
                     void* stream) {
  return call(kSecond, s, q, k, inv_freq, positions, ws, ws_bytes, stream);
}

}  // extern "C"
