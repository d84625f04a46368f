// Rotary positions: the pair (a, b) of features i of a row at position p turns
// by the angle p f_i,
//   a' = m (a cos(p f_i) - b sin(p f_i)),  b' = m (a sin(p f_i) + b cos(p f_i)),
// and the features past rotary_dim are copied.  The map is linear, so its
// backward is the same call with the angle negated (inverse), and so is the
// backward of that.
//
// Angles.  Only p f_i mod one turn matters, and far positions (p f_i of 10^5
// radians and more) lose it in 32-bit floating point.  f_i / 2 pi is taken
// from the fp64 frequency to a 64-bit fixed-point fraction of a turn (its
// product with 1 / 2 pi in two doubles); the 64-bit integer product with p
// then wraps exactly where whole turns drop out.  The error is p 2^-63
// turns.  The top 32 bits give sine and cosine.
//
// Bound: memory (x read once, y written once; positions and frequencies are a
// few KB that stay in cache).  A thread owns a chunk of pairs of one
// position and walks over a group of heads, so a sine and cosine (about 30
// instructions) serve several heads, with 16-byte accesses where the strides
// allow.  Measured: forward and backward at 8 heads x 65536 x 128, bf16, 89 us,
// 6.05 TB/s (89% of the measured copy rate); 2 x 16 heads x 4096 x 128, fp32 to
// bf16, 40 us; one token of 8 x 16 heads 2.6 us, its launch.  Slower: blocks that
// walk over several chunks, 64 or 256 threads, more heads in flight.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"
#include "ops.h"

namespace fbob {
namespace {

constexpr int kThreads = 128;

struct RotaryArgs {
  const void* x;
  void* y;
  const double* inv_freq;
  const long long* positions;  // null: offset + n
  long long pos_sb, offset;
  long long xs[3], ys[3];  // strides over batch, head, position, in elements
  int B, H, N, d, half;    // half = rotary_dim / 2 pairs
  int heads;               // heads per thread
  float magnitude, sign;   // sign of the angle
};

template <typename T, int P>
struct Vec;
template <>
struct Vec<__nv_bfloat16, 8> {
  uint4 v;
  __device__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = v; }
  __device__ void get(float (&f)[8]) const {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = __bfloat1622float2(h[i]);
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
  __device__ void set(const float (&f)[8]) {
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  }
};
template <>
struct Vec<__nv_bfloat16, 4> {
  uint2 v;
  __device__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint2*>(p); }
  __device__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint2*>(p) = v; }
  __device__ void get(float (&f)[4]) const {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 t = __bfloat1622float2(h[i]);
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
  __device__ void set(const float (&f)[4]) {
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
    for (int i = 0; i < 2; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  }
};
template <>
struct Vec<float, 4> {
  float4 v;
  __device__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
  __device__ void store(float* p) const { *reinterpret_cast<float4*>(p) = v; }
  __device__ void get(float (&f)[4]) const { f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w; }
  __device__ void set(const float (&f)[4]) { v = make_float4(f[0], f[1], f[2], f[3]); }
};
template <>
struct Vec<float, 8> {
  float4 v[2];
  __device__ void load(const float* p) {
    v[0] = reinterpret_cast<const float4*>(p)[0];
    v[1] = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = v[0];
    reinterpret_cast<float4*>(p)[1] = v[1];
  }
  __device__ void get(float (&f)[8]) const {
    f[0] = v[0].x; f[1] = v[0].y; f[2] = v[0].z; f[3] = v[0].w;
    f[4] = v[1].x; f[5] = v[1].y; f[6] = v[1].z; f[7] = v[1].w;
  }
  __device__ void set(const float (&f)[8]) {
    v[0] = make_float4(f[0], f[1], f[2], f[3]);
    v[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
};
template <typename T>
struct Vec<T, 1> {
  T v;
  __device__ void load(const T* p) { v = *p; }
  __device__ void store(T* p) const { *p = v; }
  __device__ void get(float (&f)[1]) const { f[0] = to_f32<T>(v); }
  __device__ void set(const float (&f)[1]) { v = from_f32<T>(f[0]); }
};

// Turns a chunk of P pairs held as two runs of P elements: the pairs' first
// and second members (half layout), or its first and last P elements with
// the pairs side by side (interleaved).
template <int P, bool INTERLEAVED>
__device__ __forceinline__ void turn(float (&u)[P], float (&w)[P], const float (&cs)[P],
                                     const float (&sn)[P]) {
  if constexpr (INTERLEAVED && P > 1) {
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      const float ua = u[2 * i], ub = u[2 * i + 1], wa = w[2 * i], wb = w[2 * i + 1];
      u[2 * i] = ua * cs[i] - ub * sn[i];
      u[2 * i + 1] = ua * sn[i] + ub * cs[i];
      w[2 * i] = wa * cs[P / 2 + i] - wb * sn[P / 2 + i];
      w[2 * i + 1] = wa * sn[P / 2 + i] + wb * cs[P / 2 + i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const float a = u[i], b = w[i];
      u[i] = a * cs[i] - b * sn[i];
      w[i] = a * sn[i] + b * cs[i];
    }
  }
}

// Sine and cosine of hi 2^-32 turns: the nearest quarter turn is taken off (two
// bits), and the rest, |x| <= pi / 4, goes into the Taylor series up to x^9 and
// x^10, whose next terms are below 2e-9 x and 2e-10.
__device__ __forceinline__ void sincos_turns(uint32_t hi, float& s, float& c) {
  const uint32_t q = (hi + 0x20000000u) >> 30;
  const float x = (float)(int)(hi - (q << 30)) * 1.4629180792671596e-9f;  // 2 pi 2^-32
  const float y = x * x;
  float a = fmaf(y, 1.f / 362880.f, -1.f / 5040.f);
  a = fmaf(a, y, 1.f / 120.f);
  a = fmaf(a, y, -1.f / 6.f);
  a = fmaf(a * y, x, x);
  float b = fmaf(y, -1.f / 3628800.f, 1.f / 40320.f);
  b = fmaf(b, y, -1.f / 720.f);
  b = fmaf(b, y, 1.f / 24.f);
  b = fmaf(b, y, -0.5f);
  b = fmaf(b, y, 1.f);
  const bool odd = q & 1u;
  s = odd ? b : a;
  c = odd ? a : b;
  if (q & 2u) s = -s;
  if ((q + 1u) & 2u) c = -c;
}

// Heads whose loads are in flight together.
template <typename TI, typename TO>
constexpr int kHeads = (sizeof(TI) == 2 && sizeof(TO) == 2) ? 4 : 2;

template <typename TI, typename TO, int P, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rotary_kernel(RotaryArgs a) {
  extern __shared__ unsigned long long turns[];  // [half]: 2^64 f / 2 pi mod 2^64
  constexpr int U = kHeads<TI, TO>;
  const int chunks = a.d / (2 * P) + (P == 1 ? (a.d & 1) : 0);
  const int rot_chunks = a.half / P;
  const long long items = (long long)a.B * a.N * chunks;
  const int h0 = blockIdx.y * a.heads, h1 = min(a.H, h0 + a.heads);
  const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
  const bool active = id < items;
  int c = 0, n = 0, b = 0;
  if (active) {
    if (items <= 0xffffffffll) {  // 32-bit divisions where they do
      const unsigned bn = (unsigned)id / (unsigned)chunks;
      c = (int)((unsigned)id - bn * (unsigned)chunks);
      b = (int)(bn / (unsigned)a.N);
      n = (int)(bn - (unsigned)b * (unsigned)a.N);
    } else {
      const long long bn = id / chunks;
      c = (int)(id - bn * chunks);
      b = (int)(bn / a.N);
      n = (int)(bn - (long long)b * a.N);
    }
  }
  const bool turned = active && c < rot_chunks;
  // offsets of the chunk's two halves of P elements
  int e0, e1;
  bool two = active;  // not for an odd width's last feature: one element
  if (c < rot_chunks) {
    e0 = INTERLEAVED ? 2 * P * c : P * c;
    e1 = INTERLEAVED ? e0 + P : e0 + a.half;
  } else {
    e0 = 2 * a.half + (c - rot_chunks) * 2 * P;
    e1 = e0 + P;
    two = two && e1 < a.d;
  }
  const TI* __restrict__ x = static_cast<const TI*>(a.x) + b * a.xs[0] + n * a.xs[2];
  TO* __restrict__ y = static_cast<TO*>(a.y) + b * a.ys[0] + n * a.ys[2];
  Vec<TI, P> u[U], w[U];
  auto load = [&](int hb) {
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (active && hb + i < h1) {
        const TI* xp = x + (hb + i) * a.xs[1];
        u[i].load(xp + e0);
        if (two) w[i].load(xp + e1);
      }
  };
  // the first heads and the position are on their way while the block makes
  // its table of frequencies
  load(h0);
  const long long p = !turned ? 0 : a.positions ? a.positions[b * a.pos_sb + n] : a.offset + n;
  for (int i = threadIdx.x; i < a.half; i += kThreads) {
    // 1 / (2 pi) as a sum of two doubles: the product keeps about 100 bits
    const double f = a.inv_freq[i], c1 = 0.15915494309189535, c2 = -9.839338337591243e-18;
    const double hi = f * c1;
    const double lo = fma(f, c1, -hi) + f * c2;
    const double r = hi - rint(hi);  // exact
    // both parts in units of 2^-64 turns; |r| <= 1/2, and 2^64 r is taken
    // as twice 2^63 r (an integer below 2^53 times a power of two)
    const double r63 = r * 9223372036854775808.0, whole = rint(r63);
    const double rest = 2.0 * (r63 - whole) + lo * 18446744073709551616.0;
    turns[i] = ((unsigned long long)(long long)whole << 1) + (unsigned long long)(long long)rint(rest);
  }
  __syncthreads();
  float cs[P], sn[P];
  if (turned) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const unsigned long long t = (unsigned long long)p * turns[c * P + i];
      float s, co;
      sincos_turns((uint32_t)((t + 0x80000000ull) >> 32), s, co);
      cs[i] = co * a.magnitude;
      sn[i] = s * a.magnitude * a.sign;
    }
  }
  for (int hb = h0; hb < h1; hb += U) {
    if (hb > h0) load(hb);
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (active && hb + i < h1) {
        float fu[P], fw[P];
        u[i].get(fu);
        if (two) w[i].get(fw);
        if (turned) turn<P, INTERLEAVED>(fu, fw, cs, sn);
        TO* yp = y + (hb + i) * a.ys[1];
        Vec<TO, P> r;
        r.set(fu);
        r.store(yp + e0);
        if (two) {
          r.set(fw);
          r.store(yp + e1);
        }
      }
  }
}

template <typename TI, typename TO, int P, bool INTERLEAVED>
cudaError_t launch(RotaryArgs a, LaunchLog& log) {
  const long long items = (long long)a.B * a.N * (a.d / (2 * P) + (P == 1 ? (a.d & 1) : 0));
  // heads per thread: as many as leave half a wave of threads, so that
  // few sines are computed; one where the call is small and latency counts
  a.heads = 16;
  while (a.heads > 1 && items * ((a.H + a.heads - 1) / a.heads) < kSms * 1024ll) a.heads /= 2;
  const int groups = (a.H + a.heads - 1) / a.heads;
  dim3 grid((unsigned)((items + kThreads - 1) / kThreads), (unsigned)groups);
  rotary_kernel<TI, TO, P, INTERLEAVED>
      <<<grid, kThreads, sizeof(unsigned long long) * a.half, log.stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  log.mark();
  return e;
}

// Whether chunks of P pairs tile the turned and the copied part and every
// access is aligned (16 bytes, or all P elements where they are fewer).
template <typename TI, typename TO, int P>
bool chunked(const RotaryArgs& a) {
  constexpr size_t ai = P * sizeof(TI) < 16 ? P * sizeof(TI) : 16;
  constexpr size_t ao = P * sizeof(TO) < 16 ? P * sizeof(TO) : 16;
  bool ok = a.half % P == 0 && (a.d - 2 * a.half) % (2 * P) == 0 &&
            reinterpret_cast<uintptr_t>(a.x) % ai == 0 && reinterpret_cast<uintptr_t>(a.y) % ao == 0;
  for (int i = 0; i < 3; ++i)
    ok = ok && a.xs[i] * (long long)sizeof(TI) % (long long)ai == 0 &&
         a.ys[i] * (long long)sizeof(TO) % (long long)ao == 0;
  return ok;
}

template <typename TI, typename TO, bool INTERLEAVED>
cudaError_t dispatch(const RotaryArgs& a, LaunchLog& log) {
  if (chunked<TI, TO, 8>(a)) return launch<TI, TO, 8, INTERLEAVED>(a, log);
  if (chunked<TI, TO, 4>(a)) return launch<TI, TO, 4, INTERLEAVED>(a, log);
  return launch<TI, TO, 1, INTERLEAVED>(a, log);
}

template <typename TI, typename TO>
cudaError_t dispatch(const RotaryArgs& a, bool interleaved, LaunchLog& log) {
  return interleaved ? dispatch<TI, TO, true>(a, log) : dispatch<TI, TO, false>(a, log);
}

}  // namespace
}  // namespace fbob

using namespace fbob;

extern "C" int fbob_rotary(const fbob_rotary_t* r, const void* x, const double* inv_freq,
                           const long long* positions, void* y, void* stream) {
  if (!r || !x || !y || (r->rotary_dim > 0 && !inv_freq)) return FBOB_ERR_INVALID_ARG;
  if (r->B < 1 || r->H < 1 || r->N < 1 || r->d < 1 || r->rotary_dim < 0 || r->rotary_dim > r->d ||
      (r->rotary_dim & 1) || (r->interleaved & ~1) || (r->inverse & ~1))
    return FBOB_ERR_INVALID_ARG;
  if (!(r->magnitude == r->magnitude)) return FBOB_ERR_INVALID_ARG;
  for (int dt : {r->in_dtype, r->out_dtype})
    if (dt != FBOB_BF16 && dt != FBOB_FP32) return FBOB_ERR_UNSUPPORTED;
  if (r->d > 1024 || r->H > 65535) return FBOB_ERR_UNSUPPORTED;
  if ((double)r->B * r->H * r->N * r->d > (double)(1ll << 38)) return FBOB_ERR_UNSUPPORTED;
  const size_t si = r->in_dtype == FBOB_BF16 ? 2 : 4, so = r->out_dtype == FBOB_BF16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(x) % si || reinterpret_cast<uintptr_t>(y) % so ||
      reinterpret_cast<uintptr_t>(inv_freq) % 8 || reinterpret_cast<uintptr_t>(positions) % 8)
    return FBOB_ERR_INVALID_ARG;
  RotaryArgs a;
  a.x = x;
  a.y = y;
  a.inv_freq = inv_freq;
  a.positions = positions;
  a.pos_sb = r->pos_stride;
  a.offset = r->offset;
  for (int i = 0; i < 3; ++i) {
    a.xs[i] = r->x_strides[i];
    a.ys[i] = r->y_strides[i];
  }
  a.B = r->B; a.H = r->H; a.N = r->N; a.d = r->d;
  a.half = r->rotary_dim / 2;
  a.heads = 1;
  a.magnitude = r->magnitude;
  a.sign = r->inverse ? -1.f : 1.f;
  LaunchLog log{static_cast<cudaStream_t>(stream)};
  begin_call(log);
  const bool il = r->interleaved != 0, bi = r->in_dtype == FBOB_BF16, bo = r->out_dtype == FBOB_BF16;
  const cudaError_t e = bi ? (bo ? dispatch<__nv_bfloat16, __nv_bfloat16>(a, il, log)
                                 : dispatch<__nv_bfloat16, float>(a, il, log))
                           : (bo ? dispatch<float, __nv_bfloat16>(a, il, log)
                                 : dispatch<float, float>(a, il, log));
  end_call(log);
  return e == cudaSuccess ? FBOB_OK : FBOB_ERR_CUDA;
}
