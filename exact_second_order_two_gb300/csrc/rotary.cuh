// Pieces shared by the kernels that turn feature pairs by position: vectors of
// features, sine and cosine of a fixed-point angle, and the table of angles.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace fbob {
namespace rope {

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

// 2^64 f / 2 pi mod 2^64 of each of `half` frequencies: what a step of one
// position adds to a pair's angle.  Written by the block's THREADS threads.
template <int THREADS>
__device__ __forceinline__ void turns_table(unsigned long long* turns, const double* inv_freq,
                                            int half) {
  for (int i = threadIdx.x; i < half; i += THREADS) {
    // 1 / (2 pi) as a sum of two doubles: the product keeps about 100 bits
    const double f = inv_freq[i], c1 = 0.15915494309189535, c2 = -9.839338337591243e-18;
    const double hi = f * c1;
    const double lo = fma(f, c1, -hi) + f * c2;
    const double r = hi - rint(hi);  // exact
    // both parts in units of 2^-64 turns; |r| <= 1/2, and 2^64 r is taken
    // as twice 2^63 r (an integer below 2^53 times a power of two)
    const double r63 = r * 9223372036854775808.0, whole = rint(r63);
    const double rest = 2.0 * (r63 - whole) + lo * 18446744073709551616.0;
    turns[i] = ((unsigned long long)(long long)whole << 1) + (unsigned long long)(long long)rint(rest);
  }
}

}  // namespace rope
}  // namespace fbob
