// Tiles of 128 rows x 64 fp16 columns in shared memory (128-byte swizzle) as the
// orthogonalisation's kernels finish them: a thread holds a row.
#pragma once

#include <cuda_fp16.h>

#include "orth.h"
#include "sm103.cuh"
#include "tc_common.cuh"

namespace fbob {
namespace orth {

using namespace tc;

constexpr uint32_t kTileBytes = kTile * kDepth * 2;

// Instruction descriptor: fp16 operands (formats 0), fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

// 32 columns (half h) of a thread's row in a tile: 16-byte chunks 4 h .. 4 h + 3.
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
}  // namespace orth
}  // namespace fbob
