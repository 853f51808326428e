// Device helpers of the tensor-core sliding-window kernels: visibility masks
// and 2^x on the FMA pipe.
#pragma once

#include "common.cuh"
#include "tc.cuh"
#include "window.h"

namespace dash {

// Waits for phase `phase` of a barrier (counted from 0); the answer is the
// same for the whole warp.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, int phase) {
  return __all_sync(0xffffffffu, tc::mbar_wait(bar, phase & 1));
}

// Bits [a, b] of a 32-bit word (a, b may lie outside it).
__device__ __forceinline__ uint32_t bit_range(int a, int b) {
  a = max(a, 0);
  b = min(b, 31);
  return a > b ? 0u : (0xffffffffu << a) & (0xffffffffu >> (31 - b));
}

// 2^x of a pair without the special-function unit: x = k + f with k the
// nearest integer (added and taken off again in the units of 1.5 * 2^23), f in
// [-1/2, 1/2], 2^f by a polynomial and k added to its exponent (the range
// reduction of Cody & Waite, Software Manual for the Elementary Functions).
// The coefficients are the degree-4 minimax polynomial of the relative error
// on [-1/2, 1/2] (Remez exchange): 2.6e-6.  x is taken as at least -125: the
// value below that, 2^-125, is zero for every use here.
//
// The unit computes 16 of these a clock and SM, 1/64 of the FMAs that a
// 128 x 128 score tile leaves unused, so the softmax sends part of its
// exponentials here.
__device__ __forceinline__ float2 ex2_fma2(float2 x) {
  x.x = fmaxf(x.x, -125.f);
  x.y = fmaxf(x.y, -125.f);
  const float2 big = make_float2(12582912.f, 12582912.f), nbig = make_float2(-12582912.f, -12582912.f);
  const float2 r = __fadd2_rn(x, big);
  const float2 k = __fadd2_rn(r, nbig);
  const float2 f = __ffma2_rn(k, make_float2(-1.f, -1.f), x);
  float2 p = make_float2(9.570101911e-03f, 9.570101911e-03f);
  p = __ffma2_rn(p, f, make_float2(5.591786032e-02f, 5.591786032e-02f));
  p = __ffma2_rn(p, f, make_float2(2.402474483e-01f, 2.402474483e-01f));
  p = __ffma2_rn(p, f, make_float2(6.931218147e-01f, 6.931218147e-01f));
  p = __ffma2_rn(p, f, make_float2(9.999992614e-01f, 9.999992614e-01f));
  return make_float2(__int_as_float(__float_as_int(p.x) + (__float_as_int(r.x) << 23)),
                     __int_as_float(__float_as_int(p.y) + (__float_as_int(r.y) << 23)));
}

// 16-byte stores of 8 values rounded to T.
template <typename T>
__device__ __forceinline__ uint4 pack8(const uint32_t* v, float scale) {
  uint4 w;
  w.x = pack2<T>(__uint_as_float(v[0]) * scale, __uint_as_float(v[1]) * scale);
  w.y = pack2<T>(__uint_as_float(v[2]) * scale, __uint_as_float(v[3]) * scale);
  w.z = pack2<T>(__uint_as_float(v[4]) * scale, __uint_as_float(v[5]) * scale);
  w.w = pack2<T>(__uint_as_float(v[6]) * scale, __uint_as_float(v[7]) * scale);
  return w;
}

// Zeroes rows [row0, rows) of a tile of 64-column chunks ([rows][128 bytes]
// each; the 128-byte swizzle moves bytes within a row only) and makes that
// visible to the tensor core.  Called by one converged warp.
__device__ __forceinline__ void zero_tile_rows(uint8_t* tile, int chunks, int rows, int row0, int lane) {
  for (int c = 0; c < chunks; ++c)
    for (int i = row0 * 8 + lane; i < rows * 8; i += 32)
      *reinterpret_cast<uint4*>(tile + c * rows * 128 + i * 16) = make_uint4(0u, 0u, 0u, 0u);
  tc::fence_proxy_async_smem();
  __syncwarp();
}

}  // namespace dash
