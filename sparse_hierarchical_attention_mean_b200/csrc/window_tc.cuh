// Device helpers of the tensor-core sliding-window kernels.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "tc.cuh"
#include "window.h"

namespace dash {

// Registers per thread of the calling warpgroup (all four warps call it); the
// block's sum must stay within what it was launched with.
template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}

// Waits for phase `phase` of a barrier (counted from 0); the answer is the
// same for the whole warp.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, int phase) {
  return __all_sync(0xffffffffu, tc::mbar_wait(bar, phase & 1));
}

// One arrival for a warp, after all of its lanes got here.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) tc::mbar_arrive(bar);
}

// A CTA's work items x of (n_x per head, Hkv, B), x fastest: every gridDim.x-th
// from blockIdx.x on.  The steps between them are kept as digits, so that the
// way to the next item takes no division.
struct ItemWalk {
  int x, g, b, n_x, n_g, n_b, dx, dg, db;
  __device__ ItemWalk(int n_x, int n_g, int n_b) : n_x(n_x), n_g(n_g), n_b(n_b) {
    split(blockIdx.x, &x, &g, &b);
    split(gridDim.x, &dx, &dg, &db);
  }
  __device__ void split(int i, int* x, int* g, int* b) const {
    *x = i % n_x;
    i /= n_x;
    *g = i % n_g;
    *b = i / n_g;
  }
  __device__ bool any() const { return b < n_b; }
  __device__ void next() {
    x += dx;
    const bool c = x >= n_x;
    x -= c ? n_x : 0;
    g += dg + c;
    const bool c2 = g >= n_g;
    g -= c2 ? n_g : 0;
    b += db + c2;
  }
};

// Bits [a, b] of a 32-bit word (a, b may lie outside it).
__device__ __forceinline__ uint32_t bit_range(int a, int b) {
  a = max(a, 0);
  b = min(b, 31);
  return a > b ? 0u : (0xffffffffu << a) & (0xffffffffu >> (31 - b));
}

// 2^x and the packing of a pair (the first in the low half) that keep their
// place in the instruction stream: a warp issues in order, so the softmax
// interleaves the special-function unit's instructions (8 clocks each) with
// the FMAs, sums and conversions of other elements by hand.
__device__ __forceinline__ float ex2_placed(float x) {
  float y;
  asm volatile("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
template <typename T>
__device__ __forceinline__ uint32_t pack2_placed(float2 x) {
  uint32_t r;
  if constexpr (std::is_same<T, __nv_bfloat16>::value)
    asm volatile("cvt.rn.bf16x2.f32 %0, %2, %1;\n" : "=r"(r) : "f"(x.x), "f"(x.y));
  else
    asm volatile("cvt.rn.f16x2.f32 %0, %2, %1;\n" : "=r"(r) : "f"(x.x), "f"(x.y));
  return r;
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

// 32 values of a row, scaled and rounded to T (64 bytes), in 32-byte stores
// where the row allows it.  A thread writes its own row: a warp's store touches
// 32 lines, but whole sectors of them, and needs no exchange between lanes
// (moving 8 x 8 pieces of 16 bytes between the lanes first, so that a store
// touches 4 lines, took 48 shuffles and 96 selects per 64 columns and was no
// faster: 1.05 and 1.03 ms for a 32K prompt).
template <typename T>
__device__ __forceinline__ void store_row32(T* dst, const uint32_t* v, float scale, bool wide) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint4 a = pack8<T>(v + h * 16, scale), b = pack8<T>(v + h * 16 + 8, scale);
    if (wide) {
      asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(dst + h * 16), "r"(a.x), "r"(a.y),
                   "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                   : "memory");
    } else {
      *reinterpret_cast<uint4*>(dst + h * 16) = a;
      *reinterpret_cast<uint4*>(dst + h * 16 + 8) = b;
    }
  }
}

// v <- what is left of v * scale when it is rounded to T.
template <typename T>
__device__ __forceinline__ void rounding_rest(uint32_t* v, float scale) {
#pragma unroll
  for (int j = 0; j < 32; j += 8) {
    float f[8];
    Elt<T>::to_float(pack8<T>(v + j, scale), f);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[j + e] = __float_as_uint(fmaf(__uint_as_float(v[j + e]), scale, -f[e]));
  }
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
