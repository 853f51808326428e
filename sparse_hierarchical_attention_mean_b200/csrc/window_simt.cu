// Sliding-window attention on the CUDA cores: forward and backward in fp32.
//
// Row i of head h sees key j when j <= i and (j > i - window or j < sinks):
//   s_ij = q_i . k_j / sqrt(D),  p_ij = exp(s_ij - lse_i),  o_i = sum_j p_ij v_j
//   D_i = do_i . o_i,  ds_ij = p_ij (do_i . v_j - D_i)
//   dq_i = sum_j ds_ij k_j / sqrt(D),  dk_j = sum_i ds_ij q_i / sqrt(D),
//   dv_j = sum_i p_ij do_i  (sums over the heads of the group too)
//
// Tiles of 64 rows x 64 keys in shared memory; 256 threads as 16 x 16, each
// with a 4 x 4 block of the scores and 4 rows x D / 16 columns of each
// output.  Only tiles that hold a visible pair are walked.  The products are
// bound by the fp32 FMA rate; rows and keys at or past the sequence's length
// are loaded as zeros, so what stands there is never multiplied.
#include "common.cuh"
#include "window.h"

namespace dash {
namespace {

constexpr int kT = 64;         // rows and keys per tile
constexpr int kThreads = 256;  // 16 x 16

// [64][D] tile, rows padded by 4 floats: the 16 row-blocks of a warp's reads
// fall into different banks
template <int D>
constexpr int ld() {
  return D + 4;
}

// Starts the copies of a tile (16 bytes each; rows at or past n as zeros); the
// caller commits and waits for them.
template <int D>
__device__ __forceinline__ void load_tile(float* dst, const View& v, int b, int h, int row0, int n) {
  constexpr int V = D / 4;
  const float* src = static_cast<const float*>(v.data) + (int64_t)b * v.sb + (int64_t)h * v.sh;
  for (int i = threadIdx.x; i < kT * V; i += kThreads) {
    const int r = i / V, c = (i % V) * 4;
    const bool there = row0 + r < n;
    cp_async16(dst + r * ld<D>() + c, src + (int64_t)(there ? row0 + r : 0) * v.ss + c, there);
  }
}

// acc[4][4] = rows (4 ty ..) of a . rows (tx + 16 j) of b
template <int D>
__device__ __forceinline__ void dot_tile(const float* a, const float* b, int ty, int tx, float (&acc)[4][4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll 4
  for (int e = 0; e < D; e += 4) {
    float4 x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(a + (4 * ty + i) * ld<D>() + e);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(b + (tx + 16 * j) * ld<D>() + e);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[i][j] = fmaf(x[i].x, y[j].x, acc[i][j]);
        acc[i][j] = fmaf(x[i].y, y[j].y, acc[i][j]);
        acc[i][j] = fmaf(x[i].z, y[j].z, acc[i][j]);
        acc[i][j] = fmaf(x[i].w, y[j].w, acc[i][j]);
      }
  }
}

// acc[4][D / 16] += sum over t of w[r][t] m[t][c]: rows r = 4 ty .., columns
// c = 4 tx + 64 j ..; w is [64][kT + 4], m a [64][D] tile
template <int D>
__device__ __forceinline__ void add_product(const float* w, const float* m, int ty, int tx, float (&acc)[4][D / 16]) {
#pragma unroll 4
  for (int t = 0; t < kT; ++t) {
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = w[(4 * ty + i) * (kT + 4) + t];
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      const float4 y = *reinterpret_cast<const float4*>(m + t * ld<D>() + 4 * tx + 64 * j);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[i][4 * j + 0] = fmaf(x[i], y.x, acc[i][4 * j + 0]);
        acc[i][4 * j + 1] = fmaf(x[i], y.y, acc[i][4 * j + 1]);
        acc[i][4 * j + 2] = fmaf(x[i], y.z, acc[i][4 * j + 2]);
        acc[i][4 * j + 3] = fmaf(x[i], y.w, acc[i][4 * j + 3]);
      }
    }
  }
}

template <int D>
__device__ __forceinline__ void store_rows(const View& v, int b, int h, int row0, int S, int ty, int tx,
                                           const float (&acc)[4][D / 16], const float (&scale)[4]) {
  float* dst = static_cast<float*>(const_cast<void*>(v.data)) + (int64_t)b * v.sb + (int64_t)h * v.sh;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = row0 + 4 * ty + i;
    if (r >= S) continue;
#pragma unroll
    for (int j = 0; j < D / 64; ++j)
      *reinterpret_cast<float4*>(dst + (int64_t)r * v.ss + 4 * tx + 64 * j) =
          make_float4(acc[i][4 * j] * scale[i], acc[i][4 * j + 1] * scale[i], acc[i][4 * j + 2] * scale[i],
                      acc[i][4 * j + 3] * scale[i]);
  }
}

__device__ __forceinline__ bool visible(int i, int j, int n, int window, int sinks) {
  return i < n && j <= i && (j > i - window || j < sinks);
}

// over the 16 threads that share a row
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ float row_max(float x) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

template <int D>
constexpr int tile_floats() {
  return kT * ld<D>();
}
constexpr int kScoreFloats = kT * (kT + 4);

template <int D>
__global__ void __launch_bounds__(kThreads) window_fwd_simt_kernel(WindowParams p) {
  extern __shared__ __align__(16) float smem[];
  float* qs = smem;
  float* ks = qs + tile_floats<D>();
  float* vs = ks + tile_floats<D>();
  float* ps = vs + tile_floats<D>();
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x < 32) begin_status(p, threadIdx.x);
  const int h = blockIdx.y, b = blockIdx.z, g = h / p.G;
  const int r0 = blockIdx.x * kT;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int n = window_len(p, b);
  float acc[4][D / 16], m[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = kNegInf;
    l[i] = 0.f;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) acc[i][j] = 0.f;
  }
  if (r0 < n) {
    const float scale = rsqrtf((float)D) * kLog2e;
    const KeyTiles kt(r0, min(r0 + kT, n), p.window, p.sinks, kT);
    // K of the next tile comes during this one's softmax and second product, V
    // of it during its first
    load_tile<D>(qs, p.q, b, h, r0, n);
    load_tile<D>(ks, p.k, b, g, kt.tile(0) * kT, n);
    cp_async_commit();
    load_tile<D>(vs, p.v, b, g, kt.tile(0) * kT, n);
    cp_async_commit();
    for (int t = 0; t < kt.n; ++t) {
      const int k0 = kt.tile(t) * kT, k1 = t + 1 < kt.n ? kt.tile(t + 1) * kT : p.S;  // p.S: nothing to load
      cp_async_wait<1>();
      __syncthreads();
      float s[4][4];
      dot_tile<D>(qs, ks, ty, tx, s);
      __syncthreads();
      load_tile<D>(ks, p.k, b, g, k1, min(n, k1 + kT));
      cp_async_commit();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float mx = kNegInf;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = visible(r0 + 4 * ty + i, k0 + tx + 16 * j, n, p.window, p.sinks) ? s[i][j] * scale : kNegInf;
          mx = fmaxf(mx, s[i][j]);
        }
        mx = fmaxf(m[i], row_max(mx));
        const float ref = mx == kNegInf ? 0.f : mx;  // a row that has seen no key yet
        const float corr = exp2f(m[i] - ref);
        m[i] = mx;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float e = exp2f(s[i][j] - ref);
          sum += e;
          ps[(4 * ty + i) * (kT + 4) + tx + 16 * j] = e;
        }
        l[i] = l[i] * corr + row_sum(sum);
#pragma unroll
        for (int j = 0; j < D / 16; ++j) acc[i][j] *= corr;
      }
      cp_async_wait<1>();
      __syncthreads();
      add_product<D>(ps, vs, ty, tx, acc);
      __syncthreads();
      load_tile<D>(vs, p.v, b, g, k1, min(n, k1 + kT));
      cp_async_commit();
    }
    cp_async_wait<0>();
  }
  float inv[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    inv[i] = l[i] > 0.f ? 1.f / l[i] : 0.f;
    const int r = r0 + 4 * ty + i;
    if (p.lse && tx == 0 && r < p.S)
      p.lse[((int64_t)b * p.H + h) * p.S + r] = l[i] > 0.f ? m[i] / kLog2e + logf(l[i]) : kNegInf;
  }
  store_rows<D>(p.out, b, h, r0, p.S, ty, tx, acc, inv);
}

// One 64-row tile of one head: D_i (written for the key kernel) and dq.
template <int D>
__global__ void __launch_bounds__(kThreads) window_bwd_row_simt_kernel(WindowParams p) {
  extern __shared__ __align__(16) float smem[];
  float* qs = smem;
  float* dos = qs + tile_floats<D>();
  float* ks = dos + tile_floats<D>();
  float* vs = ks + tile_floats<D>();
  float* dss = vs + tile_floats<D>();
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x < 32) begin_status(p, threadIdx.x);
  const int h = blockIdx.y, b = blockIdx.z, g = h / p.G;
  const int r0 = blockIdx.x * kT;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int n = window_len(p, b);
  float acc[4][D / 16], dd[4], lse2[4], one[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    one[i] = rsqrtf((float)D);
#pragma unroll
    for (int j = 0; j < D / 16; ++j) acc[i][j] = 0.f;
  }
  if (r0 < n) {
    const float scale = rsqrtf((float)D) * kLog2e;
    load_tile<D>(qs, p.q, b, h, r0, n);
    load_tile<D>(dos, p.dout, b, h, r0, n);
    load_tile<D>(ks, p.out, b, h, r0, n);
    cp_async_commit();
    cp_async_wait<0>();
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + 4 * ty + i;
      float x = 0.f;
      for (int e = tx; e < D; e += 16) x = fmaf(dos[(4 * ty + i) * ld<D>() + e], ks[(4 * ty + i) * ld<D>() + e], x);
      dd[i] = row_sum(x);
      lse2[i] = r < n ? p.lse[((int64_t)b * p.H + h) * p.S + r] * kLog2e : 0.f;
      if (tx == 0 && r < n) p.dd[((int64_t)b * p.H + h) * p.S + r] = dd[i];
    }
    const KeyTiles kt(r0, min(r0 + kT, n), p.window, p.sinks, kT);
    for (int t = 0; t < kt.n; ++t) {
      const int k0 = kt.tile(t) * kT;
      __syncthreads();
      load_tile<D>(ks, p.k, b, g, k0, n);
      load_tile<D>(vs, p.v, b, g, k0, n);
      cp_async_commit();
      cp_async_wait<0>();
      __syncthreads();
      float s[4][4], dp[4][4];
      dot_tile<D>(qs, ks, ty, tx, s);
      dot_tile<D>(dos, vs, ty, tx, dp);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bool vis = visible(r0 + 4 * ty + i, k0 + tx + 16 * j, n, p.window, p.sinks);
          dss[(4 * ty + i) * (kT + 4) + tx + 16 * j] =
              vis ? exp2f(fmaf(s[i][j], scale, -lse2[i])) * (dp[i][j] - dd[i]) : 0.f;
        }
      __syncwarp();
      add_product<D>(dss, ks, ty, tx, acc);
    }
  }
  store_rows<D>(p.dq, b, h, r0, p.S, ty, tx, acc, one);
}

// One 64-key tile of one KV head: dk and dv, summed over the group's heads in
// order and over the row tiles in order (no atomics: the same every time).
template <int D>
__global__ void __launch_bounds__(kThreads) window_bwd_key_simt_kernel(WindowParams p) {
  extern __shared__ __align__(16) float smem[];
  float* ks = smem;
  float* vs = ks + tile_floats<D>();
  float* qs = vs + tile_floats<D>();
  float* dos = qs + tile_floats<D>();
  float* ws = dos + tile_floats<D>();  // [key][row], p then ds
  const int g = blockIdx.y, b = blockIdx.z;
  const int k0 = blockIdx.x * kT;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int n = window_len(p, b);
  float dk[4][D / 16], dv[4][D / 16], sk[4], sv[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sk[i] = rsqrtf((float)D);
    sv[i] = 1.f;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) dk[i][j] = dv[i][j] = 0.f;
  }
  if (k0 < n) {
    const float scale = rsqrtf((float)D) * kLog2e;
    load_tile<D>(ks, p.k, b, g, k0, n);
    load_tile<D>(vs, p.v, b, g, k0, n);
    // the last row that sees a key of the tile (every later row when it holds sinks)
    const int last = k0 < p.sinks ? n - 1 : (int)min((int64_t)n - 1, (int64_t)k0 + kT - 1 + p.window - 1);
    for (int gh = 0; gh < p.G; ++gh) {
      const int h = g * p.G + gh;
      const int64_t rbase = ((int64_t)b * p.H + h) * p.S;
      for (int r0 = k0; r0 <= last; r0 += kT) {
        __syncthreads();
        load_tile<D>(qs, p.q, b, h, r0, n);
        load_tile<D>(dos, p.dout, b, h, r0, n);
        cp_async_commit();
        cp_async_wait<0>();
        __syncthreads();
        float s[4][4], dp[4][4];
        dot_tile<D>(ks, qs, ty, tx, s);
        dot_tile<D>(vs, dos, ty, tx, dp);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = r0 + tx + 16 * j;
          const float l2 = r < n ? p.lse[rbase + r] * kLog2e : 0.f, d = r < n ? p.dd[rbase + r] : 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool vis = visible(r, k0 + 4 * ty + i, n, p.window, p.sinks);
            const float e = vis ? exp2f(fmaf(s[i][j], scale, -l2)) : 0.f;
            ws[(4 * ty + i) * (kT + 4) + tx + 16 * j] = e;
            s[i][j] = vis ? e * (dp[i][j] - d) : 0.f;
          }
        }
        __syncwarp();
        add_product<D>(ws, dos, ty, tx, dv);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) ws[(4 * ty + i) * (kT + 4) + tx + 16 * j] = s[i][j];
        __syncwarp();
        add_product<D>(ws, qs, ty, tx, dk);
      }
    }
  }
  store_rows<D>(p.dk, b, g, k0, p.S, ty, tx, dk, sk);
  store_rows<D>(p.dv, b, g, k0, p.S, ty, tx, dv, sv);
}

template <typename K>
cudaError_t launch(K kern, dim3 grid, int floats, const WindowParams& p, cudaStream_t stream) {
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, floats * 4);
  if (e != cudaSuccess) return e;
  kern<<<grid, kThreads, floats * 4, stream>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t run_fwd(const WindowParams& p, cudaStream_t stream) {
  return launch(window_fwd_simt_kernel<D>, dim3((p.S + kT - 1) / kT, p.H, p.B),
                3 * tile_floats<D>() + kScoreFloats, p, stream);
}

template <int D>
cudaError_t run_bwd(const WindowParams& p, cudaStream_t stream) {
  const unsigned tiles = (p.S + kT - 1) / kT;
  const int floats = 4 * tile_floats<D>() + kScoreFloats;
  cudaError_t e = launch(window_bwd_row_simt_kernel<D>, dim3(tiles, p.H, p.B), floats, p, stream);
  if (e != cudaSuccess) return e;
  return launch(window_bwd_key_simt_kernel<D>, dim3(tiles, p.Hkv, p.B), floats, p, stream);
}

}  // namespace

cudaError_t launch_window_fwd_simt(const WindowParams& p, cudaStream_t stream) {
  return p.D == 128 ? run_fwd<128>(p, stream) : run_fwd<64>(p, stream);
}
cudaError_t launch_window_bwd_simt(const WindowParams& p, cudaStream_t stream) {
  return p.D == 128 ? run_bwd<128>(p, stream) : run_bwd<64>(p, stream);
}

}  // namespace dash
