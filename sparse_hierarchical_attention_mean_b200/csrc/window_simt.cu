// Sliding-window attention on the CUDA cores: forward and backward in fp32.
//
// Row i of head h sees key j when j <= i and (j > i - window or j < sinks):
//   s_ij = q_i . k_j / sqrt(D),  p_ij = exp(s_ij - lse_i),  o_i = sum_j p_ij v_j
//   D_i = do_i . o_i,  ds_ij = p_ij (do_i . v_j - D_i)
//   dq_i = sum_j ds_ij k_j / sqrt(D),  dk_j = sum_i ds_ij q_i / sqrt(D),
//   dv_j = sum_i p_ij do_i  (sums over the heads of the group too)
//
// A CTA owns 16 RB rows (or keys) and goes through the other side in tiles of
// 64; 256 threads as 16 x 16, each with an RB x 4 block of the scores and RB
// rows x D / 16 columns of each output.  Only tiles that hold a visible pair
// are walked.  The products are bound by the fp32 FMA rate when there are CTAs
// enough; RB is the largest of 4, 2, 1 that gives every SM one (4 heads of 200
// tokens, d 128: 40 us with RB = 4, 26 with RB = 1; 2 sequences of up to 777
// tokens, 8 heads, window 100: 38 with RB = 4, 41 with RB = 2).
// Rows and keys at or past the sequence's length are loaded as zeros, so what
// stands there is never multiplied.
#include "common.cuh"
#include "window.h"

namespace dash {
namespace {

constexpr int kT = 64;         // streamed keys (rows) per tile
constexpr int kThreads = 256;  // 16 x 16

// tile rows of D, padded by 4 floats: the 16 row-blocks of a warp's reads
// fall into different banks
template <int D>
constexpr int ld() {
  return D + 4;
}

// Starts the copies of a tile (16 bytes each; rows at or past n as zeros); the
// caller commits and waits for them.
template <int D, int R = kT>
__device__ __forceinline__ void load_tile(float* dst, const View& v, int b, int h, int row0, int n) {
  constexpr int V = D / 4;
  const float* src = static_cast<const float*>(v.data) + (int64_t)b * v.sb + (int64_t)h * v.sh;
  for (int i = threadIdx.x; i < R * V; i += kThreads) {
    const int r = i / V, c = (i % V) * 4;
    const bool there = row0 + r < n;
    cp_async16(dst + r * ld<D>() + c, src + (int64_t)(there ? row0 + r : 0) * v.ss + c, there);
  }
}

// acc = rows (RB ty ..) of a . rows (tx + 16 j) of b; the even and the odd
// elements in one paired FMA
template <int D, int RB>
__device__ __forceinline__ void dot_tile(const float* a, const float* b, int ty, int tx, float (&acc)[RB][4]) {
  float2 p[RB][4];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) p[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
  for (int e = 0; e < D; e += 4) {
    float4 x[RB], y[4];
#pragma unroll
    for (int i = 0; i < RB; ++i) x[i] = *reinterpret_cast<const float4*>(a + (RB * ty + i) * ld<D>() + e);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(b + (tx + 16 * j) * ld<D>() + e);
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        p[i][j] = __ffma2_rn(make_float2(x[i].x, x[i].y), make_float2(y[j].x, y[j].y), p[i][j]);
        p[i][j] = __ffma2_rn(make_float2(x[i].z, x[i].w), make_float2(y[j].z, y[j].w), p[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = p[i][j].x + p[i][j].y;
}

// acc += sum over t of w[r][t] m[t][c]: rows r = RB ty .., columns
// c = 4 tx + 64 j ..; w is [16 RB][kT + 4], m a [64][D] tile
template <int D, int RB>
__device__ __forceinline__ void add_product(const float* w, const float* m, int ty, int tx, float (&acc)[RB][D / 16]) {
#pragma unroll 2
  for (int t = 0; t < kT; t += 4) {
    float4 x[RB];
#pragma unroll
    for (int i = 0; i < RB; ++i) x[i] = *reinterpret_cast<const float4*>(w + (RB * ty + i) * (kT + 4) + t);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        const float4 y = *reinterpret_cast<const float4*>(m + (t + u) * ld<D>() + 4 * tx + 64 * j);
#pragma unroll
        for (int i = 0; i < RB; ++i) {
          const float xi = u == 0 ? x[i].x : u == 1 ? x[i].y : u == 2 ? x[i].z : x[i].w;
          const float2 xx = make_float2(xi, xi);
          float* o = acc[i] + 4 * j;
          const float2 lo = __ffma2_rn(xx, make_float2(y.x, y.y), make_float2(o[0], o[1]));
          const float2 hi = __ffma2_rn(xx, make_float2(y.z, y.w), make_float2(o[2], o[3]));
          o[0] = lo.x, o[1] = lo.y, o[2] = hi.x, o[3] = hi.y;
        }
      }
    }
  }
}

template <int D, int RB>
__device__ __forceinline__ void store_rows(const View& v, int b, int h, int row0, int S, int ty, int tx,
                                           const float (&acc)[RB][D / 16], const float (&scale)[RB]) {
  float* dst = static_cast<float*>(const_cast<void*>(v.data)) + (int64_t)b * v.sb + (int64_t)h * v.sh;
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    const int r = row0 + RB * ty + i;
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

template <int D, int R = kT>
constexpr int tile_floats() {
  return R * ld<D>();
}
template <int RB>
constexpr int score_floats() {
  return 16 * RB * (kT + 4);
}

template <int D, int RB>
__global__ void __launch_bounds__(kThreads) window_fwd_simt_kernel(WindowParams p) {
  constexpr int R = 16 * RB;
  extern __shared__ __align__(16) float smem[];
  float* qs = smem;
  float* ks = qs + tile_floats<D, R>();
  float* vs = ks + tile_floats<D>();
  float* ps = vs + tile_floats<D>();
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x < 32) begin_status(p, threadIdx.x);
  const int h = blockIdx.y, b = blockIdx.z, g = h / p.G;
  const int r0 = blockIdx.x * R;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int n = window_len(p, b);
  float acc[RB][D / 16], m[RB], l[RB];
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    m[i] = kNegInf;
    l[i] = 0.f;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) acc[i][j] = 0.f;
  }
  if (r0 < n) {
    const float scale = rsqrtf((float)D) * kLog2e;
    const KeyTiles kt(r0, min(r0 + R, n), p.window, p.sinks, kT);
    // K of the next tile comes during this one's softmax and second product, V
    // of it during its first
    load_tile<D, R>(qs, p.q, b, h, r0, n);
    load_tile<D>(ks, p.k, b, g, kt.tile(0) * kT, n);
    cp_async_commit();
    load_tile<D>(vs, p.v, b, g, kt.tile(0) * kT, n);
    cp_async_commit();
    for (int t = 0; t < kt.n; ++t) {
      const int k0 = kt.tile(t) * kT, k1 = t + 1 < kt.n ? kt.tile(t + 1) * kT : p.S;  // p.S: nothing to load
      cp_async_wait<1>();
      __syncthreads();
      float s[RB][4];
      dot_tile<D, RB>(qs, ks, ty, tx, s);
      __syncthreads();
      load_tile<D>(ks, p.k, b, g, k1, min(n, k1 + kT));
      cp_async_commit();
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        float mx = kNegInf;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = visible(r0 + RB * ty + i, k0 + tx + 16 * j, n, p.window, p.sinks) ? s[i][j] * scale : kNegInf;
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
          ps[(RB * ty + i) * (kT + 4) + tx + 16 * j] = e;
        }
        l[i] = l[i] * corr + row_sum(sum);
#pragma unroll
        for (int j = 0; j < D / 16; ++j) acc[i][j] *= corr;
      }
      cp_async_wait<1>();
      __syncthreads();
      add_product<D, RB>(ps, vs, ty, tx, acc);
      __syncthreads();
      load_tile<D>(vs, p.v, b, g, k1, min(n, k1 + kT));
      cp_async_commit();
    }
    cp_async_wait<0>();
  }
  float inv[RB];
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    inv[i] = l[i] > 0.f ? 1.f / l[i] : 0.f;
    const int r = r0 + RB * ty + i;
    if (p.lse && tx == 0 && r < p.S)
      p.lse[((int64_t)b * p.H + h) * p.S + r] = l[i] > 0.f ? m[i] / kLog2e + logf(l[i]) : kNegInf;
  }
  store_rows<D, RB>(p.out, b, h, r0, p.S, ty, tx, acc, inv);
}

// One 64-row tile of one head: D_i (written for the key kernel) and dq.
template <int D, int RB>
__global__ void __launch_bounds__(kThreads) window_bwd_row_simt_kernel(WindowParams p) {
  constexpr int R = 16 * RB;
  extern __shared__ __align__(16) float smem[];
  float* qs = smem;
  float* dos = qs + tile_floats<D, R>();
  float* ks = dos + tile_floats<D, R>();
  float* vs = ks + tile_floats<D>();
  float* dss = vs + tile_floats<D>();
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x < 32) begin_status(p, threadIdx.x);
  const int h = blockIdx.y, b = blockIdx.z, g = h / p.G;
  const int r0 = blockIdx.x * R;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int n = window_len(p, b);
  float acc[RB][D / 16], dd[RB], lse2[RB], one[RB];
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    one[i] = rsqrtf((float)D);
#pragma unroll
    for (int j = 0; j < D / 16; ++j) acc[i][j] = 0.f;
  }
  if (r0 < n) {
    const float scale = rsqrtf((float)D) * kLog2e;
    load_tile<D, R>(qs, p.q, b, h, r0, n);
    load_tile<D, R>(dos, p.dout, b, h, r0, n);
    load_tile<D, R>(ks, p.out, b, h, r0, n);
    cp_async_commit();
    cp_async_wait<0>();
    __syncthreads();
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      const int r = r0 + RB * ty + i;
      float x = 0.f;
      for (int e = tx; e < D; e += 16) x = fmaf(dos[(RB * ty + i) * ld<D>() + e], ks[(RB * ty + i) * ld<D>() + e], x);
      dd[i] = row_sum(x);
      lse2[i] = r < n ? p.lse[((int64_t)b * p.H + h) * p.S + r] * kLog2e : 0.f;
      if (tx == 0 && r < n) p.dd[((int64_t)b * p.H + h) * p.S + r] = dd[i];
    }
    const KeyTiles kt(r0, min(r0 + R, n), p.window, p.sinks, kT);
    for (int t = 0; t < kt.n; ++t) {
      const int k0 = kt.tile(t) * kT;
      __syncthreads();
      load_tile<D>(ks, p.k, b, g, k0, n);
      load_tile<D>(vs, p.v, b, g, k0, n);
      cp_async_commit();
      cp_async_wait<0>();
      __syncthreads();
      float s[RB][4], dp[RB][4];
      dot_tile<D, RB>(qs, ks, ty, tx, s);
      dot_tile<D, RB>(dos, vs, ty, tx, dp);
#pragma unroll
      for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bool vis = visible(r0 + RB * ty + i, k0 + tx + 16 * j, n, p.window, p.sinks);
          dss[(RB * ty + i) * (kT + 4) + tx + 16 * j] =
              vis ? exp2f(fmaf(s[i][j], scale, -lse2[i])) * (dp[i][j] - dd[i]) : 0.f;
        }
      __syncwarp();
      add_product<D, RB>(dss, ks, ty, tx, acc);
    }
  }
  store_rows<D, RB>(p.dq, b, h, r0, p.S, ty, tx, acc, one);
}

// One 64-key tile of one KV head: dk and dv, summed over the group's heads in
// order and over the row tiles in order (no atomics: the same every time).
template <int D, int RB>
__global__ void __launch_bounds__(kThreads) window_bwd_key_simt_kernel(WindowParams p) {
  constexpr int R = 16 * RB;
  extern __shared__ __align__(16) float smem[];
  float* ks = smem;
  float* vs = ks + tile_floats<D, R>();
  float* qs = vs + tile_floats<D, R>();
  float* dos = qs + tile_floats<D>();
  float* ws = dos + tile_floats<D>();  // [key][row], p then ds
  const int g = blockIdx.y, b = blockIdx.z;
  const int k0 = blockIdx.x * R;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int n = window_len(p, b);
  float dk[RB][D / 16], dv[RB][D / 16], sk[RB], sv[RB];
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    sk[i] = rsqrtf((float)D);
    sv[i] = 1.f;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) dk[i][j] = dv[i][j] = 0.f;
  }
  if (k0 < n) {
    const float scale = rsqrtf((float)D) * kLog2e;
    load_tile<D, R>(ks, p.k, b, g, k0, n);
    load_tile<D, R>(vs, p.v, b, g, k0, n);
    // the last row that sees a key of the tile (every later row when it holds sinks)
    const int last = k0 < p.sinks ? n - 1 : (int)min((int64_t)n - 1, (int64_t)k0 + R - 1 + p.window - 1);
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
        float s[RB][4], dp[RB][4];
        dot_tile<D, RB>(ks, qs, ty, tx, s);
        dot_tile<D, RB>(vs, dos, ty, tx, dp);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = r0 + tx + 16 * j;
          const float l2 = r < n ? p.lse[rbase + r] * kLog2e : 0.f, d = r < n ? p.dd[rbase + r] : 0.f;
#pragma unroll
          for (int i = 0; i < RB; ++i) {
            const bool vis = visible(r, k0 + RB * ty + i, n, p.window, p.sinks);
            const float e = vis ? exp2f(fmaf(s[i][j], scale, -l2)) : 0.f;
            ws[(RB * ty + i) * (kT + 4) + tx + 16 * j] = e;
            s[i][j] = vis ? e * (dp[i][j] - d) : 0.f;
          }
        }
        __syncwarp();
        add_product<D, RB>(ws, dos, ty, tx, dv);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) ws[(RB * ty + i) * (kT + 4) + tx + 16 * j] = s[i][j];
        __syncwarp();
        add_product<D, RB>(ws, qs, ty, tx, dk);
      }
    }
  }
  store_rows<D, RB>(p.dk, b, g, k0, p.S, ty, tx, dk, sk);
  store_rows<D, RB>(p.dv, b, g, k0, p.S, ty, tx, dv, sv);
}

template <typename K>
cudaError_t launch(K kern, dim3 grid, int floats, const WindowParams& p, cudaStream_t stream) {
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, floats * 4);
  if (e != cudaSuccess) return e;
  kern<<<grid, kThreads, floats * 4, stream>>>(p);
  return cudaGetLastError();
}

// Rows per thread: the largest with which `heads` heads give every SM a CTA.
int rows_per_thread(const WindowParams& p, int heads) {
  for (int rb = 4; rb > 1; rb /= 2)
    if ((int64_t)((p.S + 16 * rb - 1) / (16 * rb)) * heads * p.B >= p.num_sms) return rb;
  return 1;
}
dim3 grid_of(const WindowParams& p, int rb, int heads) {
  return dim3((unsigned)((p.S + 16 * rb - 1) / (16 * rb)), heads, p.B);
}

template <int D, int RB>
cudaError_t run_fwd(const WindowParams& p, cudaStream_t stream) {
  return launch(window_fwd_simt_kernel<D, RB>, grid_of(p, RB, p.H),
                tile_floats<D, 16 * RB>() + 2 * tile_floats<D>() + score_floats<RB>(), p, stream);
}
template <int D, int RB>
cudaError_t run_bwd_row(const WindowParams& p, cudaStream_t stream) {
  return launch(window_bwd_row_simt_kernel<D, RB>, grid_of(p, RB, p.H),
                2 * tile_floats<D, 16 * RB>() + 2 * tile_floats<D>() + score_floats<RB>(), p, stream);
}
template <int D, int RB>
cudaError_t run_bwd_key(const WindowParams& p, cudaStream_t stream) {
  return launch(window_bwd_key_simt_kernel<D, RB>, grid_of(p, RB, p.Hkv),
                2 * tile_floats<D, 16 * RB>() + 2 * tile_floats<D>() + score_floats<RB>(), p, stream);
}

template <int D>
cudaError_t run_fwd(const WindowParams& p, cudaStream_t stream) {
  const int rb = rows_per_thread(p, p.H);
  return rb == 4 ? run_fwd<D, 4>(p, stream) : rb == 2 ? run_fwd<D, 2>(p, stream) : run_fwd<D, 1>(p, stream);
}
template <int D>
cudaError_t run_bwd(const WindowParams& p, cudaStream_t stream) {
  int rb = rows_per_thread(p, p.H);
  const cudaError_t e = rb == 4   ? run_bwd_row<D, 4>(p, stream)
                        : rb == 2 ? run_bwd_row<D, 2>(p, stream)
                                  : run_bwd_row<D, 1>(p, stream);
  if (e != cudaSuccess) return e;
  rb = rows_per_thread(p, p.Hkv);
  return rb == 4   ? run_bwd_key<D, 4>(p, stream)
         : rb == 2 ? run_bwd_key<D, 2>(p, stream)
                   : run_bwd_key<D, 1>(p, stream);
}

}  // namespace

cudaError_t launch_window_fwd_simt(const WindowParams& p, cudaStream_t stream) {
  return p.D == 128 ? run_fwd<128>(p, stream) : run_fwd<64>(p, stream);
}
cudaError_t launch_window_bwd_simt(const WindowParams& p, cudaStream_t stream) {
  return p.D == 128 ? run_bwd<128>(p, stream) : run_bwd<64>(p, stream);
}

}  // namespace dash
