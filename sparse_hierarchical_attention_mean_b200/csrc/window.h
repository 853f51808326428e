// Parameters of the sliding-window attention kernels (forward, backward and
// one-token decode) and of the cache page kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"

namespace dash {

// Causal attention of row i over the keys j <= i with j > i - window or
// j < sinks.  The host passes window in [1, S] (S: every key) and sinks in
// [0, kMaxSinks], 0 when the window hides nothing.
constexpr int kMaxSinks = 128;
constexpr int kMaxRange = 128;  // WindowParams::n_range

struct WindowParams {
  View q, k, v, out;        // [B, S, H or Hkv, D], dtype
  View rest;                // [B, S, H, D], dtype: what rounding took from out; null data: none
  View dout, dq, dk, dv;    // backward, dtype
  int dtype;
  int B, S, H, Hkv, G, D;
  int window, sinks;
  const int32_t* seqlens;   // [B] or null: rows and keys from seqlens[b] on are not there
  float* lse;               // [B, H, S] natural log-sum-exp of the row's logits, or null
  float* dd;                // [B, H, S] dout . out (backward, CUDA-core path)
  // backward, tensor-core path, in the order of the row tiles (128 / G
  // positions x G heads): [B, Hkv, n_tiles, 128]
  float* nlse2;             // -lse in log2 units; -inf on rows that are not there
  float* ndd;               // -sum_j p_ij (dout_i . v_j)
                            // (f16: as the key kernel wants them, see the scales in window_bwd_tc.cu)
  float2* range;            // f16: [B, Hkv, n_range] largest squared norms of rows of dout and of v
  int n_range;
  int n_tiles;
  float* part;              // partial dk, dv of the first 128 keys [B, Hkv, n_chunks + 1, 2, 128, D]
  int n_chunks;             // items of chunk_tiles row tiles that see only sinks of the first 128 keys
  int chunk_tiles;
  int num_sms;
  bool wide;                // rows of every output start at multiples of 32 bytes
  DeviceStatus* status;
};

// Tiles of `step` keys that rows [r0, r1) see: first the sink tiles that end
// before the band, then the band.
struct KeyTiles {
  int n_sink, band0, n;
  __host__ __device__ KeyTiles(int r0, int r1, int window, int sinks, int step) {
    const int lo = r0 - window + 1;
    band0 = (lo > 0 ? lo : 0) / step;
    const int s = (sinks + step - 1) / step;
    n_sink = s < band0 ? s : band0;
    n = n_sink + (r1 + step - 1) / step - band0;
  }
  __host__ __device__ int tile(int i) const { return i < n_sink ? i : band0 + i - n_sink; }
};

// Valid length of sequence b, clamped to [0, S].
__device__ __forceinline__ int window_len(const WindowParams& p, int b) {
  return p.seqlens ? min(max(p.seqlens[b], 0), p.S) : p.S;
}

// The call's status word, written by one warp of the first CTA of its first
// kernel when it starts: lengths out of range, else 0.  What other CTAs report
// later is a wait that ran out, a second or more after the kernel's start.
__device__ __forceinline__ void begin_status(const WindowParams& p, int lane) {
  bool bad = false;
  if (p.seqlens)
    for (int b = lane; b < p.B; b += 32) bad = bad || p.seqlens[b] < 0 || p.seqlens[b] > p.S;
  bad = __any_sync(0xffffffffu, bad);
  if (lane == 0) {
    p.status->code = bad ? 1 /* DASH_ERR_INVALID_ARGUMENT */ : 0;
    p.status->detail = bad ? 301 : 0;
  }
}

// 4-D TMA map over a [B, S, H, D] f16/bf16 view (innermost first: D, H, S, B),
// 128-byte swizzle, box {64, box_h, box_s, 1}; no multicast.  Strides must be
// valid for every extent (solid views).  narrow: L2 fetches 128 bytes at a
// time instead of 256 (for one head's 128-byte rows among others' that are not
// wanted soon).
bool window_map(CUtensorMap* map, const View& v, int dtype, int64_t B, int64_t S, int64_t H, int D, int box_h,
                int box_s, bool narrow = false);

// f16 / bf16 tensor-core path
cudaError_t launch_window_fwd_tc(const WindowParams& p, cudaStream_t stream);
cudaError_t launch_window_bwd_tc(const WindowParams& p, cudaStream_t stream);
// fp32 CUDA-core path
cudaError_t launch_window_fwd_simt(const WindowParams& p, cudaStream_t stream);
cudaError_t launch_window_bwd_simt(const WindowParams& p, cudaStream_t stream);

// ---------------------------------------------------------------- decode
constexpr int kMaxDecodeCtas = 256;  // streaming CTAs: one per SM
struct WindowDecodeParams {
  View q, k, v, out;           // q, out [B, 1, H, D]; k, v [B, Lmax, Hkv, D] or pages [n_pages, block, Hkv, D]
  int dtype;
  int B, H, Hkv, G, D;
  int64_t Lmax;                // tokens a sequence may hold
  int window, sinks;           // window 0: every token
  const int32_t* seqlens;      // [B]
  const int32_t* block_table;  // [B, max_blocks], or null: dense cache
  int max_blocks, block;       // block: tokens per page
  int64_t n_pages;             // extent of the outermost dimension of k / v
  float* lse;                  // [B, H] natural log-sum-exp, or null
  // workspace
  DeviceStatus* status;
  int32_t* cta_status;         // [n_cta] what each streaming CTA saw (0: nothing wrong)
  float* part_o;               // [2 n_cta, heads of a unit, D] unnormalised partial outputs
  float* part_ml;              // [2 n_cta, heads of a unit, 2] their reference max (log2 units) and sum
  int n_cta;
  int units;                   // KV heads, or pairs of them, of a sequence (set by the launch)
};
cudaError_t launch_window_decode(const WindowDecodeParams& p, cudaStream_t stream);

// ---------------------------------------------------------------- cache pages
// refs[p]: how many table entries hold page p (0: free).  Sequence b holds
// the first ceil(seqlens[b] / block) entries of its row.
constexpr int kMaxPageSlots = 8192;  // sequences of one table
struct PagesParams {
  int32_t* table;  // [batch, max_blocks]
  int64_t batch, max_blocks;
  int32_t* seqlens;  // [batch]
  int32_t* refs;     // [n_pages]
  int64_t n_pages;
  int block;
  // fork / free: row dst[i] becomes a copy of row src[i] (src null: empty)
  const int32_t* src;
  const int32_t* dst;
  int n;
  // grow: tokens to make room for, and the copies of shared last pages
  const int32_t* n_new;  // [batch]
  int32_t* copy_src;     // [batch]
  int32_t* copy_dst;     // [batch]
  // compact
  int32_t* table_out;
  int32_t* refs_out;
  int32_t* move_src;  // [n_pages / 2]
  int32_t* move_dst;  // [n_pages / 2]
  int32_t* info;      // {moves, pages held}
  // workspace
  int32_t* list;  // [n_pages] (grow: the pages handed out; compact: where each page went)
  int32_t* aux;   // [n_pages] (compact: refs of the moved pages)
  int32_t* rows;  // [batch, max_blocks] (fork: the source rows, when one is overwritten)
  DeviceStatus* status;
};
cudaError_t launch_pages_fork(const PagesParams& p, cudaStream_t stream);
cudaError_t launch_pages_grow(const PagesParams& p, cudaStream_t stream);
cudaError_t launch_pages_compact(const PagesParams& p, cudaStream_t stream);

// One pool: pages of `rows` x `heads` runs of `run` bytes (rows = heads = 1:
// a page is one run).
constexpr int kMaxPools = 64;
struct PagePool {
  char* data;
  int64_t n_pages, page_stride, row_stride, head_stride;  // bytes
};
struct PageCopyParams {
  PagePool pool[kMaxPools];
  int n_pools, rows, heads;
  int64_t run;  // bytes, a multiple of 16
  const int32_t* src;
  const int32_t* dst;
  int64_t n;
};
bool pages_copy_fits(const PageCopyParams& p);  // one launch's grid holds the call
cudaError_t launch_pages_copy(const PageCopyParams& p, cudaStream_t stream);

}  // namespace dash
