// Pages of a paged KV cache: forking and freeing sequences, growing them,
// compacting the pool, and copying pages.
//
// refs[p] counts the table entries that hold page p; a page is free when it
// is 0, and the free pages handed out are always the lowest ones, so the
// state is the table, the lengths and refs, every operation is a function of
// them, and nothing depends on timing (integer atomics only).
//
// The bookkeeping kernels move kilobytes to a few megabytes and are bound by
// latency: launches and dependent passes.  Each is ONE cluster of 8 CTAs
// (8192 threads, each with a consecutive range of pages), whose passes are
// separated by cluster barriers instead of launches; the per-CTA counts of a
// pass go through distributed shared memory.  Arguments that the state does
// not allow are found before the first write: the status word says so and
// nothing changes.
#include <cooperative_groups.h>

#include "common.cuh"
#include "window.h"

namespace dash {
namespace {

namespace cg = cooperative_groups;

constexpr int kCtas = 8;
constexpr int kThreads = 1024;
constexpr int kAll = kCtas * kThreads;
constexpr int kInvalid = 1;   // DASH_ERR_INVALID_ARGUMENT
constexpr int kNoPages = 6;   // DASH_ERR_OUT_OF_PAGES

__device__ __forceinline__ int blocks_of(int64_t tokens, int block) { return (int)((tokens + block - 1) / block); }

// Exclusive prefix over the CTA's threads, and the CTA's total.  `buf` holds
// 33 ints; every thread calls it.
__device__ __forceinline__ int block_scan(int x, int* buf, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();  // the last use of buf is over
  if (lane == 31) buf[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    int w = buf[lane];
    int winc = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, winc, o);
      if (lane >= o) winc += y;
    }
    buf[lane] = winc - w;
    if (lane == 31) buf[32] = winc;
  }
  __syncthreads();
  *total = buf[32];
  return buf[warp] + inc - x;
}

// The CTA's total to every CTA of the cluster (slot = its rank).  The caller
// synchronises the cluster before reading.
__device__ __forceinline__ void publish(cg::cluster_group& cl, int* slots, int value) {
  if (threadIdx.x < kCtas) *cl.map_shared_rank(slots + cl.block_rank(), threadIdx.x) = value;
}

// ------------------------------------------------------------------ fork / free

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads, 1) pages_fork_kernel(const PagesParams p) {
  cg::cluster_group cl = cg::this_cluster();
  extern __shared__ int sm[];
  int* src = sm;             // [n]
  int* dst = src + p.n;      // [n]
  int* slen = dst + p.n;     // [n] new length of dst
  int* dlen = slen + p.n;    // [n] its old length
  __shared__ uint32_t seen[kMaxPageSlots / 32];
  __shared__ int bad, overlap;
  const int tid = threadIdx.x, gt = cl.block_rank() * kThreads + tid;
  for (int i = tid; i < kMaxPageSlots / 32; i += kThreads) seen[i] = 0u;
  if (tid == 0) bad = overlap = 0;
  __syncthreads();
  const int64_t most = p.max_blocks * p.block;
  for (int i = tid; i < p.n; i += kThreads) {
    const int d = p.dst[i], s = p.src ? p.src[i] : -1;
    dst[i] = d;
    src[i] = s;
    slen[i] = dlen[i] = 0;
    if (d < 0 || d >= p.batch || (p.src && (s < 0 || s >= p.batch))) {
      bad = 1;
      continue;
    }
    if (atomicOr(&seen[d >> 5], 1u << (d & 31)) >> (d & 31) & 1u) bad = 1;  // the same row twice
    dlen[i] = p.seqlens[d];
    if (p.src) slen[i] = p.seqlens[s];
    if (dlen[i] < 0 || dlen[i] > most || slen[i] < 0 || slen[i] > most) bad = 1;
  }
  __syncthreads();
  if (p.src && !bad)
    for (int i = tid; i < p.n; i += kThreads)
      if (src[i] != dst[i] && (seen[src[i] >> 5] >> (src[i] & 31) & 1u)) overlap = 1;
  if (gt == 0) {
    p.status->code = bad ? kInvalid : 0;
    p.status->detail = bad ? 401 : 0;
  }
  cl.sync();  // every CTA has read the lengths and found the same
  if (bad) return;
  const int warp = gt >> 5, lane = tid & 31, n_warps = kAll / 32;
  const int col_blocks = (int)((p.max_blocks + 31) / 32);
  if (overlap) {
    // some source row is overwritten: keep the sources first
    for (int64_t t = warp; t < (int64_t)p.n * col_blocks; t += n_warps) {
      const int i = (int)(t / col_blocks), c = (int)(t % col_blocks) * 32 + lane;
      if (c < blocks_of(slen[i], p.block)) p.rows[(int64_t)i * p.max_blocks + c] = p.table[src[i] * p.max_blocks + c];
    }
    cl.sync();
  }
  // eight pairs per task: the entries of one source that follow each other
  // raise a page's count once
  constexpr int kPairs = 8;
  const int groups = (p.n + kPairs - 1) / kPairs;
  for (int64_t t = warp; t < (int64_t)groups * col_blocks; t += n_warps) {
    const int i0 = (int)(t / col_blocks) * kPairs, c = (int)(t % col_blocks) * 32 + lane;
    int now[kPairs], old[kPairs];
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
      const int i = i0 + k;
      now[k] = old[k] = -1;
      if (i >= p.n || (p.src && src[i] == dst[i])) continue;
      if (c < blocks_of(slen[i], p.block))
        now[k] = overlap ? p.rows[(int64_t)i * p.max_blocks + c] : p.table[src[i] * p.max_blocks + c];
      if (c < blocks_of(dlen[i], p.block)) old[k] = p.table[dst[i] * p.max_blocks + c];
    }
    int page = -1, count = 0;
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
      const int i = i0 + k;
      if (i >= p.n || (p.src && src[i] == dst[i])) continue;
      const int nb = blocks_of(slen[i], p.block), ob = blocks_of(dlen[i], p.block);
      if (c < nb || c < ob) p.table[dst[i] * p.max_blocks + c] = c < nb ? now[k] : -1;
      if (c < nb) {
        if (now[k] != page) {
          if (count) atomicAdd(p.refs + page, count);
          page = now[k];
          count = 0;
        }
        if (page >= 0 && page < p.n_pages)
          ++count;
        else
          raise_status(p.status, kInvalid, 402);
      }
      if (c < ob) {
        if (old[k] >= 0 && old[k] < p.n_pages)
          atomicSub(p.refs + old[k], 1);
        else
          raise_status(p.status, kInvalid, 402);
      }
    }
    if (count) atomicAdd(p.refs + page, count);
  }
  if (cl.block_rank() == 0)
    for (int i = tid; i < p.n; i += kThreads) p.seqlens[dst[i]] = slen[i];
}

// ------------------------------------------------------------------ grow

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads, 1) pages_grow_kernel(const PagesParams p) {
  cg::cluster_group cl = cg::this_cluster();
  cl.barrier_arrive();  // waited for before the first write into another CTA's shared memory
  extern __shared__ int sm[];
  const int B = (int)p.batch;
  int* shared_page = sm;       // [B] the shared last page that the sequence would write into, or -1
  int* first = sm + B;         // [B] index of its first new page; bit 31: the first is a copy
  __shared__ int buf[33], totals[kCtas], bad;
  const int tid = threadIdx.x, rank = (int)cl.block_rank(), gt = rank * kThreads + tid;
  // free pages of this thread's range
  const int64_t seg = (p.n_pages + kAll - 1) / kAll;
  const int64_t p0 = min(p.n_pages, gt * seg), p1 = min(p.n_pages, p0 + seg);
  int mine = 0;
  for (int64_t i = p0; i < p1; ++i) mine += p.refs[i] == 0;
  if (tid == 0) bad = 0;
  int cta_total;
  const int before = block_scan(mine, buf, &cta_total);
  cl.barrier_wait();
  publish(cl, totals, cta_total);
  // what each sequence needs (every CTA computes all of them)
  for (int b = tid; b < B; b += kThreads) {
    const int len = p.seqlens[b], n = p.n_new[b];
    int page = -1;
    if (n < 0 || len < 0 || (int64_t)len + max(n, 0) > p.max_blocks * p.block) {
      bad = kInvalid;
    } else if (n > 0 && len % p.block) {
      page = p.table[b * p.max_blocks + len / p.block];
      if (page < 0 || page >= p.n_pages) {
        bad = kInvalid;
        page = -1;
      } else if (p.refs[page] <= 1) {
        page = -1;
      }
    }
    shared_page[b] = page;
  }
  __syncthreads();
  int need_all = 0;
  const int per = (B + kThreads - 1) / kThreads;
  {
    int need = 0;
    const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
    for (int b = b0; b < b1; ++b) {
      int copy = 0;
      const int page = shared_page[b];
      if (page >= 0) {
        // all holders that grow take a copy, in order, but the last one left
        int earlier = 0;
        for (int x = 0; x < b; ++x) earlier += shared_page[x] == page;
        copy = earlier < p.refs[page] - 1;
      }
      const int len = p.seqlens[b];
      const int add = bad ? 0 : blocks_of((int64_t)len + p.n_new[b], p.block) - blocks_of(len, p.block);
      first[b] = need | (copy << 31);
      need += add + copy;
    }
    const int base = block_scan(need, buf, &need_all);
    for (int b = b0; b < b1; ++b) first[b] = (first[b] & 0x80000000) | ((first[b] & 0x7fffffff) + base);
  }
  cl.sync();  // totals are in; every CTA has read the state
  int free_before = before, free_all = 0;
  for (int r = 0; r < kCtas; ++r) {
    if (r < rank) free_before += totals[r];
    free_all += totals[r];
  }
  const int code = bad ? bad : need_all > free_all ? kNoPages : 0;
  if (gt == 0) {
    p.status->code = code;
    p.status->detail = code ? 411 : 0;
  }
  if (code) {
    for (int b = gt; b < B; b += kAll) p.copy_src[b] = p.copy_dst[b] = -1;
    return;
  }
  if (free_before < need_all)
    for (int64_t i = p0; i < p1 && free_before < need_all; ++i)
      if (p.refs[i] == 0) {
        p.list[free_before++] = (int)i;
        p.refs[i] = 1;
      }
  cl.sync();
  // one warp per sequence
  for (int b = gt >> 5; b < B; b += kAll / 32) {
    const int lane = tid & 31, len = p.seqlens[b], n = p.n_new[b];
    const bool copy = first[b] < 0;
    const int at = first[b] & 0x7fffffff;
    const int nb0 = blocks_of(len, p.block), nb1 = blocks_of((int64_t)len + n, p.block);
    for (int c = nb0 + lane; c < nb1; c += 32) p.table[b * p.max_blocks + c] = p.list[at + copy + c - nb0];
    if (lane == 0) {
      p.copy_src[b] = copy ? shared_page[b] : -1;
      p.copy_dst[b] = copy ? p.list[at] : -1;
      if (copy) {
        p.table[b * p.max_blocks + nb0 - 1] = p.list[at];
        atomicSub(p.refs + shared_page[b], 1);
      }
    }
    __syncwarp();
    if (lane == 0) p.seqlens[b] = len + n;
  }
}

// ------------------------------------------------------------------ compact

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads, 1) pages_compact_kernel(const PagesParams p) {
  cg::cluster_group cl = cg::this_cluster();
  cl.barrier_arrive();  // waited for before the first write into another CTA's shared memory
  __shared__ int buf[33], totals[kCtas], holes_at;
  const int tid = threadIdx.x, rank = (int)cl.block_rank(), gt = rank * kThreads + tid;
  const int64_t seg = (p.n_pages + kAll - 1) / kAll;
  const int64_t p0 = min(p.n_pages, gt * seg), p1 = min(p.n_pages, p0 + seg);
  int mine = 0;
  for (int64_t i = p0; i < p1; ++i) mine += p.refs[i] > 0;
  if (tid == 0) holes_at = 0;
  int cta_total;
  int live = block_scan(mine, buf, &cta_total);
  cl.barrier_wait();
  publish(cl, totals, cta_total);
  if (gt == 0) p.status->code = p.status->detail = 0;
  cl.sync();
  int held = 0;
  for (int r = 0; r < kCtas; ++r) {
    if (r < rank) live += totals[r];
    held += totals[r];
  }
  // free pages below `held`, told by the thread that owns page `held`
  if (held >= p0 && held < p1) {
    int l = live;
    for (int64_t i = p0; i < held; ++i) l += p.refs[i] > 0;
    for (int r = 0; r < kCtas; ++r) *cl.map_shared_rank(&holes_at, r) = held - l;
  }
  cl.sync();
  const int moves = held < p.n_pages ? holes_at : 0;
  const int stay = held - moves;  // pages held below `held`
  {
    int l = live;
    for (int64_t i = p0; i < p1; ++i) {
      const int r = p.refs[i];
      if (r <= 0 && i < held) p.move_dst[i - l] = (int)i;
      if (r > 0 && i >= held) {
        p.move_src[l - stay] = (int)i;
        p.aux[l - stay] = r;
      }
      l += r > 0;
    }
    for (int64_t i = moves + gt; i < p.n_pages / 2; i += kAll) p.move_src[i] = p.move_dst[i] = -1;
    if (gt == 0) {
      p.info[0] = moves;
      p.info[1] = held;
    }
  }
  cl.sync();
  {
    int l = live;
    for (int64_t i = p0; i < p1; ++i) {
      const int r = p.refs[i];
      const bool tail = r > 0 && i >= held;
      p.list[i] = tail ? p.move_dst[l - stay] : (int)i;
      p.refs_out[i] = i >= held ? 0 : r > 0 ? r : p.aux[i - l];
      l += r > 0;
    }
  }
  cl.sync();
  for (int64_t t = gt; t < p.batch * p.max_blocks; t += kAll) {
    const int b = (int)(t / p.max_blocks);
    const int64_t c = t - b * p.max_blocks;
    const int page = p.table[t];
    int to = page;
    if (c < blocks_of(p.seqlens[b], p.block)) {
      if (page >= 0 && page < p.n_pages)
        to = p.list[page];
      else
        raise_status(p.status, kInvalid, 421);
    }
    p.table_out[t] = to;
  }
}

// ------------------------------------------------------------------ copy

// Bound by HBM: each byte read once and written once.  A CTA moves 16 KB of
// one page of one pool, four independent 16-byte loads per thread before the
// stores.
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;
constexpr int kCopyChunk = kCopyThreads * kCopyUnroll * 16;

__global__ void __launch_bounds__(kCopyThreads)
    pages_copy_kernel(const __grid_constant__ PageCopyParams p, int chunks) {
  const int64_t entry = blockIdx.x / chunks;
  const int chunk = blockIdx.x % chunks;
  const PagePool& pool = p.pool[blockIdx.y];
  const int s = p.src[entry], d = p.dst[entry];
  if (s < 0 || d < 0 || s >= pool.n_pages || d >= pool.n_pages || s == d) return;
  const uint32_t run = (uint32_t)p.run, total = run * p.rows * p.heads;
  const char* from = pool.data + s * pool.page_stride;
  char* to = pool.data + d * pool.page_stride;
  uint4 v[kCopyUnroll];
  int64_t at[kCopyUnroll];
#pragma unroll
  for (int k = 0; k < kCopyUnroll; ++k) {
    const uint32_t x = (uint32_t)chunk * kCopyChunk + (k * kCopyThreads + threadIdx.x) * 16;
    at[k] = -1;
    if (x < total) {
      const uint32_t r = x / run;
      at[k] = (r / p.heads) * pool.row_stride + (r % p.heads) * pool.head_stride + (x - r * run);
      v[k] = *reinterpret_cast<const uint4*>(from + at[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < kCopyUnroll; ++k)
    if (at[k] >= 0) *reinterpret_cast<uint4*>(to + at[k]) = v[k];
}

// `rows` rows of `row` bytes of shared memory.  The kernel's limit is state that
// all host threads share, so it is always set to that of the largest call: set
// to each call's own size, another thread's smaller one could come between it
// and the launch, which then failed.
cudaError_t launch(void (*kern)(const PagesParams), int64_t rows, int row, const PagesParams& p, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  const size_t smem = (size_t)rows * row;
  if (smem > 40 * 1024)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxPageSlots * row);
  if (e != cudaSuccess) return e;
  kern<<<kCtas, kThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_pages_fork(const PagesParams& p, cudaStream_t stream) {
  return launch(pages_fork_kernel, p.n, 16, p, stream);
}
cudaError_t launch_pages_grow(const PagesParams& p, cudaStream_t stream) {
  return launch(pages_grow_kernel, p.batch, 8, p, stream);
}
cudaError_t launch_pages_compact(const PagesParams& p, cudaStream_t stream) {
  return launch(pages_compact_kernel, 0, 0, p, stream);
}

static int64_t copy_chunks(const PageCopyParams& p) {
  return (p.run * p.rows * p.heads + kCopyChunk - 1) / kCopyChunk;
}

bool pages_copy_fits(const PageCopyParams& p) { return p.n <= 0x7fffffff / copy_chunks(p); }

cudaError_t launch_pages_copy(const PageCopyParams& p, cudaStream_t stream) {
  const int64_t chunks = copy_chunks(p);
  pages_copy_kernel<<<dim3((unsigned)(chunks * p.n), p.n_pools), kCopyThreads, 0, stream>>>(p, (int)chunks);
  return cudaGetLastError();
}

}  // namespace dash
