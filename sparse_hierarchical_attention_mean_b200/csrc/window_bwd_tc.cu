// Sliding-window (and dense causal) attention backward on the 5th-generation
// tensor cores, f16 / bf16.  With p_ij = 2^(s_ij log2e - lse2_i) (lse2: the
// forward's log-sum-exp in log2 units) and D_i = dout_i . out_i:
//   dS_ij = p_ij (dout_i . v_j - D_i)
//   dq_i = sum_j dS_ij k_j / sqrt(d),  dk_j = sum_i dS_ij q_i / sqrt(d),
//   dv_j = sum_i p_ij dout_i  (dk, dv over the heads of the group too)
// Two kernels, so that every gradient element has one writer and the result
// does not depend on timing; S and dP are computed in both (7 products
// instead of 5).  Tiles of rows are 128 = (128 / G positions) x (G heads).
// p and dS are rounded to the input type as operands of the second products;
// where the call's window and sinks are at most kFewKeys keys, whose roundings
// hardly average out, dq's product takes dS as the sum of two such values (the
// first rows of other calls see as few and do without; window 4: dq's error is
// 1.5 times that of rounding dq alone without, 1.1 with; the second product
// costs the row kernel a third of its time on long windows, nothing that shows
// on short ones).  f16 operands are scaled by powers of two into their type's
// range (Range below).  Everything else is fp32.  Every wait is bounded; on expiry the status word
// reads DASH_ERR_DEVICE_TIMEOUT and the roles wind down.
#include <cuda.h>

#include <algorithm>
#include <type_traits>

#include "window_tc.cuh"

namespace dash {
namespace {

constexpr int kRows = 128;
constexpr int kThreads = 320;
constexpr int kWorkers = 256;  // warps 0-7
constexpr int kProducerWarp = 8, kMmaWarp = 9;
constexpr int kTimeout = 5;  // DASH_ERR_DEVICE_TIMEOUT

// ------------------------------------------------------------------ f16: the range of dS and P
//
// dS is as small as dout and as large as dout times v, and f16 spans 2^-24 ..
// 2^16: a dout of 2^12 made dS overflow where the gradients can be held, one of
// 2^-10 over 2048 keys left it 7 bits.  So dS is scaled by a power of two c per
// sequence and KV head, undone at the end:
//   |dS_ij| <= p_ij (|dout_i . v_j| + |D_i|) <= 2 m,  m = max |dout_i| max |v_j|
// (D_i is a mean of dout_i . v_j), and 2^14 <= 2 m c <= 2^15, which leaves a
// factor of two for an out with errors.  Half a step of what is below f16's
// normal numbers is then 2^-25 / c <= 2^-38 m.  P, as an operand of dv, is at
// most 1 and scaled by 2^10.  A kernel takes the maxima first: it reads dout
// and v once more, 33 us of the backward's 1200 for 16K tokens of 32 / 8 heads
// of 128 (5 TB/s), 3 of 33 for 2 x 513 of 8 / 2 heads of 64.
template <typename T>
constexpr bool kScaled = std::is_same<T, __half>::value;
constexpr float kLog2P = 10.f, kScaleP = 1024.f;

// What a lane of a warp read of a KV head's maxima (squared norms as bits: they
// order like the floats, NaN above all).
struct Range {
  uint32_t dout, v;
  __device__ void ask(const WindowParams& p, int b, int g, int lane) {
    dout = v = 0u;
    const float2* r = p.range + (int64_t)(b * p.Hkv + g) * p.n_range;
#pragma unroll
    for (int i = 0; i < kMaxRange; i += 32)
      if (i + lane < p.n_range) {
        const float2 x = r[i + lane];
        dout = max(dout, __float_as_uint(x.x));
        v = max(v, __float_as_uint(x.y));
      }
  }
  __device__ float scale() const {
    const float m2 = __uint_as_float(__reduce_max_sync(0xffffffffu, dout)) *
                     __uint_as_float(__reduce_max_sync(0xffffffffu, v));
    if (!(m2 > 0.f && m2 < -kNegInf)) return 1.f;  // all zeros, or not finite
    const int e = (int)(__float_as_uint(m2) >> 23) - 127;  // m2 >= 2^e (it is a normal number: f16 squared twice)
    return __uint_as_float((uint32_t)(14 - ((e + 2) >> 1) + 127) << 23);
  }
};

constexpr int kRangeThreads = 256;
template <typename T, int D>
__global__ void __launch_bounds__(kRangeThreads) window_bwd_range_kernel(const WindowParams p) {
  constexpr int kLanes = D / 8, kPass = kRangeThreads / kLanes, kAhead = 4;  // 16 bytes a lane
  __shared__ uint32_t top[2];
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const int g = blockIdx.y, b = blockIdx.z, lg = __ffs(p.G) - 1;
  const int row = threadIdx.x / kLanes, col = threadIdx.x % kLanes * 8;
  const int per = (p.S + gridDim.x - 1) / gridDim.x;
  const int pos0 = min((int)blockIdx.x * per, p.S), pos1 = min(pos0 + per, window_len(p, b));
  if (threadIdx.x < 2) top[threadIdx.x] = 0u;
  __syncthreads();
  auto largest = [&](const View& t, int head0, int lgh) {  // over the positions' rows of 2^lgh heads
    const T* src = static_cast<const T*>(t.data) + (int64_t)b * t.sb + (int64_t)head0 * t.sh + col;
    const int64_t rows = (int64_t)max(pos1 - pos0, 0) << lgh;
    float mx = 0.f;
    for (int64_t r0 = 0; r0 < rows; r0 += kPass * kAhead) {
      uint4 x[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int64_t r = r0 + u * kPass + row;
        x[u] = r < rows ? *reinterpret_cast<const uint4*>(src + (pos0 + (r >> lgh)) * t.ss +
                                                          (r & ((1 << lgh) - 1)) * t.sh)
                        : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        float f[8], s = 0.f;
        Elt<T>::to_float(x[u], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(f[e], f[e], s);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        // (a NaN stays: as bits it is above every number)
        mx = __uint_as_float(max(__float_as_uint(mx), __float_as_uint(s)));
      }
    }
    return __reduce_max_sync(0xffffffffu, __float_as_uint(mx));
  };
  const uint32_t a = largest(p.dout, g * p.G, lg), v = largest(p.v, g, 0);
  if ((threadIdx.x & 31) == 0) {
    atomicMax(&top[0], a);
    atomicMax(&top[1], v);
  }
  __syncthreads();
  if (threadIdx.x == 0)
    p.range[(int64_t)(b * p.Hkv + g) * p.n_range + blockIdx.x] =
        make_float2(__uint_as_float(top[0]), __uint_as_float(top[1]));
}

// ------------------------------------------------------------------ rows: dq, D
//
// A CTA (one per SM) walks 128-row tiles; per tile the keys its rows see come
// in steps of 128 (at most one step of sinks before the band, then the band).
//   S = Q K^T, dP = dout V^T   A = Q, dout from TMEM
//   dS over dP in 16 bits;  dQ += dS K  (A from TMEM, K MN-major)
// Warps 0-7 are the workers (two per TMEM lane quarter, 64 keys each).  S of
// the next step runs as soon as S is in their registers, dP of the next step
// behind dQ of this one, so that the tensor core works while they do.  The next
// tile's Q, dout and out come by TMA during this one (out through the ring);
// D is formed while the last dQ runs, Q and dout are moved to TMEM before this
// tile's dq is written, so the next tile's first products overlap that.  Warp 8
// is the TMA producer, which also clears K rows behind a sequence's end; warp 9
// issues the MMAs.  TMEM: Q at 0, dout at D / 2, S, dP, dQ at 128, 256, 384.
// D is dout . out and has out's rounding in it, unless `rest` brings what that
// took.  The sum of a row's dS, which an exact D makes 0, is D's error: the key
// kernel gets the corrected D.
// (Steps of 64 keys in two buffers were slower: a 128 x 64 product takes the
// tensor core 55 clocks, not 32, and S, dP and dQ of 64 keys 1100.  So were 16
// workers of 32 keys, here and in the key kernel: 1.09 against 0.97 ms together
// at 16K tokens, window 1024.)
constexpr int kFewKeys = 16;
constexpr uint32_t kColSR = 128, kColDPR = 256, kColDQ = 384;

template <int D>
struct RowLayout {
  static constexpr int KC = D / 64;
  static constexpr int kChunk = 128 * 128, kTile = KC * kChunk;
  static constexpr int kStages = D == 128 ? 5 : 10;  // out, K and V tiles in flight
  static constexpr int kOffQ = 0, kOffDo = kTile;
  static constexpr int kOffRing = 2 * kTile;
  static constexpr int kOffBar = kOffRing + kStages * kTile;
  // exchange between the halves of the workers: [2][128] their halves of D,
  // [2][128] half 1's sum of a row's dS, of even and of odd items
  static constexpr int kOffXch = kOffBar + 512;
  static constexpr int kAlloc = kOffXch + 4 * kRows * 4;
};

struct RowBars {
  uint64_t rows_full, rows_empty;  // Q, dout in shared memory
  uint64_t stats;                  // both halves of D exchanged, out read
  uint64_t sums;                   // both halves of the sums of dS
  uint64_t ready;                  // Q and dout in TMEM
  uint64_t full[10], empty[10];
  uint64_t tail;
  uint64_t s_full, s_free, dp_full, ds_full;
  uint64_t dq_full, dq_empty;
  uint64_t drained;
  uint32_t tmem_base;
};

struct RowItem {
  int b, g, tile, pos0, n, steps;
  KeyTiles kt;
  __device__ RowItem(const WindowParams& p, int P, const ItemWalk& w)
      : b(w.b),
        g(w.g),
        tile(w.n_x - 1 - w.x),
        pos0(tile * P),
        n(window_len(p, b)),
        kt(pos0, min(pos0 + P, n), p.window, p.sinks, kRows) {
    steps = pos0 < n ? kt.n : 0;
  }
};

template <typename T, int D, bool kFew>
__global__ void __launch_bounds__(kThreads, 1)
    window_bwd_row_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                             const __grid_constant__ CUtensorMap tm_o, const __grid_constant__ CUtensorMap tm_rest,
                             const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                             const WindowParams p) {
  using L = RowLayout<D>;
  constexpr int kStages = L::kStages;
  constexpr bool kBF16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr uint32_t kIdescS = tc::idesc_f16(kRows, kRows, kBF16, false, false);
  constexpr uint32_t kIdescQ = tc::idesc_f16(kRows, D, kBF16, false, true);

  extern __shared__ __align__(1024) uint8_t smem[];
  RowBars* bars = reinterpret_cast<RowBars*>(smem + L::kOffBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lg = __ffs(p.G) - 1, P = kRows >> lg;

  if (threadIdx.x == 0) {
    tc::mbar_init(&bars->rows_full, 1);
    tc::mbar_init(&bars->rows_empty, kWorkers / 32);
    tc::mbar_init(&bars->stats, kWorkers / 32);
    tc::mbar_init(&bars->sums, kWorkers / 32);
    tc::mbar_init(&bars->ready, kWorkers / 32);
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(&bars->full[s], 1);
      tc::mbar_init(&bars->empty[s], 1);
    }
    tc::mbar_init(&bars->tail, 1);
    tc::mbar_init(&bars->s_full, 1);
    tc::mbar_init(&bars->s_free, kWorkers / 32);
    tc::mbar_init(&bars->dp_full, 1);
    tc::mbar_init(&bars->ds_full, kWorkers / 32);
    tc::mbar_init(&bars->dq_full, 1);
    tc::mbar_init(&bars->dq_empty, kWorkers / 32);
    tc::mbar_init(&bars->drained, 1);
    tc::fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(&bars->tmem_base, 512);
    tc::tmem_relinquish();
  }
  if (warp == kProducerWarp && lane == 0) {
    tc::prefetch_tensormap(&tm_q);
    tc::prefetch_tensormap(&tm_do);
    tc::prefetch_tensormap(&tm_o);
    if (p.rest.data) tc::prefetch_tensormap(&tm_rest);
    tc::prefetch_tensormap(&tm_k);
    tc::prefetch_tensormap(&tm_v);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = bars->tmem_base;
  bool ok = true;
  // the key kernel may take the SMs that are or get free; it waits for this
  // grid's end before it reads lse2 and D
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  if constexpr (kScaled<T>) asm volatile("griddepcontrol.wait;\n" ::: "memory");  // the maxima

  // ring tiles of an item: out (and rest), then K and V of each step
  const int n_out = p.rest.data ? 2 : 1;
  if (warp == kProducerWarp) {
    // ------------------------------------------------------------ producer
    if (blockIdx.x == 0) begin_status(p, lane);
    int x = 0, items = 0, tails = 0;
    ItemWalk it(p.n_tiles, p.Hkv, p.B);
    auto seek = [&] {  // the first item with steps
      while (it.any() && RowItem(p, P, it).steps == 0) it.next();
    };
    auto load_rows = [&] {  // Q and dout of an item, when the one before has left their place
      if (items > 0) ok = ok && warp_wait(&bars->rows_empty, items - 1);
      if (!ok) return;
      const RowItem w(p, P, it);
      if (lane == 0) {
        tc::mbar_arrive_expect_tx(&bars->rows_full, 2 * L::kTile);
        for (int kc = 0; kc < L::KC; ++kc) {
          uint8_t* dst = smem + kc * L::kChunk;
          tc::tma_load_4d(dst + L::kOffQ, &tm_q, &bars->rows_full, kc * 64, w.g * p.G, w.pos0, w.b);
          tc::tma_load_4d(dst + L::kOffDo, &tm_do, &bars->rows_full, kc * 64, w.g * p.G, w.pos0, w.b);
        }
      }
      ++items;
    };
    seek();
    if (it.any()) load_rows();
    while (ok && it.any()) {
      const RowItem w(p, P, it);
      it.next();
      seek();
      for (int i = 0; ok && i < n_out + 2 * w.steps; ++i, ++x) {
        const int st = x % kStages;
        if (x >= kStages) ok = warp_wait(&bars->empty[st], x / kStages - 1);
        if (!ok) break;
        uint8_t* dst = smem + L::kOffRing + st * L::kTile;
        const int y = i - n_out;  // K of step y / 2, V of it
        const int tok0 = y >= 0 ? w.kt.tile(y >> 1) * kRows : 0;
        const bool is_k = y >= 0 && !(y & 1);
        const bool clear = is_k && tok0 + kRows > w.n && w.n < p.S;
        uint64_t* bar = clear ? &bars->tail : &bars->full[st];
        if (lane == 0) {
          tc::mbar_arrive_expect_tx(bar, L::kTile);
          for (int kc = 0; kc < L::KC; ++kc) {
            if (y < 0)
              tc::tma_load_4d(dst + kc * L::kChunk, i == 0 ? &tm_o : &tm_rest, bar, kc * 64, w.g * p.G, w.pos0, w.b);
            else
              tc::tma_load_4d(dst + kc * L::kChunk, is_k ? &tm_k : &tm_v, bar, kc * 64, w.g, tok0, w.b);
          }
        }
        if (clear) {
          // dS is 0 there, but 0 x NaN is not
          ok = warp_wait(&bars->tail, tails++);
          zero_tile_rows(dst, L::KC, kRows, w.n - tok0, lane);
          if (lane == 0) tc::mbar_arrive(&bars->full[st]);
        }
        // the next item's rows, once this one's ring is filled
        if (i == min(4, n_out + 2 * w.steps - 1) && it.any()) load_rows();
      }
    }
    // every copy lands before the CTA retires
    if (items > 0) tc::mbar_wait(&bars->rows_full, (items - 1) & 1);
    for (int j = max(0, x - kStages); j < x; ++j) tc::mbar_wait(&bars->full[j % kStages], (j / kStages) & 1);
    if (!ok) raise_status(p.status, kTimeout, 331);
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    auto wait = [&](uint64_t* bar, int phase) {
      ok = ok && warp_wait(bar, phase);
      tc::fence_after_sync();
      return ok;
    };
    const uint64_t r0 = tc::smem_desc_sw128(smem + L::kOffRing, 16, 1024);
    const uint64_t rmn0 = tc::smem_desc_sw128(smem + L::kOffRing, L::kChunk, 1024);
    auto at = [&](int x) { return (uint64_t)(((x % kStages) * L::kTile) >> 4); };
    // S or dP: A from TMEM, B = the ring tile x
    auto issue = [&](uint32_t dst, uint32_t a, int x, uint64_t* bar) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        tc::mma_f16_ts_w(tmem + dst, tmem + a + k * 8,
                         r0 + at(x) + (uint64_t)((((k >> 2) * L::kChunk) + (k & 3) * 32) >> 4), kIdescS,
                         k > 0 ? 1u : 0u);
      tc::mma_commit_w(bar);
    };
    int x = 0, items = 0, step = 0;  // x: the item's first ring tile (out)
    for (ItemWalk it(p.n_tiles, p.Hkv, p.B); ok && it.any(); it.next()) {
      const RowItem w(p, P, it);
      if (w.steps == 0) continue;
      auto s_of = [&](int i) {
        const int k = x + n_out + 2 * i;
        if (wait(&bars->full[k % kStages], k / kStages)) issue(kColSR, 0, k, &bars->s_full);
      };
      auto dp_of = [&](int i) {
        const int v = x + n_out + 1 + 2 * i;
        if (!wait(&bars->full[v % kStages], v / kStages)) return;
        issue(kColDPR, D / 2, v, &bars->dp_full);
        tc::mma_commit_w(&bars->empty[v % kStages]);
      };
      if (!wait(&bars->ready, items)) break;
      s_of(0);
      if (ok) dp_of(0);
      for (int i = 0; ok && i < w.steps; ++i) {
        const int k = x + n_out + 2 * i;
        if (!wait(&bars->s_free, step + i)) break;
        if (i + 1 < w.steps) s_of(i + 1);
        if (i == 0 && items > 0) wait(&bars->dq_empty, items - 1);
        if (!ok || !wait(&bars->ds_full, step + i)) break;
        // dQ += dS K: keys 0-63 of the operand packed at dP's column 0, 64-127
        // at its column 64, low parts 32 columns further
#pragma unroll 1
        for (int low = 0; low <= (kFew ? 1 : 0); ++low)
#pragma unroll
          for (int kk = 0; kk < kRows / 16; ++kk)
            tc::mma_f16_ts_w(tmem + kColDQ, tmem + kColDPR + (kk >> 2) * 64 + low * 32 + (kk & 3) * 8,
                             rmn0 + at(k) + (uint64_t)((kk * 2048) >> 4), kIdescQ,
                             (i > 0 || kk > 0 || low > 0) ? 1u : 0u);
        if (i == w.steps - 1) tc::mma_commit_w(&bars->dq_full);
        tc::mma_commit_w(&bars->empty[k % kStages]);
        if (i + 1 < w.steps) dp_of(i + 1);
      }
      if (!ok) break;
      x += n_out + 2 * w.steps;
      step += w.steps;
      ++items;
    }
    if (!ok) raise_status(p.status, kTimeout, 332);
    tc::mma_commit_w(&bars->drained);
    tc::mbar_wait(&bars->drained, 0);
  } else {
    // ------------------------------------------------------------ workers
    const int half = warp >> 2, q4 = warp & 3, r = q4 * 32 + lane;
    const uint32_t tb = tmem + ((uint32_t)(q4 * 32) << 16);
    const uint32_t s_tm = tb + kColSR + half * 64, d_tm = tb + kColDPR + half * 64;
    const float sc = rsqrtf((float)D) * kLog2e;
    float* xch = reinterpret_cast<float*>(smem + L::kOffXch) + r;
    float nlse2 = 0.f, ndd = 0.f;  // -lse2 and -D of the current item's row
    float lse_next = 0.f;          // the next item's log-sum-exp
    [[maybe_unused]] Range range_next;
    [[maybe_unused]] float ds_scale = 1.f;  // c of the current item; D is kept times c
    int x = 0, items = 0, step = 0;

    // on to the first item with steps; tiles behind the sequence's end get
    // dq = 0 and lse2 = inf (p = 0) on the way
    auto seek = [&](ItemWalk& it) {
      for (; it.any(); it.next()) {
        const RowItem w(p, P, it);
        if (w.steps > 0) break;
        const int pos = w.pos0 + (r >> lg), head = w.g * p.G + (r & (p.G - 1));
        if (half == 0) {
          const int64_t at = ((int64_t)(w.b * p.Hkv + w.g) * p.n_tiles + w.tile) * kRows + r;
          p.nlse2[at] = kNegInf;
          p.ndd[at] = 0.f;
        } else if (pos < p.S) {
          T* dst = static_cast<T*>(const_cast<void*>(p.dq.data)) + (int64_t)w.b * p.dq.sb + (int64_t)pos * p.dq.ss +
                   (int64_t)head * p.dq.sh;
#pragma unroll
          for (int e = 0; e < D / 8; ++e) *reinterpret_cast<uint4*>(dst + e * 8) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
    };
    // the log-sum-exp of an item's row, asked for one item ahead
    auto ask_lse = [&](const ItemWalk& it) {
      const RowItem w(p, P, it);
      const int pos = w.pos0 + (r >> lg), head = w.g * p.G + (r & (p.G - 1));
      if (pos < w.n) lse_next = p.lse[((int64_t)w.b * p.H + head) * p.S + pos];
      if constexpr (kScaled<T>) range_next.ask(p, w.b, w.g, lane);
    };
    // lse2 and D = dout . out of an item's row: each half takes half of the
    // columns
    auto row_stats = [&](const ItemWalk& it) {
      const RowItem w(p, P, it);
      const bool live = w.pos0 + (r >> lg) < w.n;
      nlse2 = live ? -lse_next * kLog2e : kNegInf;
      ok = warp_wait(&bars->rows_full, items) && ok;
      for (int y = x; y < x + n_out; ++y) ok = warp_wait(&bars->full[y % kStages], y / kStages) && ok;
      const uint8_t* po = smem + L::kOffRing + (x % kStages) * L::kTile + r * 128;
      const uint8_t* pr = smem + L::kOffRing + ((x + 1) % kStages) * L::kTile + r * 128;
      const uint8_t* pd = smem + L::kOffDo + r * 128;
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int v = 0; v < D / 16; ++v) {
        const int e = half * (D / 16) + v;  // 16-byte piece of the row
        const int at = (e >> 3) * L::kChunk + (((e & 7) ^ (r & 7)) << 4);
        float fd[8], fo[8];
        Elt<T>::to_float(*reinterpret_cast<const uint4*>(pd + at), fd);
        Elt<T>::to_float(*reinterpret_cast<const uint4*>(po + at), fo);
#pragma unroll
        for (int e2 = 0; e2 < 8; ++e2) acc[e2 & 3] = fmaf(fd[e2], fo[e2], acc[e2 & 3]);
        if (n_out > 1) {
          Elt<T>::to_float(*reinterpret_cast<const uint4*>(pr + at), fo);
#pragma unroll
          for (int e2 = 0; e2 < 8; ++e2) acc[e2 & 3] = fmaf(fd[e2], fo[e2], acc[e2 & 3]);
        }
      }
      const float mine = (acc[0] + acc[1]) + (acc[2] + acc[3]);
      xch[half * kRows] = mine;
      warp_arrive(&bars->stats, lane);
      ok = warp_wait(&bars->stats, items) && ok;
      const float a = half == 0 ? mine : xch[0], b = half == 0 ? xch[kRows] : mine;
      if constexpr (kScaled<T>) ds_scale = range_next.scale();
      ndd = live ? -(a + b) * ds_scale : 0.f;  // the same sum in both halves
      if (threadIdx.x == 0)  // every worker has read out
        for (int y = x; y < x + n_out; ++y) tc::mbar_arrive(&bars->empty[y % kStages]);
    };
    // Q (half 0) and dout (half 1) into TMEM
    auto rows_to_tmem = [&] {
      const uint8_t* src = smem + (half == 0 ? L::kOffQ : L::kOffDo) + r * 128;
#pragma unroll
      for (int cc = 0; cc < L::KC; ++cc) {
        uint32_t w32[32];
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          const uint4 t = *reinterpret_cast<const uint4*>(src + cc * L::kChunk + ((v ^ (r & 7)) << 4));
          w32[4 * v] = t.x, w32[4 * v + 1] = t.y, w32[4 * v + 2] = t.z, w32[4 * v + 3] = t.w;
        }
        tc::tmem_st32(tb + half * (D / 2) + cc * 32, w32);
      }
      tc::tmem_wait_st();
      tc::fence_before_sync();
      warp_arrive(&bars->rows_empty, lane);
      warp_arrive(&bars->ready, lane);
    };

    ItemWalk it(p.n_tiles, p.Hkv, p.B);
    seek(it);
    if (it.any()) {
      ask_lse(it);
      row_stats(it);
      if (ok) rows_to_tmem();
    }
    for (bool more = it.any(); ok && more;) {
      const RowItem w(p, P, it);
      it.next();
      seek(it);
      more = it.any();
      if (more) ask_lse(it);
      const int pos = w.pos0 + (r >> lg);
      const int lo = pos - p.window + 1;
      // the warp's rows: first and last position
      const int pos_a = w.pos0 + ((q4 * 32) >> lg), pos_b = w.pos0 + ((q4 * 32 + 31) >> lg);
      const float row_nlse2 = nlse2, row_ndd = ndd, row_scale = ds_scale;
      float2 ds_sum = make_float2(0.f, 0.f);
      for (int i = 0; i < w.steps; ++i) {
        const int y = step + i, key0 = w.kt.tile(i) * kRows + half * 64;  // the warp's keys [key0, key0 + 64)
        // none of the warp's pairs is visible, or all are
        const bool none = key0 > pos_b || (key0 + 63 < pos_a - p.window + 1 && key0 >= p.sinks);
        const bool all = key0 + 63 <= pos_a && key0 >= pos_b - p.window + 1;
        if (!(ok = warp_wait(&bars->s_full, y))) break;
        tc::fence_after_sync();
        uint32_t pf[64];
        tc::tmem_ld32(s_tm, pf);
        tc::tmem_ld32(s_tm + 32, pf + 32);
        tc::tmem_wait_ld();
        tc::fence_before_sync();
        warp_arrive(&bars->s_free, lane);
        if (!none) {
          const float2 sc2 = make_float2(sc, sc), off2 = make_float2(nlse2, nlse2);
          auto scaled = [&](int j) {
            return __ffma2_rn(make_float2(__uint_as_float(pf[2 * j]), __uint_as_float(pf[2 * j + 1])), sc2, off2);
          };
          float2 a = scaled(0), b = scaled(1);
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            float2 c = a, e = b;
            pf[2 * j] = __float_as_uint(ex2_placed(a.x));
            if (j + 2 < 32) c = scaled(j + 2);
            pf[2 * j + 1] = __float_as_uint(ex2_placed(a.y));
            pf[2 * j + 2] = __float_as_uint(ex2_placed(b.x));
            if (j + 2 < 32) e = scaled(j + 3);
            pf[2 * j + 3] = __float_as_uint(ex2_placed(b.y));
            a = c;
            b = e;
          }
        }
        if (!(ok = warp_wait(&bars->dp_full, y))) break;
        tc::fence_after_sync();
        const float2 nd2 = make_float2(ndd, ndd);
        [[maybe_unused]] const float2 c2 = make_float2(ds_scale, ds_scale);
        [[maybe_unused]] uint32_t low[2][16];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t dw[16];
          if (none) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              dw[j] = 0u;
              if constexpr (kFew) low[c][j] = 0u;
            }
          } else {
            uint32_t dv[32];
            tc::tmem_ld32(d_tm + c * 32, dv);
            tc::tmem_wait_ld();
            float2 ds[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const int e = c * 32 + 2 * j;
              const float2 dp = make_float2(__uint_as_float(dv[2 * j]), __uint_as_float(dv[2 * j + 1]));
              ds[j] = __fmul2_rn(make_float2(__uint_as_float(pf[e]), __uint_as_float(pf[e + 1])),
                                 kScaled<T> ? __ffma2_rn(dp, c2, nd2) : __fadd2_rn(dp, nd2));
            }
            if (!all) {
              // hidden pairs are cleared after the products: what they hold may not be finite
              const int t0 = key0 + c * 32;
              const uint32_t seen = bit_range(lo - t0, pos - t0) | bit_range(0, min(pos, p.sinks - 1) - t0);
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                if (!(seen & (1u << (2 * j)))) ds[j].x = 0.f;
                if (!(seen & (2u << (2 * j)))) ds[j].y = 0.f;
              }
            }
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              ds_sum = __fadd2_rn(ds_sum, __fadd2_rn(__fadd2_rn(ds[j], ds[j + 1]), __fadd2_rn(ds[j + 2], ds[j + 3])));
#pragma unroll
              for (int u = 0; u < 4; ++u) dw[j + u] = pack2<T>(ds[j + u].x, ds[j + u].y);
              if constexpr (kFew) {
                float hi[8];
                Elt<T>::to_float(make_uint4(dw[j], dw[j + 1], dw[j + 2], dw[j + 3]), hi);
#pragma unroll
                for (int u = 0; u < 4; ++u)
                  low[c][j + u] = pack2<T>(ds[j + u].x - hi[2 * u], ds[j + u].y - hi[2 * u + 1]);
              }
            }
          }
          tc::tmem_st16(d_tm + c * 16, dw);
        }
        if constexpr (kFew) {  // over columns whose dP has been read
          tc::tmem_st16(d_tm + 32, low[0]);
          tc::tmem_st16(d_tm + 48, low[1]);
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        warp_arrive(&bars->ds_full, lane);
      }
      step += w.steps;
      x += n_out + 2 * w.steps;
      const int item = items++;
      // Half 0 reads half 1's sum after it has let the next item start, and
      // nothing holds that item's workers back when it has one step: the next
      // sum goes to the other slot.  The one after it comes back to this slot
      // only once half 0 has handed over that item's rows, after its read.
      const float my_sum = ds_sum.x + ds_sum.y;
      float* const sum1 = xch + (2 + (item & 1)) * kRows;
      if (half == 1) *sum1 = my_sum;
      warp_arrive(&bars->sums, lane);
      if (more) row_stats(it);  // (while the last dQ runs)
      if (!ok || !(ok = warp_wait(&bars->dq_full, item))) break;
      tc::fence_after_sync();
      if (more) rows_to_tmem();
      // ---- for the key kernel: -lse2 and -D, corrected by the sum of dS
      if (!(ok = warp_wait(&bars->sums, item))) break;
      if (half == 0) {
        const int64_t at = ((int64_t)(w.b * p.Hkv + w.g) * p.n_tiles + w.tile) * kRows + r;
        p.nlse2[at] = row_nlse2 + (kScaled<T> ? kLog2P : 0.f);
        p.ndd[at] = pos < w.n ? (row_ndd - (my_sum + *sum1)) * (kScaled<T> ? 1.f / kScaleP : 1.f) : 0.f;
      }
      // ---- dq of the item, each half of the workers takes half of the columns
      const bool live = pos < w.n;
      T* dst = static_cast<T*>(const_cast<void*>(p.dq.data)) + (int64_t)w.b * p.dq.sb +
               (int64_t)min(pos, p.S - 1) * p.dq.ss + (int64_t)(w.g * p.G + (r & (p.G - 1))) * p.dq.sh;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const int col = (half * (D / 64) + c) * 32;
        uint32_t v[32];
        tc::tmem_ld32(tb + kColDQ + col, v);
        tc::tmem_wait_ld();
        if (!live) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = 0u;
        }
        if (pos < p.S) store_row32(dst + col, v, rsqrtf((float)D) / row_scale, p.wide);
      }
      tc::fence_before_sync();
      warp_arrive(&bars->dq_empty, lane);
    }
    if (!ok) raise_status(p.status, kTimeout, 333);
  }

  tc::fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ keys: dk, dv
//
// A CTA (one per SM) walks items of 128 keys of one KV head; per item it goes
// through the row tiles that see one of the keys, in order:
//   S^T = K Q^T, dP^T = V dout^T     A, B from shared memory
//   P^T over S^T, dS^T over dP^T in 16 bits (lane = key, column = row)
//   dV += P^T dout,  dK += dS^T Q    A from TMEM, B MN-major
// The tensor core's order per tile is dV, S^T of the next tile, dK, dP^T of
// the next tile: while the workers form P^T of a tile it runs dK and dP^T,
// while they form dS^T it runs dV and the next S^T.  TMEM is full: S^T, dP^T,
// dV, dK at 0, 128, 256, 384.  Warps 0-7 are the workers (two per lane
// quarter, 64 rows each; P stays in fp32 registers until dS^T); warp 8 brings
// Q, dout and the rows' lse2 and D (and clears Q and dout rows behind a
// sequence's end), warp 9 issues the MMAs.
//
// The first `sinks` keys are seen by every later row, so the first item of a
// KV head would be S / window times as long as the others: the row tiles past
// its band are split into chunks, items of their own, whose fp32 partials the
// join kernel adds in order.
constexpr uint32_t kColST = 0, kColDPT = 128, kColDV = 256, kColDK = 384;
constexpr int kNS = 2;  // Q / dout stages

template <int D>
struct KeyLayout {
  static constexpr int KC = D / 64;
  static constexpr int kChunk = 128 * 128, kTile = KC * kChunk;
  static constexpr int kOffK = 0, kOffV = kTile;
  static constexpr int kOffQ = 2 * kTile;              // [kNS] Q, dout
  static constexpr int kOffInfo = kOffQ + kNS * 2 * kTile;  // [kNS] -lse2[128], -D[128]
  static constexpr int kOffBar = kOffInfo + kNS * 1024;
  static constexpr int kAlloc = kOffBar + 256 + 1024;
};

struct KeyBars {
  uint64_t kv_full, kv_empty;
  uint64_t q_full[kNS], q_empty[kNS];
  uint64_t tail;
  uint64_t s_full, dp_full, p_full[2], ds_full;
  uint64_t acc_full, acc_empty;
  uint64_t drained;
  uint32_t tmem_base;
};

struct KeyItem {
  int b, g, k0, slot, n, t0, t1;  // keys from k0; partial slot, -1: final; row tiles [t0, t1)
  __device__ KeyItem(const WindowParams& p, int lgp, const ItemWalk& w) : b(w.b), g(w.g), n(window_len(p, b)) {
    if (w.x < p.n_chunks) {
      // the band's row tiles of key tile 0 end before these
      const int first_far = (min(p.S - 1, kRows + p.window - 2) >> lgp) + 1;
      k0 = 0;
      slot = 1 + w.x;
      t0 = first_far + w.x * p.chunk_tiles;
      t1 = min(t0 + p.chunk_tiles, (n + (1 << lgp) - 1) >> lgp);
    } else {
      k0 = (w.x - p.n_chunks) * kRows;
      slot = k0 == 0 && p.n_chunks > 0 ? 0 : -1;
      t0 = k0 >> lgp;
      // the last row that sees a key of the tile
      t1 = k0 < n ? ((int)min((int64_t)n - 1, (int64_t)k0 + kRows - 1 + p.window - 1) >> lgp) + 1 : t0;
    }
    t1 = max(t1, t0);
  }
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    window_bwd_key_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                             const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                             const WindowParams p, int n_x) {
  using L = KeyLayout<D>;
  constexpr bool kBF16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr uint32_t kIdescS = tc::idesc_f16(kRows, kRows, kBF16, false, false);
  constexpr uint32_t kIdescKV = tc::idesc_f16(kRows, D, kBF16, false, true);

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  KeyBars* bars = reinterpret_cast<KeyBars*>(smem + L::kOffBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lg = __ffs(p.G) - 1, lgp = 7 - lg, P = 1 << lgp;  // positions of a row tile

  if (threadIdx.x == 0) {
    tc::mbar_init(&bars->kv_full, 1);
    tc::mbar_init(&bars->kv_empty, 1);
    for (int s = 0; s < kNS; ++s) {
      tc::mbar_init(&bars->q_full[s], 1);
      tc::mbar_init(&bars->q_empty[s], 1 + kWorkers / 32);
    }
    tc::mbar_init(&bars->tail, 1);
    tc::mbar_init(&bars->s_full, 1);
    tc::mbar_init(&bars->dp_full, 1);
    for (int c = 0; c < 2; ++c) tc::mbar_init(&bars->p_full[c], kWorkers / 32);
    tc::mbar_init(&bars->ds_full, kWorkers / 32);
    tc::mbar_init(&bars->acc_full, 1);
    tc::mbar_init(&bars->acc_empty, kWorkers / 32);
    tc::mbar_init(&bars->drained, 1);
    tc::fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(&bars->tmem_base, 512);
    tc::tmem_relinquish();
  }
  if (warp == kProducerWarp && lane == 0) {
    tc::prefetch_tensormap(&tm_q);
    tc::prefetch_tensormap(&tm_do);
    tc::prefetch_tensormap(&tm_k);
    tc::prefetch_tensormap(&tm_v);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = bars->tmem_base;
  bool ok = true;
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  // the row kernel's lse2 and D; all roles wait here, so that the limits of
  // their own waits do not run while that kernel does
  asm volatile("griddepcontrol.wait;\n" ::: "memory");

  if (warp == kProducerWarp) {
    // ------------------------------------------------------------ producer
    int q = 0, items = 0, tails = 0;
    for (ItemWalk it(n_x, p.Hkv, p.B); ok && it.any(); it.next()) {
      const KeyItem w(p, lgp, it);
      if (w.t0 == w.t1) continue;
      if (items > 0) ok = warp_wait(&bars->kv_empty, items - 1);
      if (!ok) break;
      if (lane == 0) {
        tc::mbar_arrive_expect_tx(&bars->kv_full, 2 * L::kTile);
        for (int kc = 0; kc < L::KC; ++kc) {
          tc::tma_load_4d(smem + L::kOffK + kc * L::kChunk, &tm_k, &bars->kv_full, kc * 64, w.g, w.k0, w.b);
          tc::tma_load_4d(smem + L::kOffV + kc * L::kChunk, &tm_v, &bars->kv_full, kc * 64, w.g, w.k0, w.b);
        }
      }
      ++items;
      for (int t = w.t0; ok && t < w.t1; ++t, ++q) {
        const int st = q % kNS;
        if (q >= kNS) ok = warp_wait(&bars->q_empty[st], q / kNS - 1);
        if (!ok) break;
        uint8_t* dst = smem + L::kOffQ + st * 2 * L::kTile;
        const bool clear = (t + 1) * P > w.n && w.n < p.S;
        uint64_t* bar = clear ? &bars->tail : &bars->q_full[st];
        if (lane == 0) {
          tc::mbar_arrive_expect_tx(bar, 2 * L::kTile + 1024);
          for (int kc = 0; kc < L::KC; ++kc) {
            tc::tma_load_4d(dst + kc * L::kChunk, &tm_q, bar, kc * 64, w.g * p.G, t * P, w.b);
            tc::tma_load_4d(dst + L::kTile + kc * L::kChunk, &tm_do, bar, kc * 64, w.g * p.G, t * P, w.b);
          }
          const int64_t at = ((int64_t)(w.b * p.Hkv + w.g) * p.n_tiles + t) * kRows;
          tc::bulk_load(smem + L::kOffInfo + st * 1024, p.nlse2 + at, 512, bar);
          tc::bulk_load(smem + L::kOffInfo + st * 1024 + 512, p.ndd + at, 512, bar);
        }
        if (clear) {
          // p and dS are 0 there, but 0 x NaN is not
          ok = warp_wait(&bars->tail, tails++);
          const int row0 = (w.n - t * P) * p.G;
          zero_tile_rows(dst, L::KC, kRows, row0, lane);
          zero_tile_rows(dst + L::kTile, L::KC, kRows, row0, lane);
          if (lane == 0) tc::mbar_arrive(&bars->q_full[st]);
        }
      }
    }
    // every copy lands before the CTA retires
    if (items > 0) tc::mbar_wait(&bars->kv_full, (items - 1) & 1);
    for (int j = max(0, q - kNS); j < q; ++j) tc::mbar_wait(&bars->q_full[j % kNS], (j / kNS) & 1);
    if (!ok) raise_status(p.status, kTimeout, 341);
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    auto wait = [&](uint64_t* bar, int phase) {
      ok = ok && warp_wait(bar, phase);
      tc::fence_after_sync();
      return ok;
    };
    const uint64_t kd = tc::smem_desc_sw128(smem + L::kOffK, 16, 1024);
    const uint64_t vd = tc::smem_desc_sw128(smem + L::kOffV, 16, 1024);
    const uint64_t q0 = tc::smem_desc_sw128(smem + L::kOffQ, 16, 1024);
    const uint64_t qmn0 = tc::smem_desc_sw128(smem + L::kOffQ, L::kChunk, 1024);
    auto stage = [&](int x) { return (uint64_t)(((x % kNS) * 2 * L::kTile) >> 4); };
    // S^T or dP^T: contraction over d
    auto issue_ss = [&](uint32_t col, uint64_t a, uint64_t b, uint64_t* bar) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint64_t off = (uint64_t)((((k >> 2) * L::kChunk) + (k & 3) * 32) >> 4);
        tc::mma_f16_ss_w(tmem + col, a + off, b + off, kIdescS, k > 0 ? 1u : 0u);
      }
      tc::mma_commit_w(bar);
    };
    // dV or dK: contraction over the tile's rows, slices of 16; rows 0-63 of
    // the operand are packed at col, rows 64-127 at col + 64 (each worker
    // half's own columns)
    auto issue_ts = [&](uint32_t dst, uint32_t col, uint64_t b, int k, bool first) {
      tc::mma_f16_ts_w(tmem + dst, tmem + col + (k >> 2) * 64 + (k & 3) * 8, b + (uint64_t)((k * 2048) >> 4),
                       kIdescKV, first ? 0u : 1u);
    };
    const uint64_t tile16 = (uint64_t)(L::kTile >> 4);
    int q = 0, items = 0;
    for (ItemWalk it(n_x, p.Hkv, p.B); ok && it.any(); it.next()) {
      const KeyItem w(p, lgp, it);
      if (w.t0 == w.t1) continue;
      const int n = w.t1 - w.t0;
      if (!wait(&bars->kv_full, items) || !wait(&bars->q_full[q % kNS], q / kNS)) break;
      issue_ss(kColST, kd, q0 + stage(q), &bars->s_full);
      issue_ss(kColDPT, vd, q0 + tile16 + stage(q), &bars->dp_full);
      for (int i = 0; i < n; ++i) {
        const int x = q + i;
        if (i == 0 && items > 0 && !wait(&bars->acc_empty, items - 1)) break;
        // the rows of the workers' first 32 columns, then those of the second
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (!wait(&bars->p_full[c], x)) break;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            issue_ts(kColDV, kColST, qmn0 + tile16 + stage(x), (k >> 1) * 4 + c * 2 + (k & 1),
                     i == 0 && c == 0 && k == 0);
        }
        if (!ok) break;
        if (i + 1 < n) {
          if (!wait(&bars->q_full[(x + 1) % kNS], (x + 1) / kNS)) break;
          issue_ss(kColST, kd, q0 + stage(x + 1), &bars->s_full);
        }
        if (!wait(&bars->ds_full, x)) break;
#pragma unroll
        for (int k = 0; k < kRows / 16; ++k)
          issue_ts(kColDK, kColDPT, qmn0 + stage(x), k, i == 0 && k == 0);
        tc::mma_commit_w(&bars->q_empty[x % kNS]);
        if (i + 1 < n) issue_ss(kColDPT, vd, q0 + tile16 + stage(x + 1), &bars->dp_full);
      }
      if (!ok) break;
      tc::mma_commit_w(&bars->kv_empty);
      tc::mma_commit_w(&bars->acc_full);
      q += n;
      ++items;
    }
    if (!ok) raise_status(p.status, kTimeout, 342);
    tc::mma_commit_w(&bars->drained);
    tc::mbar_wait(&bars->drained, 0);
  } else {
    // ------------------------------------------------------------ workers
    const int q4 = warp & 3, half = warp >> 2;
    const int k = q4 * 32 + lane;  // key of the item = TMEM lane
    const uint32_t tb = tmem + ((uint32_t)(q4 * 32) << 16);
    const float sc = rsqrtf((float)D) * kLog2e;
    int q = 0, items = 0;
    for (ItemWalk it(n_x, p.Hkv, p.B); ok && it.any(); it.next()) {
      const KeyItem w(p, lgp, it);
      const int key = w.k0 + k;
      [[maybe_unused]] float ds_scale = 1.f;
      if constexpr (kScaled<T>) {
        Range range;
        range.ask(p, w.b, w.g, lane);
        ds_scale = range.scale();
      }
      // (dS is formed of P x 2^10)
      [[maybe_unused]] const float2 c2 = make_float2(ds_scale / kScaleP, ds_scale / kScaleP);
      for (int t = w.t0; t < w.t1; ++t, ++q) {
        const int st = q % kNS, pos0 = t * P;
        const float* info = reinterpret_cast<const float*>(smem + L::kOffInfo + st * 1024) + half * 64;
        // the warp's keys [key_a, key_a + 32) and rows, from position pos_a to
        // pos_b: none of their pairs is visible, or all are
        const int key_a = w.k0 + q4 * 32, pos_a = pos0 + ((half * 64) >> lg), pos_b = pos0 + ((half * 64 + 63) >> lg);
        const bool none = pos_b < key_a || (pos_a > key_a + 31 + p.window - 1 && key_a >= p.sinks);
        const bool all = pos_a >= key_a + 31 && pos_b <= key_a + p.window - 1;
        // ---- P^T
        if (!(ok = warp_wait(&bars->q_full[st], q / kNS) && warp_wait(&bars->s_full, q))) break;
        tc::fence_after_sync();
        uint32_t pf[64];
        const uint32_t s_tm = tb + kColST + half * 64;
        tc::tmem_ld32(s_tm, pf);
        tc::tmem_ld32(s_tm + 32, pf + 32);
        tc::tmem_wait_ld();
        uint32_t m[2] = {0xffffffffu, 0xffffffffu};  // visible rows
        if (!all) {
          // from the key's own row on, to the last whose window holds it
          const int64_t ca = (int64_t)(key - pos0) << lg;
          const int64_t cb = key < p.sinks ? kRows : ((int64_t)key + p.window - pos0) << lg;
          const int a = (int)max((int64_t)-1, min((int64_t)kRows, ca)) - half * 64;
          const int b = (int)max((int64_t)0, min((int64_t)kRows, cb)) - 1 - half * 64;
          m[0] = none ? 0u : bit_range(a, b);
          m[1] = none ? 0u : bit_range(a - 32, b - 32);
        }
        const float2 sc2 = make_float2(sc, sc);
        auto hand_over = [&](int c) {  // (the first part while the second is under way: its stores have ended by then)
          tc::tmem_wait_st();
          tc::fence_before_sync();
          warp_arrive(&bars->p_full[c], lane);
        };
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pw[16];
          if (none) {
#pragma unroll
            for (int j = 0; j < 32; ++j) pf[c * 32 + j] = 0u;
#pragma unroll
            for (int j = 0; j < 16; ++j) pw[j] = 0u;
          } else {
            auto scaled = [&](int j, float2* y) {  // logits of rows j .. j + 3 minus their log-sum-exps
              const float4 l4 = *reinterpret_cast<const float4*>(info + c * 32 + j);
              const uint32_t* v = pf + c * 32 + j;
              y[0] = __ffma2_rn(make_float2(__uint_as_float(v[0]), __uint_as_float(v[1])), sc2,
                                make_float2(l4.x, l4.y));
              y[1] = __ffma2_rn(make_float2(__uint_as_float(v[2]), __uint_as_float(v[3])), sc2,
                                make_float2(l4.z, l4.w));
            };
            float2 y[2], next[2];
            scaled(0, y);
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              uint32_t* v = pf + c * 32 + j;
              v[0] = __float_as_uint(ex2_placed(y[0].x));
              v[1] = __float_as_uint(ex2_placed(y[0].y));
              if (j + 4 < 32) scaled(j + 4, next);
              v[2] = __float_as_uint(ex2_placed(y[1].x));
              v[3] = __float_as_uint(ex2_placed(y[1].y));
              if (!all) {
#pragma unroll
                for (int u = 0; u < 4; ++u)
                  if (!(m[c] & (1u << (j + u)))) v[u] = 0u;
              }
              y[0] = next[0];
              y[1] = next[1];
              pw[j / 2] = pack2<T>(__uint_as_float(v[0]), __uint_as_float(v[1]));
              pw[j / 2 + 1] = pack2<T>(__uint_as_float(v[2]), __uint_as_float(v[3]));
              if (c == 1 && j == 8) hand_over(0);
            }
          }
          if (c == 1 && none) hand_over(0);
          tc::tmem_st16(s_tm + c * 16, pw);
          if (c == 1) hand_over(1);
        }
        // ---- dS^T
        if (!(ok = warp_wait(&bars->dp_full, q))) break;
        tc::fence_after_sync();
        const uint32_t d_tm = tb + kColDPT + half * 64;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t dv[32], dw[16];
          tc::tmem_ld32(d_tm + c * 32, dv);
          tc::tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 d4 = *reinterpret_cast<const float4*>(info + 128 + c * 32 + j);
            const int e = c * 32 + j;
            auto less_d = [&](int x, float2 nd) {
              const float2 dp = make_float2(__uint_as_float(dv[x]), __uint_as_float(dv[x + 1]));
              return kScaled<T> ? __ffma2_rn(dp, c2, nd) : __fadd2_rn(dp, nd);
            };
            const float2 a = __fmul2_rn(make_float2(__uint_as_float(pf[e]), __uint_as_float(pf[e + 1])),
                                        less_d(j, make_float2(d4.x, d4.y)));
            const float2 b = __fmul2_rn(make_float2(__uint_as_float(pf[e + 2]), __uint_as_float(pf[e + 3])),
                                        less_d(j + 2, make_float2(d4.z, d4.w)));
            dw[j >> 1] = pack2<T>(a.x, a.y);
            dw[(j >> 1) + 1] = pack2<T>(b.x, b.y);
          }
          tc::tmem_st16(d_tm + c * 16, dw);
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        warp_arrive(&bars->ds_full, lane);
        warp_arrive(&bars->q_empty[st], lane);
      }
      if (!ok) break;
      // ---- dk, dv: each half of the workers takes half of the columns
      const bool any = w.t1 > w.t0;
      if (any) {
        if (!(ok = warp_wait(&bars->acc_full, items))) break;
        tc::fence_after_sync();
        ++items;
      }
      const float ksc = rsqrtf((float)D) / ds_scale, vsc = kScaled<T> ? 1.f / kScaleP : 1.f;
      const bool live = key < w.n;
      // each half of the workers takes half of the columns
#pragma unroll 1
      for (int o = 0; o < 2; ++o) {
        const View& out = o ? p.dv : p.dk;
        T* dst = static_cast<T*>(const_cast<void*>(out.data)) + (int64_t)w.b * out.sb +
                 (int64_t)min(key, p.S - 1) * out.ss + (int64_t)w.g * out.sh;
        // [b, g][slot][dk, dv][128][D] fp32
        const int64_t slot = (int64_t)(w.b * p.Hkv + w.g) * (p.n_chunks + 1) + w.slot;
        float* part = p.part + ((slot * 2 + o) * kRows + k) * D;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          const int col = (half * (D / 64) + c) * 32;
          uint32_t v[32];
          if (any) {
            tc::tmem_ld32(tb + (o ? kColDV : kColDK) + col, v);
            tc::tmem_wait_ld();
          }
          if (!any || !live) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = 0u;
          }
          if (w.slot >= 0) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4*>(part + col + e) = make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]);
          } else if (key < p.S) {
            store_row32(dst + col, v, o ? vsc : ksc, p.wide);
          }
        }
      }
      if (any) {
        tc::fence_before_sync();
        warp_arrive(&bars->acc_empty, lane);
      }
    }
    if (!ok) raise_status(p.status, kTimeout, 343);
  }

  tc::fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// dk, dv of the first 128 keys: the band's partial and the chunks', in order.
template <typename T, int D>
__global__ void __launch_bounds__(256) window_bwd_join_kernel(const WindowParams p) {
  const int bg = blockIdx.x, b = bg / p.Hkv, g = bg % p.Hkv;
  const int i = (blockIdx.y * 256 + threadIdx.x) * 4;  // element of [dk, dv][128][D]
  const int key = i / D % kRows, c = i % D;
  const float* src = p.part + (int64_t)bg * (p.n_chunks + 1) * 2 * kRows * D + i;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  float ds_scale = 1.f;
  if constexpr (kScaled<T>) {
    Range range;
    range.ask(p, b, g, threadIdx.x & 31);
    ds_scale = range.scale();
  }
  if (key >= p.S) return;
  for (int x = 0; x <= p.n_chunks; ++x) {
    const float4 v = *reinterpret_cast<const float4*>(src + (int64_t)x * 2 * kRows * D);
    s.x += v.x;
    s.y += v.y;
    s.z += v.z;
    s.w += v.w;
  }
  const bool is_v = i >= kRows * D;
  const View& out = is_v ? p.dv : p.dk;
  const float f = is_v ? (kScaled<T> ? 1.f / kScaleP : 1.f) : rsqrtf((float)D) / ds_scale;
  T* dst = static_cast<T*>(const_cast<void*>(out.data)) + (int64_t)b * out.sb + (int64_t)key * out.ss +
           (int64_t)g * out.sh + c;
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<T>(s.x * f, s.y * f), pack2<T>(s.z * f, s.w * f));
}

// A launch that may start before the kernel in front of it ends; it waits for
// that kernel's results itself (griddepcontrol.wait).
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kern)(Params...), dim3 grid, int threads, int smem, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <typename T, int D>
cudaError_t run(const WindowParams& p, cudaStream_t stream) {
  const int P = kRows / p.G;
  const int64_t row_items = (int64_t)p.n_tiles * p.Hkv * p.B;
  const int64_t key_items = ((int64_t)(p.S + kRows - 1) / kRows + p.n_chunks) * p.Hkv * p.B;
  if (std::max(row_items, key_items) > 0x7fffffff - 4096) return cudaErrorInvalidValue;
  cudaError_t e;
  CUtensorMap mq, mdo, mo, mr, mk, mv;
  if (!window_map(&mq, p.q, p.dtype, p.B, p.S, p.H, D, p.G, P) ||
      !window_map(&mdo, p.dout, p.dtype, p.B, p.S, p.H, D, p.G, P) ||
      !window_map(&mo, p.out, p.dtype, p.B, p.S, p.H, D, p.G, P) ||
      !window_map(&mr, p.rest.data ? p.rest : p.out, p.dtype, p.B, p.S, p.H, D, p.G, P) ||
      !window_map(&mk, p.k, p.dtype, p.B, p.S, p.Hkv, D, 1, kRows) ||
      !window_map(&mv, p.v, p.dtype, p.B, p.S, p.Hkv, D, 1, kRows))
    return cudaErrorInvalidValue;
  {
    using L = RowLayout<D>;
    auto kern = p.window + p.sinks <= kFewKeys ? window_bwd_row_tc_kernel<T, D, true>
                                               : window_bwd_row_tc_kernel<T, D, false>;
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc)) != cudaSuccess)
      return e;
    const dim3 grid((unsigned)std::min<int64_t>(row_items, p.num_sms));
    if constexpr (kScaled<T>) {
      window_bwd_range_kernel<T, D><<<dim3(p.n_range, p.Hkv, p.B), kRangeThreads, 0, stream>>>(p);
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
      e = launch_early(kern, grid, kThreads, L::kAlloc, stream, mq, mdo, mo, mr, mk, mv, p);
    } else {
      kern<<<grid, kThreads, L::kAlloc, stream>>>(mq, mdo, mo, mr, mk, mv, p);
      e = cudaGetLastError();
    }
    if (e != cudaSuccess) return e;
  }
  {
    using L = KeyLayout<D>;
    auto kern = window_bwd_key_tc_kernel<T, D>;
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc)) != cudaSuccess)
      return e;
    const dim3 grid((unsigned)std::min<int64_t>(key_items, p.num_sms));
    const int per_head = (p.S + kRows - 1) / kRows + p.n_chunks;
    e = launch_early(kern, grid, kThreads, L::kAlloc, stream, mq, mdo, mk, mv, p, per_head);
    if (e != cudaSuccess) return e;
  }
  if (p.n_chunks > 0)
    e = launch_early(window_bwd_join_kernel<T, D>, dim3(p.B * p.Hkv, 2 * kRows * D / 1024), 256, 0, stream, p);
  return e;
}

}  // namespace

cudaError_t launch_window_bwd_tc(const WindowParams& p, cudaStream_t stream) {
  if (p.D == 128) return p.dtype == 1 ? run<__half, 128>(p, stream) : run<__nv_bfloat16, 128>(p, stream);
  return p.dtype == 1 ? run<__half, 64>(p, stream) : run<__nv_bfloat16, 64>(p, stream);
}

}  // namespace dash
