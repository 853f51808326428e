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
// everything else is fp32.  Every wait is bounded; on expiry the status word
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

// ------------------------------------------------------------------ rows: dq, D
//
// A CTA (one per SM) walks 128-row tiles; per tile the keys its rows see come
// in steps of 64 (sink steps before the band, then the band).
//   S = Q K^T, dP = dout V^T   A = Q, dout from TMEM; two buffers
//   dS over S in 16 bits;  dQ += dS K  (A from TMEM, K MN-major)
// Warps 0-3 take the even steps, 4-7 the odd ones: while one group forms dS,
// the tensor core works for the other.  The next tile's Q, dout and out come
// by TMA during this one, and are moved to TMEM (with D) before this tile's dq
// is written, so its first products overlap that.  Warp 8 is the TMA
// producer, which also clears K rows behind a sequence's end; warp 9 issues
// the MMAs.  TMEM: Q at 0, dout at D / 2, buffers at 128 + 128 b (S, dP), dQ
// at 384.
constexpr int kStepR = 64;
constexpr uint32_t kColBuf = 128, kColDQ = 384;

template <int D>
struct RowLayout {
  static constexpr int KC = D / 64;
  static constexpr int kRowChunk = kRows * 128, kRowTile = KC * kRowChunk;
  static constexpr int kKeyChunk = kStepR * 128, kKeyTile = KC * kKeyChunk;
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr int kOffQ = 0, kOffDo = kRowTile, kOffO = 2 * kRowTile;
  static constexpr int kOffKV = 3 * kRowTile;  // [kStages] K, V
  static constexpr int kOffBar = kOffKV + kStages * 2 * kKeyTile;
  static constexpr int kAlloc = kOffBar + 512 + 1024;
};

struct RowBars {
  uint64_t rows_full, rows_empty;  // Q, dout, out in shared memory
  uint64_t ready;                  // Q and dout in TMEM
  uint64_t kv_full[8], kv_empty[8];
  uint64_t tail;
  uint64_t s_full[2], ds_full[2];
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
        kt(pos0, min(pos0 + P, n), p.window, p.sinks, kStepR) {
    steps = pos0 < n ? kt.n : 0;
  }
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    window_bwd_row_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                             const __grid_constant__ CUtensorMap tm_o, const __grid_constant__ CUtensorMap tm_k,
                             const __grid_constant__ CUtensorMap tm_v, const WindowParams p) {
  using L = RowLayout<D>;
  constexpr int kStages = L::kStages;
  constexpr bool kBF16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr uint32_t kIdescS = tc::idesc_f16(kRows, kStepR, kBF16, false, false);
  constexpr uint32_t kIdescQ = tc::idesc_f16(kRows, D, kBF16, false, true);

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  RowBars* bars = reinterpret_cast<RowBars*>(smem + L::kOffBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lg = __ffs(p.G) - 1, P = kRows >> lg;

  if (threadIdx.x == 0) {
    tc::mbar_init(&bars->rows_full, 1);
    tc::mbar_init(&bars->rows_empty, kWorkers);
    tc::mbar_init(&bars->ready, kWorkers);
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(&bars->kv_full[s], 1);
      tc::mbar_init(&bars->kv_empty[s], 1);
    }
    tc::mbar_init(&bars->tail, 1);
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(&bars->s_full[s], 1);
      tc::mbar_init(&bars->ds_full[s], kRows);
    }
    tc::mbar_init(&bars->dq_full, 1);
    tc::mbar_init(&bars->dq_empty, kWorkers);
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

  if (warp == kProducerWarp) {
    // ------------------------------------------------------------ producer
    if (blockIdx.x == 0) begin_status(p, lane);
    int kv = 0, items = 0, tails = 0;
    for (ItemWalk it(p.n_tiles, p.Hkv, p.B); ok && it.any(); it.next()) {
      const RowItem w(p, P, it);
      if (w.steps == 0) continue;
      if (items > 0) ok = warp_wait(&bars->rows_empty, items - 1);
      if (!ok) break;
      if (lane == 0) {
        tc::mbar_arrive_expect_tx(&bars->rows_full, 3 * L::kRowTile);
        for (int kc = 0; kc < L::KC; ++kc) {
          uint8_t* dst = smem + kc * L::kRowChunk;
          tc::tma_load_4d(dst + L::kOffQ, &tm_q, &bars->rows_full, kc * 64, w.g * p.G, w.pos0, w.b);
          tc::tma_load_4d(dst + L::kOffDo, &tm_do, &bars->rows_full, kc * 64, w.g * p.G, w.pos0, w.b);
          tc::tma_load_4d(dst + L::kOffO, &tm_o, &bars->rows_full, kc * 64, w.g * p.G, w.pos0, w.b);
        }
      }
      ++items;
      for (int i = 0; ok && i < w.steps; ++i, ++kv) {
        const int st = kv % kStages, tok0 = w.kt.tile(i) * kStepR;
        if (kv >= kStages) ok = warp_wait(&bars->kv_empty[st], (kv / kStages) - 1);
        if (!ok) break;
        uint8_t* dst = smem + L::kOffKV + st * 2 * L::kKeyTile;
        const bool clear = tok0 + kStepR > w.n && w.n < p.S;
        uint64_t* bar = clear ? &bars->tail : &bars->kv_full[st];
        if (lane == 0) {
          tc::mbar_arrive_expect_tx(bar, 2 * L::kKeyTile);
          for (int kc = 0; kc < L::KC; ++kc) {
            tc::tma_load_4d(dst + kc * L::kKeyChunk, &tm_k, bar, kc * 64, w.g, tok0, w.b);
            tc::tma_load_4d(dst + L::kKeyTile + kc * L::kKeyChunk, &tm_v, bar, kc * 64, w.g, tok0, w.b);
          }
        }
        if (clear) {
          // dS is 0 there, but 0 x NaN is not
          ok = warp_wait(&bars->tail, tails++);
          zero_tile_rows(dst, L::KC, kStepR, w.n - tok0, lane);
          if (lane == 0) tc::mbar_arrive(&bars->kv_full[st]);
        }
      }
    }
    // every copy lands before the CTA retires
    if (items > 0) tc::mbar_wait(&bars->rows_full, (items - 1) & 1);
    for (int j = max(0, kv - kStages); j < kv; ++j) tc::mbar_wait(&bars->kv_full[j % kStages], (j / kStages) & 1);
    if (!ok) raise_status(p.status, kTimeout, 331);
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    auto wait = [&](uint64_t* bar, int phase) {
      ok = ok && warp_wait(bar, phase);
      tc::fence_after_sync();
      return ok;
    };
    const uint64_t k0 = tc::smem_desc_sw128(smem + L::kOffKV, 16, 1024);
    const uint64_t v0 = tc::smem_desc_sw128(smem + L::kOffKV + L::kKeyTile, 16, 1024);
    const uint64_t kmn0 = tc::smem_desc_sw128(smem + L::kOffKV, L::kKeyChunk, 1024);
    int kv = 0, items = 0;
    for (ItemWalk it(p.n_tiles, p.Hkv, p.B); ok && it.any(); it.next()) {
      const RowItem w(p, P, it);
      if (w.steps == 0) continue;
      if (!wait(&bars->ready, items)) break;
      // dQ += dS K of the item's step j (step x of the CTA)
      auto issue_dq = [&](int j) {
        const int x = kv + j;
        if (j == 0 && items > 0 && !wait(&bars->dq_empty, items - 1)) return;
        if (!wait(&bars->ds_full[x & 1], x >> 1)) return;
        const uint64_t kd = kmn0 + (uint64_t)(((x % kStages) * 2 * L::kKeyTile) >> 4);
#pragma unroll
        for (int k = 0; k < kStepR / 16; ++k)
          tc::mma_f16_ts_w(tmem + kColDQ, tmem + kColBuf + (x & 1) * 128 + k * 8, kd + (uint64_t)((k * 2048) >> 4),
                           kIdescQ, (j > 0 || k > 0) ? 1u : 0u);
        tc::mma_commit_w(&bars->kv_empty[x % kStages]);
      };
      for (int i = 0; ok && i < w.steps; ++i) {
        const int x = kv + i;
        if (!wait(&bars->kv_full[x % kStages], x / kStages)) break;
        const uint64_t off = (uint64_t)(((x % kStages) * 2 * L::kKeyTile) >> 4);
        const uint32_t s_tm = tmem + kColBuf + (x & 1) * 128;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t o = off + (uint64_t)((((k >> 2) * L::kKeyChunk) + (k & 3) * 32) >> 4);
          tc::mma_f16_ts_w(s_tm, tmem + k * 8, k0 + o, kIdescS, k > 0 ? 1u : 0u);
        }
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t o = off + (uint64_t)((((k >> 2) * L::kKeyChunk) + (k & 3) * 32) >> 4);
          tc::mma_f16_ts_w(s_tm + 64, tmem + D / 2 + k * 8, v0 + o, kIdescS, k > 0 ? 1u : 0u);
        }
        tc::mma_commit_w(&bars->s_full[x & 1]);
        if (i > 0) issue_dq(i - 1);
      }
      if (ok) issue_dq(w.steps - 1);
      if (!ok) break;
      tc::mma_commit_w(&bars->dq_full);
      kv += w.steps;
      ++items;
    }
    if (!ok) raise_status(p.status, kTimeout, 332);
    tc::mma_commit_w(&bars->drained);
    tc::mbar_wait(&bars->drained, 0);
  } else {
    // ------------------------------------------------------------ rows
    const int wg = warp >> 2, q4 = warp & 3, r = q4 * 32 + lane;
    const uint32_t tb = tmem + ((uint32_t)(q4 * 32) << 16);
    const float sc = rsqrtf((float)D) * kLog2e;
    float lse2 = 0.f, dd = 0.f;  // of the current item's row
    int items = 0, step = 0;

    // the first item with steps from `it` on; tiles behind the sequence's end
    // get dq = 0 and lse2 = inf (p = 0) on the way
    auto seek = [&](ItemWalk& it) {
      for (; it.any(); it.next()) {
        const RowItem w(p, P, it);
        if (w.steps > 0) break;
        const int pos = w.pos0 + (r >> lg), head = w.g * p.G + (r & (p.G - 1));
        if (wg == 0) {
          const int64_t at = ((int64_t)(w.b * p.Hkv + w.g) * p.n_tiles + w.tile) * kRows + r;
          p.lse2[at] = -kNegInf;
          p.dd[at] = 0.f;
        } else if (pos < p.S) {
          T* dst = static_cast<T*>(const_cast<void*>(p.dq.data)) + (int64_t)w.b * p.dq.sb + (int64_t)pos * p.dq.ss +
                   (int64_t)head * p.dq.sh;
#pragma unroll
          for (int x = 0; x < D / 8; ++x) *reinterpret_cast<uint4*>(dst + x * 8) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
    };
    // Q (warps 0-3) and dout (4-7) into TMEM, D = dout . out and lse2
    auto load_rows = [&](const ItemWalk& it) {
      const RowItem w(p, P, it);
      const int pos = w.pos0 + (r >> lg), head = w.g * p.G + (r & (p.G - 1));
      const bool live = pos < w.n;
      lse2 = live ? p.lse[((int64_t)w.b * p.H + head) * p.S + pos] * kLog2e : -kNegInf;
      if (!warp_wait(&bars->rows_full, items)) return false;
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int cc = 0; cc < L::KC; ++cc) {
        const uint8_t* base = smem + cc * L::kRowChunk + r * 128;
        uint32_t w32[32];
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          const int at = (v ^ (r & 7)) * 16;
          const uint4 xd = *reinterpret_cast<const uint4*>(base + L::kOffDo + at);
          const uint4 xo = *reinterpret_cast<const uint4*>(base + L::kOffO + at);
          const uint4 xt = wg == 0 ? *reinterpret_cast<const uint4*>(base + L::kOffQ + at) : xd;
          w32[4 * v] = xt.x, w32[4 * v + 1] = xt.y, w32[4 * v + 2] = xt.z, w32[4 * v + 3] = xt.w;
          float fd[8], fo[8];
          Elt<T>::to_float(xd, fd);
          Elt<T>::to_float(xo, fo);
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e & 3] = fmaf(fd[e], fo[e], acc[e & 3]);
        }
        tc::tmem_st32(tb + (wg == 0 ? 0 : D / 2) + cc * 32, w32);
      }
      dd = live ? (acc[0] + acc[1]) + (acc[2] + acc[3]) : 0.f;
      if (wg == 0) {
        const int64_t at = ((int64_t)(w.b * p.Hkv + w.g) * p.n_tiles + w.tile) * kRows + r;
        p.lse2[at] = lse2;
        p.dd[at] = dd;
      }
      tc::tmem_wait_st();
      tc::fence_before_sync();
      tc::mbar_arrive(&bars->rows_empty);
      tc::mbar_arrive(&bars->ready);
      return true;
    };

    ItemWalk it(p.n_tiles, p.Hkv, p.B);
    seek(it);
    if (it.any()) ok = load_rows(it);
    while (ok && it.any()) {
      const RowItem w(p, P, it);
      const int pos = w.pos0 + (r >> lg), head = w.g * p.G + (r & (p.G - 1));
      const int lo = pos - p.window + 1;
      const int lo_b = w.pos0 + P - p.window;  // the last row's lo
      for (int i = (step & 1) == wg ? 0 : 1; i < w.steps; i += 2) {
        const int x = step + i, tok0 = w.kt.tile(i) * kStepR;
        const uint32_t s_tm = tb + kColBuf + (x & 1) * 128;
        if (!(ok = warp_wait(&bars->s_full[x & 1], x >> 1))) break;
        tc::fence_after_sync();
        const bool edge = tok0 + kStepR - 1 > w.pos0 || tok0 < lo_b;
        const float2 sc2 = make_float2(sc, sc), off2 = make_float2(-lse2, -lse2), nd2 = make_float2(-dd, -dd);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t sv[32], pv[32], dw[16];
          tc::tmem_ld32(s_tm + c * 32, sv);
          tc::tmem_ld32(s_tm + 64 + c * 32, pv);
          tc::tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float2 y = __ffma2_rn(make_float2(__uint_as_float(sv[j]), __uint_as_float(sv[j + 1])), sc2, off2);
            const float2 e = make_float2(tc::ex2(y.x), tc::ex2(y.y));
            const float2 d =
                __fadd2_rn(make_float2(__uint_as_float(pv[j]), __uint_as_float(pv[j + 1])), nd2);
            const float2 ds = __fmul2_rn(e, d);
            sv[j] = __float_as_uint(ds.x);
            sv[j + 1] = __float_as_uint(ds.y);
          }
          if (edge) {
            const int t0 = tok0 + c * 32;
            const uint32_t seen = bit_range(lo - t0, pos - t0) | bit_range(0, min(pos, p.sinks - 1) - t0);
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!(seen & (1u << j))) sv[j] = 0u;
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) dw[j] = pack2<T>(__uint_as_float(sv[2 * j]), __uint_as_float(sv[2 * j + 1]));
          tc::tmem_st16(s_tm + c * 16, dw);
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        tc::mbar_arrive(&bars->ds_full[x & 1]);
      }
      step += w.steps;
      if (!ok || !(ok = warp_wait(&bars->dq_full, items))) break;
      tc::fence_after_sync();
      ++items;
      it.next();
      seek(it);
      if (it.any() && !(ok = load_rows(it))) break;
      // ---- dq of this item, each group half of the columns
      T* dst = static_cast<T*>(const_cast<void*>(p.dq.data)) + (int64_t)w.b * p.dq.sb +
               (int64_t)min(pos, p.S - 1) * p.dq.ss + (int64_t)head * p.dq.sh;
      const bool live = pos < w.n;
#pragma unroll
      for (int cc = wg * (D / 64); cc < (wg + 1) * (D / 64); ++cc) {
        uint32_t v[32];
        tc::tmem_ld32(tb + kColDQ + cc * 32, v);
        tc::tmem_wait_ld();
        if (!live) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = 0u;
        }
        if (pos < p.S) {
#pragma unroll
          for (int x = 0; x < 4; ++x)
            *reinterpret_cast<uint4*>(dst + cc * 32 + x * 8) = pack8<T>(v + x * 8, rsqrtf((float)D));
        }
      }
      tc::fence_before_sync();
      tc::mbar_arrive(&bars->dq_empty);
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
  static constexpr int kOffInfo = kOffQ + kNS * 2 * kTile;  // [kNS] lse2[128], D[128]
  static constexpr int kOffBar = kOffInfo + kNS * 1024;
  static constexpr int kAlloc = kOffBar + 256 + 1024;
};

struct KeyBars {
  uint64_t kv_full, kv_empty;
  uint64_t q_full[kNS], q_empty[kNS];
  uint64_t tail;
  uint64_t s_full, dp_full, p_full, ds_full;
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
  const int lgp = 8 - __ffs(p.G), P = 1 << lgp;  // positions of a row tile

  if (threadIdx.x == 0) {
    tc::mbar_init(&bars->kv_full, 1);
    tc::mbar_init(&bars->kv_empty, 1);
    for (int s = 0; s < kNS; ++s) {
      tc::mbar_init(&bars->q_full[s], 1);
      tc::mbar_init(&bars->q_empty[s], 1 + kWorkers);
    }
    tc::mbar_init(&bars->tail, 1);
    tc::mbar_init(&bars->s_full, 1);
    tc::mbar_init(&bars->dp_full, 1);
    tc::mbar_init(&bars->p_full, kWorkers);
    tc::mbar_init(&bars->ds_full, kWorkers);
    tc::mbar_init(&bars->acc_full, 1);
    tc::mbar_init(&bars->acc_empty, kWorkers);
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
          tc::bulk_load(smem + L::kOffInfo + st * 1024, p.lse2 + at, 512, bar);
          tc::bulk_load(smem + L::kOffInfo + st * 1024 + 512, p.dd + at, 512, bar);
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
    // dV or dK: contraction over the tile's rows; rows 0-63 of the operand are
    // packed at col, rows 64-127 at col + 64 (each worker half's own columns)
    auto issue_ts = [&](uint32_t dst, uint32_t col, uint64_t b, bool first) {
#pragma unroll
      for (int k = 0; k < kRows / 16; ++k)
        tc::mma_f16_ts_w(tmem + dst, tmem + col + (k >> 2) * 64 + (k & 3) * 8, b + (uint64_t)((k * 2048) >> 4),
                         kIdescKV, (!first || k > 0) ? 1u : 0u);
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
        if (!wait(&bars->p_full, x)) break;
        issue_ts(kColDV, kColST, qmn0 + tile16 + stage(x), i == 0);
        if (i + 1 < n) {
          if (!wait(&bars->q_full[(x + 1) % kNS], (x + 1) / kNS)) break;
          issue_ss(kColST, kd, q0 + stage(x + 1), &bars->s_full);
        }
        if (!wait(&bars->ds_full, x)) break;
        issue_ts(kColDK, kColDPT, qmn0 + stage(x), i == 0);
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
      for (int t = w.t0; t < w.t1; ++t, ++q) {
        const int st = q % kNS, pos0 = t * P;
        const float* info = reinterpret_cast<const float*>(smem + L::kOffInfo + st * 1024) + half * 64;
        const bool edge = pos0 < w.k0 + kRows - 1 || pos0 + P - 1 > w.k0 + p.window - 1;
        // ---- P^T
        if (!(ok = warp_wait(&bars->q_full[st], q / kNS) && warp_wait(&bars->s_full, q))) break;
        tc::fence_after_sync();
        uint32_t pf[64];
        const uint32_t s_tm = tb + kColST + half * 64;
        tc::tmem_ld32(s_tm, pf);
        tc::tmem_ld32(s_tm + 32, pf + 32);
        tc::tmem_wait_ld();
        const float2 sc2 = make_float2(sc, sc);
#pragma unroll
        for (int j = 0; j < 64; j += 4) {
          const float4 l4 = *reinterpret_cast<const float4*>(info + j);
          const float2 a = __ffma2_rn(make_float2(__uint_as_float(pf[j]), __uint_as_float(pf[j + 1])), sc2,
                                      make_float2(-l4.x, -l4.y));
          const float2 b = __ffma2_rn(make_float2(__uint_as_float(pf[j + 2]), __uint_as_float(pf[j + 3])), sc2,
                                      make_float2(-l4.z, -l4.w));
          pf[j] = __float_as_uint(tc::ex2(a.x));
          pf[j + 1] = __float_as_uint(tc::ex2(a.y));
          pf[j + 2] = __float_as_uint(tc::ex2(b.x));
          pf[j + 3] = __float_as_uint(tc::ex2(b.y));
        }
        if (edge) {
          // rows from the key's own on, to the last whose window holds it
          const int64_t ca = (int64_t)(key - pos0) * p.G;
          const int64_t cb = key < p.sinks ? kRows : ((int64_t)key + p.window - pos0) * p.G;
          const int a = (int)max((int64_t)-1, min((int64_t)kRows, ca)) - half * 64;
          const int b = (int)max((int64_t)0, min((int64_t)kRows, cb)) - 1 - half * 64;
          const uint32_t m0 = bit_range(a, b), m1 = bit_range(a - 32, b - 32);
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            if (!(m0 & (1u << j))) pf[j] = 0u;
            if (!(m1 & (1u << j))) pf[32 + j] = 0u;
          }
        }
        {
          uint32_t pw[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) pw[j] = pack2<T>(__uint_as_float(pf[2 * j]), __uint_as_float(pf[2 * j + 1]));
          tc::tmem_st32(s_tm, pw);
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        tc::mbar_arrive(&bars->p_full);
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
            const float2 a = __fmul2_rn(make_float2(__uint_as_float(pf[e]), __uint_as_float(pf[e + 1])),
                                        __fadd2_rn(make_float2(__uint_as_float(dv[j]), __uint_as_float(dv[j + 1])),
                                                   make_float2(-d4.x, -d4.y)));
            const float2 b = __fmul2_rn(make_float2(__uint_as_float(pf[e + 2]), __uint_as_float(pf[e + 3])),
                                        __fadd2_rn(make_float2(__uint_as_float(dv[j + 2]), __uint_as_float(dv[j + 3])),
                                                   make_float2(-d4.z, -d4.w)));
            dw[j >> 1] = pack2<T>(a.x, a.y);
            dw[(j >> 1) + 1] = pack2<T>(b.x, b.y);
          }
          tc::tmem_st16(d_tm + c * 16, dw);
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        tc::mbar_arrive(&bars->ds_full);
        tc::mbar_arrive(&bars->q_empty[st]);
      }
      if (!ok) break;
      // ---- dk, dv: each half of the workers takes half of the columns
      const bool any = w.t1 > w.t0;
      if (any) {
        if (!(ok = warp_wait(&bars->acc_full, items))) break;
        tc::fence_after_sync();
        ++items;
      }
      const float ksc = rsqrtf((float)D);
      const bool live = key < w.n;
#pragma unroll 1
      for (int cc = half * (D / 64); cc < (half + 1) * (D / 64); ++cc) {
        uint32_t v[32], d[32];
        if (any) {
          tc::tmem_ld32(tb + kColDV + cc * 32, v);
          tc::tmem_ld32(tb + kColDK + cc * 32, d);
          tc::tmem_wait_ld();
        }
        if (!any || !live) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = d[j] = 0u;
        }
        if (w.slot >= 0) {
          // [b, g][slot][dk, dv][128][D] fp32
          float* dst = p.part + ((((int64_t)(w.b * p.Hkv + w.g) * (p.n_chunks + 1) + w.slot) * 2) * kRows + k) * D +
                       cc * 32;
#pragma unroll
          for (int x = 0; x < 32; x += 4) {
            *reinterpret_cast<uint4*>(dst + x) = make_uint4(d[x], d[x + 1], d[x + 2], d[x + 3]);
            *reinterpret_cast<uint4*>(dst + kRows * D + x) = make_uint4(v[x], v[x + 1], v[x + 2], v[x + 3]);
          }
        } else if (key < p.S) {
          T* dk = static_cast<T*>(const_cast<void*>(p.dk.data)) + (int64_t)w.b * p.dk.sb + (int64_t)key * p.dk.ss +
                  (int64_t)w.g * p.dk.sh + cc * 32;
          T* dv = static_cast<T*>(const_cast<void*>(p.dv.data)) + (int64_t)w.b * p.dv.sb + (int64_t)key * p.dv.ss +
                  (int64_t)w.g * p.dv.sh + cc * 32;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            *reinterpret_cast<uint4*>(dk + x * 8) = pack8<T>(d + x * 8, ksc);
            *reinterpret_cast<uint4*>(dv + x * 8) = pack8<T>(v + x * 8, 1.f);
          }
        }
      }
      if (any) {
        tc::fence_before_sync();
        tc::mbar_arrive(&bars->acc_empty);
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
  if (key >= p.S) return;
  const float* src = p.part + (int64_t)bg * (p.n_chunks + 1) * 2 * kRows * D + i;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  for (int x = 0; x <= p.n_chunks; ++x) {
    const float4 v = *reinterpret_cast<const float4*>(src + (int64_t)x * 2 * kRows * D);
    s.x += v.x;
    s.y += v.y;
    s.z += v.z;
    s.w += v.w;
  }
  const bool is_v = i >= kRows * D;
  const View& out = is_v ? p.dv : p.dk;
  const float f = is_v ? 1.f : rsqrtf((float)D);
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
  CUtensorMap mq, mdo, mo, mk, mv;
  if (!make_map(&mq, p.q, p.dtype, p.B, p.S, p.H, D, p.G, P) ||
      !make_map(&mdo, p.dout, p.dtype, p.B, p.S, p.H, D, p.G, P) ||
      !make_map(&mo, p.out, p.dtype, p.B, p.S, p.H, D, p.G, P))
    return cudaErrorInvalidValue;
  {
    using L = RowLayout<D>;
    if (!make_map(&mk, p.k, p.dtype, p.B, p.S, p.Hkv, D, 1, kStepR) ||
        !make_map(&mv, p.v, p.dtype, p.B, p.S, p.Hkv, D, 1, kStepR))
      return cudaErrorInvalidValue;
    auto kern = window_bwd_row_tc_kernel<T, D>;
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc)) != cudaSuccess)
      return e;
    kern<<<(unsigned)std::min<int64_t>(row_items, p.num_sms), kThreads, L::kAlloc, stream>>>(mq, mdo, mo, mk, mv, p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  {
    using L = KeyLayout<D>;
    if (!make_map(&mk, p.k, p.dtype, p.B, p.S, p.Hkv, D, 1, kRows) ||
        !make_map(&mv, p.v, p.dtype, p.B, p.S, p.Hkv, D, 1, kRows))
      return cudaErrorInvalidValue;
    auto kern = window_bwd_key_tc_kernel<T, D>;
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc)) != cudaSuccess)
      return e;
    if ((e = launch_early(kern, dim3((unsigned)std::min<int64_t>(key_items, p.num_sms)), kThreads, L::kAlloc, stream, mq,
                          mdo, mk, mv, p, (p.S + kRows - 1) / kRows + p.n_chunks)) != cudaSuccess)
      return e;
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
