// Sliding-window (and dense causal) attention forward on the 5th-generation
// tensor cores, f16 / bf16.
//
// Row i of head h sees key j when j <= i and (j > i - window or j < sinks):
//   s_ij = q_i . k_j / sqrt(D);  o_i = sum_j 2^(s_ij log2e - m) v_j / l
//
// A tile is 128 rows = (128 / G positions) x (G heads of one KV group), so
// each K/V tile serves the group's heads and a tile's band is narrow: its keys
// are the window plus 128 / G.  A work item is two adjacent tiles of one KV
// head; each CTA (one per SM) walks items.  Per item the keys come in steps of
// 128: at most one step of sink tokens before the band, then the band; only
// steps that hold a visible pair are walked, and only steps at an edge of the
// band are masked (bit masks per row).
//
// Tensor memory: S of tile t at 128 t (P written back over it in 16 bits), O
// of tile t at 256 + 128 t.  Shared memory: the Q tiles and a ring of K / V
// tiles.  The tensor core runs, per tile, O += P V of the step before, then
// S = Q K^T of this step, while the other tile's softmax runs.  The stream of
// steps does not stop at the end of an item: the next item's first products
// run during this one's epilogue.
//   warps 0-3, 4-7  softmax of tile 0 / 1: a thread owns a row (TMEM lane)
//   warp 8          TMA producer; also clears V rows behind a sequence's end
//                   (they may hold anything; P is 0 there, but 0 x NaN is not)
//   warp 9          MMA issuer and TMEM owner
// Measured slower than this (1.09 ms for a 32K prompt with window 2048 before
// the stream ran on over items): steps of 64 keys with two S buffers per tile,
// so that the softmax never waits for S (1.16 ms: the tensor core takes about
// 56 clocks for a 128 x 64 product with both operands in shared memory, almost
// those of 128 x 128); P handed over in two halves (1.22 ms); two threads per
// row, 16 softmax warps (1.54 ms); an MMA issuer per tile (1.29 ms: the tiles
// fall into step, and the softmax of both then waits for the products of both).
//
// The softmax keeps a reference m per row; while a step's sum shows no p
// above 2^12 the row maximum is not needed.  A larger one makes the row take
// its maximum, and O is rescaled when that moved by more than 2^8 (rare after
// the first step).  The warp goes that way together, but only the rows whose
// own sum asked for it move their reference: a row's bits do not depend on
// the others of its warp, and rows behind a sequence's end, whose logits may
// be anything, ask for nothing.  P is rounded to the input type for the second
// product (the tensor core's operand type); sums, m, l and O are fp32.
//
// Bound by the chain softmax -> P V -> S of a tile, of which two are in flight
// (tensor memory has room for two): about 1600 + 1250 clocks per 128 keys,
// where the tensor cores and the special-function units need 2048 each for the
// two tiles at D = 128.  A share of the exponentials by a polynomial on the FMA
// pipe was slower at every share tried: its 14 instructions per pair lengthen
// the chain more than the unit's time shortens.
// Every wait is bounded; on expiry the status word reads
// DASH_ERR_DEVICE_TIMEOUT and the roles wind down.
#include <cuda.h>

#include <algorithm>
#include <type_traits>

#include "window_tc.cuh"

namespace dash {
namespace {

constexpr int kRows = 128;
constexpr int kTiles = 2;
constexpr int kStep = 128;
constexpr int kProducerWarp = 8, kMmaWarp = 9;
// 12 warps (10 and 11 only give registers away): 168 registers a thread at
// launch, 504 = 3 x 168 per lane of the three warpgroups, split as 2 x 216 + 72
constexpr int kThreads = 384;
constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;
constexpr uint32_t kColS = 0, kColO = 256;
constexpr float kRescaleLog2 = 8.f;
constexpr float kMaxSum = 4096.f;

template <int D>
struct Layout {
  static constexpr int KC = D / 64;
  static constexpr int kChunk = 128 * 128, kTile = KC * kChunk;
  static constexpr int kStages = D == 128 ? 5 : 8;  // K and V tiles in flight
  static constexpr int kOffQ = 0;
  static constexpr int kOffKV = kTiles * kTile;
  static constexpr int kOffBar = kOffKV + kStages * kTile;
  static constexpr int kAlloc = kOffBar + 512 + 1024;
};

struct Bars {
  uint64_t q_full[kTiles], q_empty[kTiles];
  uint64_t kv_full[8], kv_empty[8];
  uint64_t tail;  // a V tile with rows to clear has landed
  uint64_t s_full[kTiles], p_full[kTiles];
  uint64_t o_full[kTiles], o_empty[kTiles];
  uint64_t drained;
  uint32_t tmem_base;
};

struct Item {
  int b, g, pos0, n, steps;
  KeyTiles kt;
  __device__ Item(const WindowParams& p, int P, const ItemWalk& w)
      : b(w.b),
        g(w.g),
        pos0((w.n_x - 1 - w.x) * kTiles * P),  // the longest rows of a causal prompt first
        n(window_len(p, b)),
        kt(pos0, min(pos0 + kTiles * P, n), p.window, p.sinks, kStep) {
    steps = pos0 < n ? kt.n : 0;
  }
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    window_fwd_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const WindowParams p, int n_pairs) {
  using L = Layout<D>;
  constexpr int kStages = L::kStages;
  constexpr bool kBF16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr uint32_t kIdescS = tc::idesc_f16(kRows, kStep, kBF16, false, false);
  constexpr uint32_t kIdescO = tc::idesc_f16(kRows, D, kBF16, false, true);

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + L::kOffBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lg = __ffs(p.G) - 1, P = kRows >> lg;

  if (threadIdx.x == 0) {
    for (int x = 0; x < kStages; ++x) {
      tc::mbar_init(&bars->kv_full[x], 1);
      tc::mbar_init(&bars->kv_empty[x], 1);
    }
    tc::mbar_init(&bars->tail, 1);
    tc::mbar_init(&bars->drained, 1);
    for (int t = 0; t < kTiles; ++t) {
      tc::mbar_init(&bars->q_full[t], 1);
      tc::mbar_init(&bars->q_empty[t], 1);
      tc::mbar_init(&bars->s_full[t], 1);
      tc::mbar_init(&bars->p_full[t], kRows / 32);
      tc::mbar_init(&bars->o_full[t], 1);
      tc::mbar_init(&bars->o_empty[t], kRows / 32);
    }
    tc::fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(&bars->tmem_base, 512);
    tc::tmem_relinquish();
  }
  if (warp == kProducerWarp && lane == 0) {
    tc::prefetch_tensormap(&tm_q);
    tc::prefetch_tensormap(&tm_k);
    tc::prefetch_tensormap(&tm_v);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = bars->tmem_base;
  bool ok = true;

  if (warp >= 4 * kTiles) {
    reg_dec<kOtherRegs>();
    if (warp == kProducerWarp) {
      // ------------------------------------------------------------ producer
      if (blockIdx.x == 0) begin_status(p, lane);
      int kv = 0, items = 0, tails = 0;  // ring slots filled, items with steps, cleared tiles
      int q[kTiles] = {};                // Q tiles brought in
      for (ItemWalk it(n_pairs, p.Hkv, p.B); ok && it.any(); it.next()) {
        const Item w(p, P, it);
        if (w.steps == 0) continue;
        for (int t = 0; ok && t < kTiles; ++t) {
          if (items > 0 && !(ok = warp_wait(&bars->q_empty[t], items - 1))) break;
          if (lane == 0) {
            tc::mbar_arrive_expect_tx(&bars->q_full[t], L::kTile);
            for (int kc = 0; kc < L::KC; ++kc)
              tc::tma_load_4d(smem + L::kOffQ + t * L::kTile + kc * L::kChunk, &tm_q, &bars->q_full[t], kc * 64,
                              w.g * p.G, w.pos0 + t * P, w.b);
          }
          ++q[t];
        }
        ++items;
        for (int x = 0; ok && x < 2 * w.steps; ++x, ++kv) {  // K and V of each step
          const int st = kv % kStages, tok0 = w.kt.tile(x >> 1) * kStep;
          if (kv >= kStages) ok = warp_wait(&bars->kv_empty[st], kv / kStages - 1);
          if (!ok) break;
          uint8_t* dst = smem + L::kOffKV + st * L::kTile;
          const bool is_v = x & 1;
          const bool clear = is_v && tok0 + kStep > w.n && w.n < p.S;
          uint64_t* bar = clear ? &bars->tail : &bars->kv_full[st];
          if (lane == 0) {
            tc::mbar_arrive_expect_tx(bar, L::kTile);
            for (int kc = 0; kc < L::KC; ++kc)
              tc::tma_load_4d(dst + kc * L::kChunk, is_v ? &tm_v : &tm_k, bar, kc * 64, w.g, tok0, w.b);
          }
          if (clear) {
            ok = warp_wait(&bars->tail, tails++);
            zero_tile_rows(dst, L::KC, kStep, w.n - tok0, lane);
            if (lane == 0) tc::mbar_arrive(&bars->kv_full[st]);
          }
        }
      }
      // every copy lands before the CTA retires
      for (int t = 0; t < kTiles; ++t)
        if (q[t] > 0) tc::mbar_wait(&bars->q_full[t], (q[t] - 1) & 1);
      for (int j = max(0, kv - kStages); j < kv; ++j) tc::mbar_wait(&bars->kv_full[j % kStages], (j / kStages) & 1);
      if (!ok) raise_status(p.status, 5 /* DASH_ERR_DEVICE_TIMEOUT */, 321);
    } else if (warp == kMmaWarp) {
      // ------------------------------------------------------------ MMA issuer
      auto wait = [&](uint64_t* bar, int phase) {
        ok = ok && warp_wait(bar, phase);
        tc::fence_after_sync();
        return ok;
      };
      const uint64_t q0 = tc::smem_desc_sw128(smem + L::kOffQ, 16, 1024);
      const uint64_t k0 = tc::smem_desc_sw128(smem + L::kOffKV, 16, 1024);
      const uint64_t v0 = tc::smem_desc_sw128(smem + L::kOffKV, L::kChunk, 1024);
      int x = 0, items = 0;           // steps and items so far: K of step x is ring tile 2 x, V is 2 x + 1
      bool first = false, last = false;  // whether the step before was the first / last of its item
      // O(t) += P(t) V of the step before, of the CTA's `item`-th item
      auto issue_pv = [&](int t, int item) {
        const int y = x - 1, v = 2 * y + 1;
        if (t == 0 && !wait(&bars->kv_full[v % kStages], v / kStages)) return;
        if (first && item > 1 && !wait(&bars->o_empty[t], item - 2)) return;
        if (!wait(&bars->p_full[t], y)) return;
        const uint64_t vd = v0 + (uint64_t)(((v % kStages) * L::kTile) >> 4);
        const uint32_t d_tm = tmem + kColO + t * 128, a_tm = tmem + kColS + t * 128;
#pragma unroll
        for (int k = 0; k < kStep / 16; ++k)
          tc::mma_f16_ts_w(d_tm, a_tm + k * 8, vd + (uint64_t)((k * 2048) >> 4), kIdescO, (!first || k > 0) ? 1u : 0u);
        if (last) tc::mma_commit_w(&bars->o_full[t]);
        if (t == kTiles - 1) tc::mma_commit_w(&bars->kv_empty[v % kStages]);
      };
      for (ItemWalk it(n_pairs, p.Hkv, p.B); ok && it.any(); it.next()) {
        const Item w(p, P, it);
        if (w.steps == 0) continue;
        ++items;
        for (int i = 0; ok && i < w.steps; ++i, ++x) {
          const int kt = 2 * x;
          const uint64_t kd = k0 + (uint64_t)(((kt % kStages) * L::kTile) >> 4);
#pragma unroll 1
          for (int t = 0; t < kTiles; ++t) {
            if (x > 0) issue_pv(t, items - (i == 0));
            if (t == 0) wait(&bars->kv_full[kt % kStages], kt / kStages);
            if (i == 0) wait(&bars->q_full[t], items - 1);
            if (!ok) break;
            const uint64_t qd = q0 + (uint64_t)((t * L::kTile) >> 4);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint64_t off = (uint64_t)((((k >> 2) * L::kChunk) + (k & 3) * 32) >> 4);
              tc::mma_f16_ss_w(tmem + kColS + t * 128, qd + off, kd + off, kIdescS, k > 0 ? 1u : 0u);
            }
            tc::mma_commit_w(&bars->s_full[t]);
            if (i == w.steps - 1) tc::mma_commit_w(&bars->q_empty[t]);
          }
          if (!ok) break;
          tc::mma_commit_w(&bars->kv_empty[kt % kStages]);
          first = i == 0;
          last = i == w.steps - 1;
        }
      }
      if (x > 0)
        for (int t = 0; ok && t < kTiles; ++t) issue_pv(t, items);
      if (!ok) raise_status(p.status, 5, 322);
      tc::mma_commit_w(&bars->drained);
      tc::mbar_wait(&bars->drained, 0);
    }
  } else {
    // ------------------------------------------------------------ softmax
    reg_inc<kSoftmaxRegs>();
    const int t = warp >> 2, q4 = warp & 3, r = q4 * 32 + lane;
    const uint32_t tb = tmem + ((uint32_t)(q4 * 32) << 16);
    const uint32_t tb_o = tb + kColO + t * 128;
    const float qk_scale = rsqrtf((float)D) * kLog2e;
    int items = 0, step = 0;
    for (ItemWalk it(n_pairs, p.Hkv, p.B); ok && it.any(); it.next()) {
      const Item w(p, P, it);
      const int pos_a = w.pos0 + t * P, lo_b = pos_a + P - p.window;  // the tile's first position, its last row's lo
      const int pos = pos_a + (r >> lg), head = w.g * p.G + (r & (p.G - 1));
      const int lo = pos - p.window + 1;  // first key of the row's window
      // a row behind the end starts from +inf: its p are 0 or NaN, and never call for another reference
      float m_used = pos < w.n ? kNegInf : -kNegInf, lsum = 0.f;
      for (int i = 0; i < w.steps; ++i) {
        const int x = step + i, tok0 = w.kt.tile(i) * kStep;
        if (!(ok = warp_wait(&bars->s_full[t], x))) break;
        tc::fence_after_sync();
        const uint32_t tb_s = tb + kColS + t * 128;
        uint32_t sv[kStep];
#pragma unroll
        for (int c = 0; c < 4; ++c) tc::tmem_ld32(tb_s + c * 32, sv + c * 32);
        tc::tmem_wait_ld();
        const bool edge = tok0 + kStep - 1 > pos_a || tok0 < lo_b;
        if (edge) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int t0 = tok0 + c * 32;
            const uint32_t seen = bit_range(lo - t0, pos - t0) | bit_range(0, min(pos, p.sinks - 1) - t0);
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!(seen & (1u << j))) sv[c * 32 + j] = __float_as_uint(kNegInf);
          }
        }
        // p = 2^(s scale + off) into tensor memory; their sum.  Two pairs at a
        // time: while their exponentials run, the two before are summed and
        // packed and the two after scaled (1.09 -> 1.05 ms for a 32K prompt
        // with window 2048 against the compiler's order).
        auto exps = [&](float off) -> float {
          const float2 sc2 = make_float2(qk_scale, qk_scale), off2 = make_float2(off, off);
          auto scaled = [&](int j) {
            return __ffma2_rn(make_float2(__uint_as_float(sv[2 * j]), __uint_as_float(sv[2 * j + 1])), sc2, off2);
          };
          constexpr int kPairs = kStep / 2;
          float2 sum[4], y[4], z[4];
          uint32_t pw[16];
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[e] = make_float2(0.f, 0.f);
          y[0] = scaled(0);
          y[1] = scaled(1);
#pragma unroll
          for (int j = 0; j < kPairs + 2; ++j) {
            const int o = j - 2;  // the pair that is finished here
            if (j < kPairs) z[j & 3].x = ex2_placed(y[j & 3].x);
            if (o >= 0) sum[o & 3] = __fadd2_rn(sum[o & 3], z[o & 3]);
            if (j + 2 < kPairs) y[(j + 2) & 3] = scaled(j + 2);
            if (j < kPairs) z[j & 3].y = ex2_placed(y[j & 3].y);
            if (o >= 0) pw[o & 15] = pack2_placed<T>(z[o & 3]);
            if (o >= 0 && (o & 15) == 15) tc::tmem_st16(tb_s + (o >> 4) * 16, pw);
          }
          const float2 s = __fadd2_rn(__fadd2_rn(sum[0], sum[1]), __fadd2_rn(sum[2], sum[3]));
          return s.x + s.y;
        };
        // the stores in exps are warp-wide, so the warp takes one path: the
        // second one when a row of it has no reference yet or left its range
        float corr = 1.f, lstep = 0.f;
        bool moves = m_used == kNegInf;  // this row takes its maximum
        if (__any_sync(0xffffffffu, !moves)) {
          lstep = exps(moves ? 0.f : -m_used);
          moves = moves || lstep > kMaxSum;
        }
        if (__any_sync(0xffffffffu, moves)) {
          float mx = kNegInf;
#pragma unroll
          for (int j = 0; j < kStep; ++j) mx = fmaxf(mx, __uint_as_float(sv[j]));
          mx *= qk_scale;
          bool resc = false;
          if (moves && mx != kNegInf) {
            if (m_used == kNegInf) {
              m_used = mx;
            } else if (mx > m_used + kRescaleLog2) {
              corr = tc::ex2(m_used - mx);
              m_used = mx;
              resc = true;
            }
          }
          lstep = exps(m_used == kNegInf ? 0.f : -m_used);
          if (__any_sync(0xffffffffu, resc)) {
            // O is stable: P V of the step before ended before this S
#pragma unroll 1
            for (int cc = 0; cc < D / 32; ++cc) {
              uint32_t ov[32];
              tc::tmem_ld32(tb_o + cc * 32, ov);
              tc::tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; ++j) ov[j] = __float_as_uint(__uint_as_float(ov[j]) * corr);
              tc::tmem_st32(tb_o + cc * 32, ov);
            }
          }
        }
        lsum = lsum * corr + lstep;
        tc::tmem_wait_st();
        tc::fence_before_sync();
        warp_arrive(&bars->p_full[t], lane);
      }
      if (!ok) break;
      // ---- the rows' output (zeros where there is no token) and log-sum-exp
      const bool live = pos < w.n;
      if (p.lse && pos < p.S)
        p.lse[((int64_t)w.b * p.H + head) * p.S + pos] = live ? (m_used + log2f(lsum)) / kLog2e : kNegInf;
      const float inv = live ? 1.f / lsum : 0.f;
      if (w.steps > 0) {
        if (!(ok = warp_wait(&bars->o_full[t], items))) break;
        tc::fence_after_sync();
      }
      T* dst = static_cast<T*>(const_cast<void*>(p.out.data)) + (int64_t)w.b * p.out.sb +
               (int64_t)min(pos, p.S - 1) * p.out.ss + (int64_t)head * p.out.sh;
#pragma unroll
      for (int cc = 0; cc < D / 32; ++cc) {
        uint32_t ov[32];
        if (w.steps > 0) {
          tc::tmem_ld32(tb_o + cc * 32, ov);
          tc::tmem_wait_ld();
        }
        if (!live) {
#pragma unroll
          for (int j = 0; j < 32; ++j) ov[j] = 0u;
        }
        if (pos < p.S) {
          store_row32(dst + cc * 32, ov, inv, p.wide);
          if (p.rest.data) {
            rounding_rest<T>(ov, inv);
            T* rest = static_cast<T*>(const_cast<void*>(p.rest.data)) + (int64_t)w.b * p.rest.sb +
                      (int64_t)pos * p.rest.ss + (int64_t)head * p.rest.sh;
            store_row32(rest + cc * 32, ov, 1.f, p.wide);
          }
        }
      }
      if (w.steps > 0) {
        tc::fence_before_sync();
        warp_arrive(&bars->o_empty[t], lane);
        step += w.steps;
        ++items;
      }
    }
    if (!ok) raise_status(p.status, 5, 323);
  }

  tc::fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

template <typename T, int D>
cudaError_t run(const WindowParams& p, cudaStream_t stream) {
  using L = Layout<D>;
  CUtensorMap mq, mk, mv;
  const int P = kRows / p.G;
  if (!window_map(&mq, p.q, p.dtype, p.B, p.S, p.H, D, p.G, P) ||
      !window_map(&mk, p.k, p.dtype, p.B, p.S, p.Hkv, D, 1, kStep) ||
      !window_map(&mv, p.v, p.dtype, p.B, p.S, p.Hkv, D, 1, kStep))
    return cudaErrorInvalidValue;
  auto kern = window_fwd_tc_kernel<T, D>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
  if (e != cudaSuccess) return e;
  const int64_t n_pairs = (p.S + kTiles * P - 1) / (kTiles * P), n_items = n_pairs * p.Hkv * p.B;
  if (n_items > 0x7fffffff - 4096) return cudaErrorInvalidValue;
  kern<<<(unsigned)std::min<int64_t>(n_items, p.num_sms), kThreads, L::kAlloc, stream>>>(mq, mk, mv, p,
                                                                                         (int)n_pairs);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_window_fwd_tc(const WindowParams& p, cudaStream_t stream) {
  if (p.D == 128) return p.dtype == 1 ? run<__half, 128>(p, stream) : run<__nv_bfloat16, 128>(p, stream);
  return p.dtype == 1 ? run<__half, 64>(p, stream) : run<__nv_bfloat16, 64>(p, stream);
}

}  // namespace dash
