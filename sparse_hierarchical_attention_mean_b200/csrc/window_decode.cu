// Attention of one new token per sequence over its KV cache (dense or paged),
// whole context or sliding window + first tokens, split over the cache.
//
// The token of sequence b stands at L - 1 (L = seqlens[b]) and sees the
// tokens t < L with t >= L - window or t < sinks:
//   o_h = sum_t p_t v_t / sum_t p_t,  p_t = 2^(q_h . k_t log2(e) / sqrt(D) - m)
//
// Bound by reading the visible K and V once.  The unit of work is a step of
// 64 tokens of one (sequence, KV head); the steps of all of them, in order,
// are one line that is cut into parts, one per CTA (Cut below), so every SM
// streams the same number of bytes whatever the lengths.  A CTA is one producer warp,
// which fills a ring of shared-memory stages (K and V of a step, two TMA
// copies each at D = 128; the block table is read 32 entries at a time), and four
// consumer warps that own 16 tokens of each step.  A (sequence, KV head) that
// falls into one CTA is finished there; one that a cut divides leaves a
// partial (o, m, l) per CTA, at most two per CTA, and the join kernel merges
// them in order (the result does not depend on timing).
//
// With 64-wide heads a unit takes two adjacent KV heads (HP = 2), two consumer
// warps each: one head's 128 bytes of a token at a time reached 4.4 TB/s.
//
// G <= 8 query heads are rows 0-7 of a warp-level m16n8k16 MMA (the products
// need 1% of the tensor rate, the 64-row minimum of tcgen05 would waste eight
// times that).  In the second product P goes into rows 0-7 rounded to the
// cache's type, the MMA's operand type, and what that rounding took, rounded
// too, into rows 8-15, which are padding otherwise: no further MMA, and P's
// error is u^2 of it instead of u (rounded once, P added as much to the
// output's error as the output's own rounding does).  It costs no time: 64 x
// 4096 visible tokens 96.6 us in a graph with and without, 32 x 48K 930 and
// 928.  m, l and o are fp32.
//
// What stands in the cache at masked tokens is never used: masked logits are
// replaced before the maximum, and masked V values are cleared in registers
// (only in the steps that hold a mask's edge), so NaN there is harmless.
#include <cuda.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "mma_sync.cuh"
#include "tc.cuh"
#include "window.h"

namespace dash {
namespace {

constexpr int kStep = 64;
constexpr int kConsumers = 4;
constexpr int kThreads = (kConsumers + 1) * 32;
constexpr int kPairSteps = 2;   // steps of pairs of heads a CTA gets at least, or heads go one by one

template <int D, int HP>
struct Layout {
  static constexpr int KC = HP * D / 64;             // 64-column chunks of a token
  static constexpr int kChunk = kStep * 128;         // 64 tokens x 128 bytes
  static constexpr int kTile = KC * kChunk;          // K (or V) of a step
  static constexpr int kStages = 12 / KC;            // 192 KB in flight per SM
  static constexpr int kOffO = 2 * kStages * kTile;  // merge buffer [4][8][D] fp32
  static constexpr int kOffMl = kOffO + kConsumers * 8 * D * 4;
  static constexpr int kOffBar = kOffMl + kConsumers * 8 * 2 * 4;
  static constexpr int kBytes = kOffBar + 2 * kStages * 8 + 16;
  static constexpr int kAlloc = kBytes + 1024;
};

// The steps of one sequence: sink tiles that end before the band, then the band.
struct SeqSteps {
  int L, lo, n_sink, band0, n;
  __device__ SeqSteps(const WindowDecodeParams& p, int b) {
    const int raw = p.seqlens[b];
    L = (int)min((int64_t)max(raw, 0), p.Lmax);
    lo = p.window > 0 ? max(0, L - p.window) : 0;
    band0 = lo / kStep;
    n_sink = min((p.sinks + kStep - 1) / kStep, band0);
    n = n_sink + (L + kStep - 1) / kStep - band0;
  }
  __device__ int tok0(int s) const { return (s < n_sink ? s : band0 + s - n_sink) * kStep; }
};

// Steps of the sequences [b0, b0 + 32), one per lane (0 past the batch).
__device__ __forceinline__ int lane_steps(const WindowDecodeParams& p, int b0, int lane) {
  return b0 + lane < p.B ? SeqSteps(p, b0 + lane).n : 0;
}

__device__ __forceinline__ long long warp_sum_ll(long long x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Steps of the whole batch per KV head (every lane of a warp calls it), and
// the steps of the sequences before b.
__device__ __forceinline__ void batch_steps(const WindowDecodeParams& p, int b, int lane, long long* total,
                                            long long* before) {
  long long t = 0, f = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int n = lane_steps(p, b0, lane);
    t += n;
    if (b0 + lane < b) f += n;
  }
  *total = warp_sum_ll(t);
  if (before) *before = warp_sum_ll(f);
}

// How the line of `units` steps is cut: n parts of `per` whole steps each, the
// last maybe shorter.  No part is longer than with n_cta equal parts (which
// end within a step of each other too), and more cuts fall between two units,
// which saves a CTA a second merge: 512 steps of 32 units 9.3 us instead of
// 10.2; long lines gained up to 4% in a graph, nothing on cold caches.  At least 2 or 4 steps
// a part (fewer partials to join) were slower: one sequence of 1792 tokens 8.3
// us with 2, 9.2 with 4; of 640 tokens 7.0 with 1, 7.4 with 2.
struct Cut {
  long long units, per;
  int n;
  __device__ Cut(long long u, int n_cta)
      : units(u), per(max(1ll, (u + n_cta - 1) / n_cta)), n((int)((u + per - 1) / per)) {}
  __device__ long long start(int c) const { return min(units, per * c); }
  __device__ int owner(long long u) const { return (int)(u / per); }
};

// Walks a part of the line: the (sequence, KV head or pair of them) segments in
// order.
struct Walk {
  int b, g, s0, s1;    // segment: steps [s0, s1) of (b, g)
  bool whole;          // the segment is all of (b, g)
  bool head;           // it starts before this part
  long long left;      // steps of the part from s0 on
  __device__ bool begin(const WindowDecodeParams& p, const Cut& cut, int c, int lane) {
    long long u = cut.start(c);
    left = cut.start(c + 1) - u;
    if (c >= cut.n || left <= 0) return false;
    // the sequence that holds step u
    long long base = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const long long n = (long long)lane_steps(p, b0, lane) * p.units;
      long long inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, base + inc > u);
      if (hit) {
        const int w = __ffs(hit) - 1;
        const long long first = base + __shfl_sync(0xffffffffu, inc - n, w);
        const int steps = (int)(__shfl_sync(0xffffffffu, n, w) / p.units);
        b = b0 + w;
        g = (int)((u - first) / steps);
        s0 = (int)((u - first) % steps);
        return true;
      }
      base += __shfl_sync(0xffffffffu, inc, 31);
    }
    return false;
  }
  __device__ void open(const SeqSteps& q) {
    s1 = (int)min((long long)q.n, s0 + left);
    whole = s0 == 0 && s1 == q.n;
    head = s0 > 0;
  }
  // to the next segment; false at the end of the part
  __device__ bool next(const WindowDecodeParams& p, SeqSteps& q) {
    left -= s1 - s0;
    if (left <= 0) return false;
    s0 = 0;
    if (++g == p.units) {
      g = 0;
      do {
        ++b;
        q = SeqSteps(p, b);
      } while (q.n == 0);
    }
    return true;
  }
};

// A packed pair as floats.
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (std::is_same<T, __half>::value)
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  else
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

template <typename T, int D, int HP>
__global__ void __launch_bounds__(kThreads, 1)
    window_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                         const WindowDecodeParams p) {
  using L = Layout<D, HP>;
  constexpr int kStages = L::kStages;
  constexpr int KS = D / 16;             // k slices of S = Q K^T
  constexpr int NT = D / 8;              // 8-wide tiles of O
  constexpr int kShare = kConsumers / HP;  // warps of a KV head
  constexpr int TG = kStep / kShare / 16;  // 16-token groups of a warp in a step
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* obuf = reinterpret_cast<float*>(smem + L::kOffO);
  float* mlbuf = reinterpret_cast<float*>(smem + L::kOffMl);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint64_t* empty = full + kStages;
  int* bad = reinterpret_cast<int*>(empty + kStages);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], kConsumers);
    }
    *bad = 0;
    tc::fence_barrier_init();
  }
  if (warp == kConsumers && lane == 0) {
    tc::prefetch_tensormap(&tm_k);
    tc::prefetch_tensormap(&tm_v);
  }
  __syncthreads();

  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  long long total;
  batch_steps(p, 0, lane, &total, nullptr);
  const Cut cut(total * p.units, p.n_cta);
  Walk w;
  const bool any = total > 0 && w.begin(p, cut, blockIdx.x, lane);

  if (any && warp == kConsumers) {
    // ------------------------------------------------------------ producer
    SeqSteps q(p, w.b);
    int i = 0, pages = 0;
    bool ok = true;
    do {
      w.open(q);
      for (int s = w.s0; ok && s < w.s1; ++s) {
        const int tok = q.tok0(s);
        int c2 = tok, c3 = w.b;
        if (p.block_table) {
          // 32 page numbers at a time, one per lane
          if (((s - w.s0) & 31) == 0)
            pages = s + lane < w.s1
                        ? __ldg(p.block_table + (int64_t)w.b * p.max_blocks + q.tok0(s + lane) / p.block)
                        : 0;
          const int page = __shfl_sync(0xffffffffu, pages, (s - w.s0) & 31);
          c2 = tok % p.block;
          c3 = page;
          if (page < 0 || page >= p.n_pages) {
            if (lane == 0) atomicMax(bad, 1 /* DASH_ERR_INVALID_ARGUMENT */);
            c3 = (int)p.n_pages;  // past the pool's end: the copy fills the stage with zeros
          }
        }
        const int st = i % kStages;
        if (i >= kStages) ok = tc::mbar_wait(&empty[st], ((i / kStages) - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          tc::mbar_arrive_expect_tx(&full[st], 2 * L::kTile);
#pragma unroll
          for (int kc = 0; kc < L::KC; ++kc) {
            uint8_t* dst = smem + st * 2 * L::kTile + kc * L::kChunk;
            const int col = HP == 2 ? 0 : kc * 64, head = HP == 2 ? w.g * 2 + kc : w.g;
            tc::tma_load_4d(dst, &tm_k, &full[st], col, head, c2, c3);
            tc::tma_load_4d(dst + L::kTile, &tm_v, &full[st], col, head, c2, c3);
          }
        }
        ++i;
      }
    } while (ok && w.next(p, q));
    if (!ok && lane == 0) atomicMax(bad, 5 /* DASH_ERR_DEVICE_TIMEOUT */);
    // every copy lands before the CTA retires
    for (int j = i > kStages ? i - kStages : 0; j < i; ++j) tc::mbar_wait(&full[j % kStages], (j / kStages) & 1);
  } else if (any) {
    // ------------------------------------------------------------ consumers
    const int G = p.G, gq = lane >> 2, tq = lane & 3;
    const int hs = warp / kShare, tok_w = warp % kShare * TG * 16;  // KV head of the unit, first token of a step
    const float qk_scale = rsqrtf((float)D) * kLog2e;
    SeqSteps q(p, w.b);
    int i = 0;
    bool ok = true;
    do {
      w.open(q);
      // A fragments of the query heads (rows gq >= G and 8..15 are zero)
      uint32_t qa[KS][2];
      {
        const T* src = static_cast<const T*>(p.q.data) + (int64_t)w.b * p.q.sb +
                       (int64_t)((w.g * HP + hs) * G + gq) * p.q.sh;
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
          qa[kk][0] = gq < G ? *reinterpret_cast<const uint32_t*>(src + kk * 16 + 2 * tq) : 0u;
          qa[kk][1] = gq < G ? *reinterpret_cast<const uint32_t*>(src + kk * 16 + 8 + 2 * tq) : 0u;
        }
      }
      float o[NT][4];  // [..][0, 1]: of P's high part; [2, 3]: of its low part
#pragma unroll
      for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
      float m_used = kNegInf, lpart = 0.f;
      for (int s = w.s0; s < w.s1; ++s, ++i) {
        const int st = i % kStages;
        // a wait that ran out ends this warp's work, but not its part in the
        // CTA's named barriers below
        ok = ok && __all_sync(0xffffffffu, tc::mbar_wait(&full[st], (i / kStages) & 1));
        if (!ok) break;
        const uint32_t kst = smem_u32(smem + st * 2 * L::kTile), vst = kst + L::kTile;
        const int mt = lane >> 3, rr = lane & 7;
        // S = Q K^T of this warp's tokens, 8 a tile
        float sacc[2 * TG][4];
#pragma unroll
        for (int n = 0; n < 2 * TG; ++n) sacc[n][0] = sacc[n][1] = sacc[n][2] = sacc[n][3] = 0.f;
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
          const int c = 2 * (kk & 3) + (mt & 1), chunk = HP == 2 ? hs : kk >> 2;
          const uint32_t a[4] = {qa[kk][0], 0u, qa[kk][1], 0u};
#pragma unroll
          for (int t = 0; t < TG; ++t) {
            const int row = tok_w + t * 16 + (mt >> 1) * 8 + rr;
            uint32_t bf[4];
            ldsm_x4(kst + chunk * L::kChunk + row * 128 + ((c ^ (row & 7)) << 4), bf);
            mma16816<T>(sacc[2 * t], a, bf[0], bf[1]);
            mma16816<T>(sacc[2 * t + 1], a, bf[2], bf[3]);
          }
        }
        // logits of head gq (log2 units) for tokens 8 n + 2 tq and the next one
        const int tok0 = q.tok0(s);
        const bool edge = tok0 + kStep > q.L || tok0 < q.lo;  // some token of the step may be hidden
        uint32_t vm[2 * TG];
        float mx = kNegInf;
#pragma unroll
        for (int n = 0; n < 2 * TG; ++n) {
          vm[n] = 0xffffffffu;
          sacc[n][0] *= qk_scale;
          sacc[n][1] *= qk_scale;
          if (edge) {
            const int t = tok0 + tok_w + n * 8 + 2 * tq;
            const bool s0 = t < q.L && (t >= q.lo || t < p.sinks);
            const bool s1 = t + 1 < q.L && (t + 1 >= q.lo || t + 1 < p.sinks);
            if (!s0) sacc[n][0] = kNegInf;
            if (!s1) sacc[n][1] = kNegInf;
            vm[n] = (s0 ? 0xffffu : 0u) | (s1 ? 0xffff0000u : 0u);
          }
          mx = fmaxf(mx, fmaxf(sacc[n][0], sacc[n][1]));
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        float corr = 1.0f;
        bool resc = false;
        if (mx != kNegInf) {
          if (m_used == kNegInf) {
            m_used = mx;
          } else if (mx > m_used + 8.0f) {  // P stays <= 2^8, in range of both types
            corr = tc::ex2(m_used - mx);
            m_used = mx;
            resc = true;
          }
        }
        if (__any_sync(0xffffffffu, resc)) {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            o[n][0] *= corr;
            o[n][1] *= corr;
            o[n][2] *= corr;
            o[n][3] *= corr;
          }
          lpart *= corr;
        }
        const float off = m_used == kNegInf ? 0.f : m_used;
        uint32_t pw[2 * TG], pl[2 * TG];
#pragma unroll
        for (int n = 0; n < 2 * TG; ++n) {
          const float e0 = tc::ex2(sacc[n][0] - off), e1 = tc::ex2(sacc[n][1] - off);
          lpart += e0 + e1;
          pw[n] = pack2<T>(e0, e1);
          const float2 hi = unpack2<T>(pw[n]);
          pl[n] = pack2<T>(e0 - hi.x, e1 - hi.y);
        }
        // O += P V
#pragma unroll
        for (int t = 0; t < TG; ++t) {
          const uint32_t pa[4] = {pw[2 * t], pl[2 * t], pw[2 * t + 1], pl[2 * t + 1]};
          const int row = tok_w + t * 16 + (mt & 1) * 8 + rr;
#pragma unroll
          for (int j = 0; j < NT / 2; ++j) {
            const int c = 2 * j + (mt >> 1), chunk = HP == 2 ? hs : c >> 3;
            uint32_t bf[4];
            ldsm_x4_t(vst + chunk * L::kChunk + row * 128 + (((c & 7) ^ (row & 7)) << 4), bf);
            if (edge) {
              bf[0] &= vm[2 * t];
              bf[1] &= vm[2 * t + 1];
              bf[2] &= vm[2 * t];
              bf[3] &= vm[2 * t + 1];
            }
            mma16816<T>(o[2 * j], pa, bf[0], bf[1]);
            mma16816<T>(o[2 * j + 1], pa, bf[2], bf[3]);
          }
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&empty[st]);
      }
      // merge the warps of each KV head
      float l = lpart;
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      if (gq < G) {
        if (tq == 0) {
          mlbuf[(warp * 8 + gq) * 2] = m_used;
          mlbuf[(warp * 8 + gq) * 2 + 1] = l;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
          *reinterpret_cast<float2*>(obuf + (warp * 8 + gq) * D + n * 8 + 2 * tq) =
              make_float2(o[n][0] + o[n][2], o[n][1] + o[n][3]);
      }
      asm volatile("bar.sync 1, %0;\n" ::"n"(kConsumers * 32) : "memory");
      const int64_t slot = 2 * (int64_t)blockIdx.x + (w.head ? 0 : 1);
      for (int e = threadIdx.x * 2; e < HP * G * D; e += kConsumers * 64) {
        const int uh = e / D, c = e % D;  // query head of the unit
        const bool second = HP == 2 && uh >= G;
        const int w0 = second ? kShare : 0, h = second ? uh - G : uh;
        float M = kNegInf;
#pragma unroll
        for (int u = 0; u < kShare; ++u) M = fmaxf(M, mlbuf[((w0 + u) * 8 + h) * 2]);
        const float Mu = M == kNegInf ? 0.f : M;
        float a0 = 0.f, a1 = 0.f, sum = 0.f;
#pragma unroll
        for (int u = 0; u < kShare; ++u) {
          const float f = tc::ex2(mlbuf[((w0 + u) * 8 + h) * 2] - Mu);
          const float2 ov = *reinterpret_cast<const float2*>(obuf + ((w0 + u) * 8 + h) * D + c);
          a0 = fmaf(f, ov.x, a0);
          a1 = fmaf(f, ov.y, a1);
          sum = fmaf(f, mlbuf[((w0 + u) * 8 + h) * 2 + 1], sum);
        }
        if (w.whole) {
          const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);  // NaN stays NaN
          const int head = w.g * HP * G + uh;
          T* dst = static_cast<T*>(const_cast<void*>(p.out.data)) + (int64_t)w.b * p.out.sb + (int64_t)head * p.out.sh;
          *reinterpret_cast<uint32_t*>(dst + c) = pack2<T>(a0 * inv, a1 * inv);
          if (p.lse && c == 0)
            p.lse[(int64_t)w.b * p.H + head] = sum == 0.f ? kNegInf : (M + log2f(sum)) / kLog2e;
        } else {
          *reinterpret_cast<float2*>(p.part_o + (slot * HP * G + uh) * D + c) = make_float2(a0, a1);
          if (c == 0) *reinterpret_cast<float2*>(p.part_ml + (slot * HP * G + uh) * 2) = make_float2(M, sum);
        }
      }
      asm volatile("bar.sync 1, %0;\n" ::"n"(kConsumers * 32) : "memory");
    } while (w.next(p, q));
    if (!ok && lane == 0) atomicMax(bad, 5 /* DASH_ERR_DEVICE_TIMEOUT */);
  }
  __syncthreads();
  if (threadIdx.x == 0) p.cta_status[blockIdx.x] = *bad;
}

// One CTA per (unit's KV heads, sequence): merges the partials of a divided one in
// order, writes zeros for a sequence without tokens; the first CTA also
// writes the status word (its last warp, so that no weight waits for that).
// Bound by latency: a thread asks for the outputs of the first 16 parts, then a
// warp per head makes the weights of all parts, so that the two loads overlap
// (one sequence of 1792 tokens, in a graph with the kernel before: 11.5 us
// without, 9.7 with the first 8 parts, 8.2 with 16).
constexpr int kJoinThreads = 256;
template <typename T, int HP>
__global__ void __launch_bounds__(kJoinThreads) window_decode_join_kernel(const WindowDecodeParams p) {
  __shared__ float weight[kMaxDecodeCtas][8 * HP];  // of part i for head h of the unit, 1 / l included
  const int g = blockIdx.x, b = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = HP * p.G, D = p.D;  // query heads of a unit
  long long total, before;
  batch_steps(p, b, lane, &total, &before);
  const SeqSteps q(p, b);
  const Cut cut(total * p.units, p.n_cta);
  const long long u0 = before * p.units + (long long)g * q.n;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  if (g == 0 && b == 0 && warp == kJoinThreads / 32 - 1) {
    int code = 0;
    for (int c = lane; c < p.n_cta; c += 32) code = max(code, p.cta_status[c]);
    for (int i = lane; i < p.B; i += 32)
      if (p.seqlens[i] < 0 || p.seqlens[i] > p.Lmax) code = max(code, 1 /* DASH_ERR_INVALID_ARGUMENT */);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) code = max(code, __shfl_xor_sync(0xffffffffu, code, o));
    if (lane == 0) {
      p.status->code = code;
      p.status->detail = code ? 311 : 0;
    }
  }
  T* dst = static_cast<T*>(const_cast<void*>(p.out.data)) + (int64_t)b * p.out.sb + (int64_t)g * G * p.out.sh;
  if (q.n == 0) {
    for (int e = threadIdx.x * 2; e < G * D; e += kJoinThreads * 2) {
      *reinterpret_cast<uint32_t*>(dst + (int64_t)(e / D) * p.out.sh + e % D) = 0u;
      if (p.lse && e % D == 0) p.lse[(int64_t)b * p.H + g * G + e / D] = kNegInf;
    }
    return;
  }
  const int c0 = cut.owner(u0), parts = cut.owner(u0 + q.n - 1) - c0 + 1;
  if (parts == 1) return;  // finished by its CTA
  // part i lies in the second slot of the first CTA, then in the first slot of the others
  auto slot = [&](int i) { return 2 * (int64_t)(c0 + i) + (i == 0 ? 1 : 0); };
  constexpr int kAhead = 16;
  float2 ahead[kAhead];
  const int e0 = threadIdx.x * 2;
#pragma unroll
  for (int i0 = 0; i0 < kAhead; i0 += 8)
    if (i0 < parts && e0 < G * D) {
#pragma unroll
      for (int i = i0; i < i0 + 8; ++i)
        ahead[i] = i < parts ? *reinterpret_cast<const float2*>(p.part_o + slot(i) * G * D + e0)
                             : make_float2(0.f, 0.f);
    }
  for (int h = warp; h < G; h += kJoinThreads / 32) {
    float l = 0.f;
    auto part_ml = [&](int i) { return *reinterpret_cast<const float2*>(p.part_ml + (slot(i) * G + h) * 2); };
    const float2 own = lane < parts ? part_ml(lane) : make_float2(kNegInf, 0.f);
    float m = own.x;
    for (int i = lane + 32; i < parts; i += 32) m = fmaxf(m, part_ml(i).x);
    const float M = warp_max(m), Mu = M == kNegInf ? 0.f : M;
    for (int i = lane; i < parts; i += 32) {
      const float2 ml = i == lane ? own : part_ml(i);
      const float f = tc::ex2(ml.x - Mu);
      weight[i][h] = f;
      l = fmaf(f, ml.y, l);
    }
    l = warp_sum(l);
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // NaN stays NaN
    for (int i = lane; i < parts; i += 32) weight[i][h] *= inv;
    if (p.lse && lane == 0) p.lse[(int64_t)b * p.H + g * G + h] = l == 0.f ? kNegInf : (M + log2f(l)) / kLog2e;
  }
  __syncthreads();
  for (int e = threadIdx.x * 2; e < G * D; e += kJoinThreads * 2) {
    const int h = e / D, c = e % D;
    const float* src = p.part_o + (int64_t)h * D + c;
    float a0 = 0.f, a1 = 0.f;
    int rest = 0;
    if (e == e0) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (i < parts) {
          a0 = fmaf(weight[i][h], ahead[i].x, a0);
          a1 = fmaf(weight[i][h], ahead[i].y, a1);
        }
      rest = kAhead;
    }
#pragma unroll 8
    for (int i = rest; i < parts; ++i) {
      const float2 ov = *reinterpret_cast<const float2*>(src + slot(i) * G * D);
      a0 = fmaf(weight[i][h], ov.x, a0);
      a1 = fmaf(weight[i][h], ov.y, a1);
    }
    *reinterpret_cast<uint32_t*>(dst + (int64_t)h * p.out.sh + c) = pack2<T>(a0, a1);
  }
}

template <typename T, int D, int HP>
cudaError_t run(WindowDecodeParams p, cudaStream_t stream) {
  using L = Layout<D, HP>;
  p.units = p.Hkv / HP;
  CUtensorMap mk, mv;
  const int64_t rows = p.block_table ? p.block : p.Lmax, outer = p.block_table ? p.n_pages : p.B;
  // a single 64-wide head: with 256-byte L2 fetches the next head's 128 bytes
  // came too and were gone again before their turn (705 MB read for 537)
  const bool narrow = D == 64 && HP == 1;
  if (!window_map(&mk, p.k, p.dtype, outer, rows, p.Hkv, D, 1, kStep, narrow) ||
      !window_map(&mv, p.v, p.dtype, outer, rows, p.Hkv, D, 1, kStep, narrow))
    return cudaErrorInvalidValue;
  auto kern = window_decode_kernel<T, D, HP>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
  if (e != cudaSuccess) return e;
  kern<<<p.n_cta, kThreads, L::kAlloc, stream>>>(mk, mv, p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  // the join's launch overlaps the streaming kernel's end; it waits for its results itself
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.units, p.B);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, window_decode_join_kernel<T, HP>, p);
}

}  // namespace

cudaError_t launch_window_decode(const WindowDecodeParams& p, cudaStream_t stream) {
  if (p.D == 128)
    return p.dtype == 1 ? run<__half, 128, 1>(p, stream) : run<__nv_bfloat16, 128, 1>(p, stream);
  // pairs of heads when the visible tokens, if the sequences are as long as
  // they may be, give every CTA two steps of pairs (lengths are the device's)
  const int64_t seen = p.window > 0 ? std::min<int64_t>(p.Lmax, (int64_t)p.window + p.sinks) : p.Lmax;
  const int64_t steps = (seen + kStep - 1) / kStep * p.B * (p.Hkv / 2);
  if (p.Hkv % 2 == 0 && steps >= kPairSteps * (int64_t)p.n_cta)
    return p.dtype == 1 ? run<__half, 64, 2>(p, stream) : run<__nv_bfloat16, 64, 2>(p, stream);
  return p.dtype == 1 ? run<__half, 64, 1>(p, stream) : run<__nv_bfloat16, 64, 1>(p, stream);
}

}  // namespace dash
