// Attention for a batch of sequences that share one long prefix (h3b_attention_prefix), on
// tcgen05.  Every query of sequence b attends to the prefix's keys and values and to the first
// kv_len[b] of its own sequence's; with `causal`, query i sees own keys up to
// i + kv_len[b] - q_len[b].
//
// Mathematics: one pass over the keys with a running maximum m and sum l (base 2, the scale
// folded in): P = 2^(S - m), O += P V, l += sum P; where m grows by more than 8, O and l are
// multiplied by 2^(m_old - m_new) (P stays below 2^8, far inside fp16 and bf16).  A row's state
// (m, l, O) from two ranges of keys joins into one: m = max, each side weighted by 2^(m_side -
// m).  m, l and O are fp32 throughout; P is rounded to the operands' 16 bits for the tensor
// core (its rounding errors average out over the keys), the output once at the store.  A row
// that sees no key has l = 0 and gets 0.
//
// Wide form.  A unit is (sequence, head, 256-query block): two 128-query tiles that share every
// K and V tile, the steps of a unit the prefix's 128-key tiles, then its own.  The units'
// work, laid end to end, is cut into one equal range per CTA (one CTA per SM), whatever the
// lengths are: they are read on the device, so a captured graph follows them.  A unit cut
// between CTAs is finished by the one holding its last step, which joins the states that the
// others left in the workspace; each CTA walks its range from its end, so what it leaves for
// another is computed first.
// Roles (384 threads): warp 0 loads by TMA, warps 1 and 2 issue the tensor core's products of
// tile 0 and 1, warpgroups 1 and 2 are their softmax (a thread owns a query row).
// TMEM: S0 [0, 128), S1 [128, 256), O0 [256, 384), O1 [384, 512).  Shared memory: Q0, Q1, P0,
// P1 and a ring of three K / V tiles in the order of use (K of step t + 1 before V of step t).
// Measured on B200, bf16, 24 heads of 128: six clips of 1,600 queries and 900 to 1,600 own keys
// over 1,024 shared ones 243 to 256 us in a burst of calls, 0.52 of the cuBLAS rate of 1,663 TFLOP/s,
// and 287 to 296 once the calls go on and the power limit lowers the clocks (0.51 of 1,413, cuBLAS's
// then); 11,344 tokens over 1,024 1,597 us, 1,080 TFLOP/s, where the vendor library's attention over
// joined keys takes 1,175.  A tile's S, softmax and P V are a chain; two of them share the tensor core and the
// exponentials, which are busy 45% and 43% of the time: in between both wait for the chains.
#include "kernels.h"
#include "prefix_sched.h"
#include "ptx.cuh"
#include "tmap.h"

#include <algorithm>
#include <atomic>
#include <cuda_fp16.h>
#include <type_traits>

namespace h3b {

namespace {

constexpr uint32_t kBox = 128 * 128;  // 128 rows of 128 bytes, swizzled
constexpr int kRing = 3;

template <int HD>
struct WideCfg {
  static constexpr int kNBox = HD / 64;
  static constexpr uint32_t kTile = kNBox * kBox;  // 128 rows of Q, K or V
  static constexpr uint32_t kPBytes = 2 * kBox;
  static constexpr size_t kSmem = 1024 + 2 * size_t(kTile) + 2 * size_t(kPBytes) +
                                  size_t(kRing) * kTile + 512;
  static_assert(kSmem <= 232448, "above 227 KB");
};

// Total work, and the unit that holds position pos (0 < pos <= total).  All lanes of a warp.
__device__ inline int total_work(const PrefixArgs& a, int lane) {
  int sum = 0;
  for (int b = lane; b < a.batch; b += 32) sum += a.heads * head_work(a, lens_of(a, b));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

__device__ inline void unit_at(const PrefixArgs& a, int pos, int lane, Unit& u) {
  int base = 0;
  for (int b0 = 0;; b0 += 32) {
    const int b = b0 + lane;
    Lens l{0, 0};
    int w = 0;
    if (b < a.batch) {
      l = lens_of(a, b);
      w = a.heads * head_work(a, l);
    }
    int end = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += v;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, w > 0 && base + end >= pos);
    if (hit) {
      const int src = __ffs(hit) - 1;
      u.b = b0 + src;
      u.len.q = __shfl_sync(0xffffffffu, l.q, src);
      u.len.kv = __shfl_sync(0xffffffffu, l.kv, src);
      const int hw = __shfl_sync(0xffffffffu, w, src) / a.heads;
      base += __shfl_sync(0xffffffffu, end - w, src);
      u.h = (pos - base - 1) / hw;
      base += u.h * hw;
      break;
    }
    base += __shfl_sync(0xffffffffu, end, 31);
    if (b0 + 32 >= a.batch) {  // not reached: pos <= total
      u = Unit{};
      return;
    }
  }
  u.qb = 0;
  u.base = base;
  unit_set(a, u);
  const int last = blocks_of(u.len) - 1;
  while (u.qb < last && u.base + kWorkUnit + u.steps * u.step_work < pos) {
    u.base += kWorkUnit + u.steps * u.step_work;
    ++u.qb;
    unit_set(a, u);
  }
}

// Weight of a state with maximum m in a joint one with maximum top.
__device__ __forceinline__ float weight_of(float m, float top) {
  return m == -INFINITY ? 0.0f : ex2_approx(m - top);
}

struct FirstWalk {
  Walk walk;
  Cut cut;
};

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (std::is_same_v<T, __half>) return pack_f16x2(lo, hi);
  else return pack_bf16x2(lo, hi);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float m;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
  return m;
}

__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (global_timer_ns() - t0 > kWaitLimitNs) return;
  }
}

// wait_bar, without its look at the timer before the first polls: most waits here end within
// a microsecond, and the timer's read alone takes a good part of that.
__device__ __forceinline__ bool wait_soon(uint64_t* bar, uint32_t parity,
                                          volatile uint32_t* abort_flag, uint32_t* err,
                                          uint32_t code) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return wait_bar(bar, parity, abort_flag, err, code);
}

// The same by a whole warp; the answer is the warp's.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity,
                                          volatile uint32_t* abort_flag, uint32_t* err,
                                          uint32_t code) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, wait_bar(bar, parity, abort_flag, err, code));
}

__device__ __forceinline__ bool wait_flag(const unsigned long long* f, unsigned long long seq,
                                          volatile uint32_t* abort_flag, uint32_t* err) {
  if (ld_acquire_u64(f) == seq) return true;
  const uint64_t t0 = global_timer_ns();
  while (ld_acquire_u64(f) != seq) {
    if (*abort_flag || global_timer_ns() - t0 > kWaitLimitNs) {
      *abort_flag = 1u;
      atomicCAS(err, 0u, kErrAttnWait);
      return false;
    }
  }
  return true;
}

// Softmax of a row's 128 scores s, those from lim on hidden, against the running maximum m
// (base 2).  First the maximum: the factor by which O has to be multiplied (1 where m stays).
__device__ __forceinline__ float softmax_max(float (&s)[128], int lim, float sl2, float& m) {
  if (lim < 128) {
#pragma unroll
    for (int q = 0; q < 128; ++q)
      if (q >= lim) s[q] = -INFINITY;
  }
  float m8[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m8[i] = fmaxf(s[i], s[8 + i]);
#pragma unroll
    for (int q = 16; q < 128; q += 16) m8[i] = max3(m8[i], s[q + i], s[q + 8 + i]);
  }
  const float mxs =
      max3(max3(m8[0], m8[1], m8[2]), max3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7])) * sl2;
  float alpha = 1.0f;
  if (mxs > m + 8.0f) {  // the first finite maximum of a row too (m = -inf: alpha = 0)
    alpha = ex2_approx(m - mxs);
    m = mxs;
  }
  return alpha;
}

// Then the weights: s becomes P, packed; l the new running sum.
template <typename T>
__device__ __forceinline__ void softmax_exp(const float (&s)[128], float sl2, float m, float alpha,
                                            float& l, uint32_t (&p)[64]) {
  const float base = m == -INFINITY ? 0.0f : -m;
  const uint64_t sl2x2 = pack_f32x2(sl2, sl2), base2 = pack_f32x2(base, base);
  uint64_t sum[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
  for (int q = 0; q < 128; q += 2) {
    float x0, x1;
    const uint64_t x2 = fma_f32x2(pack_f32x2(s[q], s[q + 1]), sl2x2, base2);
    unpack_f32x2(x2, x0, x1);
    x0 = ex2_approx(x0);
    x1 = ex2_approx(x1);
    sum[(q >> 1) & 3] = add_f32x2(sum[(q >> 1) & 3], pack_f32x2(x0, x1));
    p[q >> 1] = pack2<T>(x0, x1);
  }
  float a, b;
  unpack_f32x2(add_f32x2(add_f32x2(sum[0], sum[1]), add_f32x2(sum[2], sum[3])), a, b);
  l = fmaf(l, alpha, a + b);
}

struct Maps {
  CUtensorMap q, kp, vp, k, v;
};

template <typename T, int HD>
__global__ void __launch_bounds__(384, 1)
    k_prefix_wide(const __grid_constant__ Maps tm, const __grid_constant__ PrefixArgs a) {
  using Cfg = WideCfg<HD>;
  constexpr bool kF16 = std::is_same_v<T, __half>;
  constexpr uint32_t IDESC_S = kF16 ? idesc_fp16(128, 128, false) : idesc_bf16(128, 128, false);
  constexpr uint32_t IDESC_PV = kF16 ? idesc_fp16(128, HD, true) : idesc_bf16(128, HD, true);
  constexpr uint32_t kTmemCols = 512;
  constexpr uint32_t kOCol = 256;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;                      // 2 tiles
  uint8_t* sP = sQ + 2 * Cfg::kTile;       // 2 tiles
  uint8_t* sKV = sP + 2 * Cfg::kPBytes;    // kRing slots
  uint64_t* bars = reinterpret_cast<uint64_t*>(sKV + kRing * Cfg::kTile);
  uint64_t* q_full = bars + 0;
  uint64_t* q_empty = bars + 1;
  uint64_t* kv_full = bars + 2;   // [kRing]
  uint64_t* kv_empty = bars + 5;  // [kRing]
  uint64_t* s_full = bars + 8;    // [2 tiles]
  uint64_t* s_free = bars + 10;   // [2]
  uint64_t* p_full = bars + 12;   // [2]
  uint64_t* p_free = bars + 14;   // [2]
  uint64_t* o_empty = bars + 16;  // [2]
  uint64_t* drain = bars + 18;    // [2 issuers]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 20);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  FirstWalk* first = reinterpret_cast<FirstWalk*>(bars + 24);
  static_assert(24 * 8 + sizeof(FirstWalk) <= 512, "barrier area");

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 2);
    for (int s = 0; s < kRing; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 2);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&s_full[w], 1);
      mbar_init(&s_free[w], 4);
      mbar_init(&p_full[w], 4);
      mbar_init(&p_free[w], 1);
      mbar_init(&o_empty[w], 4);
    }
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    *abort_flag = 0u;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  if (warp == 4) {  // this CTA's range
    const Cut all = cut(total_work(a, lane), gridDim.x);
    Walk w{};
    w.begin = all.begin(blockIdx.x);
    w.end = all.begin(blockIdx.x + 1);
    w.more = w.end > w.begin;
    if (w.more) {
      unit_at(a, w.end, lane, w.u);
      w.settle(a);
    }
    if (lane == 0) *first = FirstWalk{w, all};
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // registers: 128 threads x 104 and 256 x 200 are the launch's 384 x 168
  if (warp < 4) {
    regs_dealloc<104>();
    if (warp == 0 && lane == 0) {
      // ------------------------------------------------------------------ producer
      // Per step t, K(t) then V(t - 1); at a segment's first step (not the walk's first)
      // V(t - 1) goes first.  A segment's Q tiles go before its first K.
      bool ok = true;
      int slot = 0;
      uint32_t ring_phase = 0;
      int armed[kRing] = {-1, -1, -1};
      int q_armed = -1;
      auto load = [&](bool is_v, const Unit& u, int j) -> bool {
        if (!wait_soon(&kv_empty[slot], ring_phase ^ 1u, abort_flag, a.err, kErrAttnWait))
          return false;
        mbar_arrive_expect_tx(&kv_full[slot], Cfg::kTile);
        const bool far = j < a.prefix_tiles;
        const CUtensorMap* m = far ? (is_v ? &tm.vp : &tm.kp) : (is_v ? &tm.v : &tm.k);
        const int tok = (far ? j : j - a.prefix_tiles) * 128;
#pragma unroll
        for (int x = 0; x < Cfg::kNBox; ++x)
          tma_load_4d(sKV + slot * Cfg::kTile + x * kBox, m, &kv_full[slot], 64 * x, tok,
                      u.h / a.group, far ? 0 : u.b);
        armed[slot] = static_cast<int>(ring_phase);
        if (++slot == kRing) {
          slot = 0;
          ring_phase ^= 1u;
        }
        return true;
      };
      Walk w = first->walk;
      Unit pu{};          // the step before's
      int pj = -1, n = 0;
      while (w.more && ok) {
        if (pj >= 0) ok = load(true, pu, pj);
        for (int j = w.j0; j < w.j1 && ok; ++j) {
          if (j == w.j0) {
            if (n > 0 && !wait_soon(q_empty, static_cast<uint32_t>(n - 1) & 1u, abort_flag, a.err,
                                   kErrAttnWait)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(q_full, 2 * Cfg::kTile);
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int x = 0; x < Cfg::kNBox; ++x)
                tma_load_4d(sQ + t * Cfg::kTile + x * kBox, &tm.q, q_full, 64 * x,
                            w.u.qb * kBlockQ + t * 128, w.u.h, w.u.b);
            q_armed = n & 1;
          }
          ok = load(false, w.u, j) && (j == w.j0 || load(true, w.u, j - 1));
        }
        pu = w.u;
        pj = w.j1 - 1;
        ++n;
        w.next(a);
      }
      if (ok && pj >= 0) ok = load(true, pu, pj);
      if (!ok) {
        if (q_armed >= 0) drain_wait(q_full, static_cast<uint32_t>(q_armed));
        for (int s = 0; s < kRing; ++s)
          if (armed[s] >= 0) drain_wait(&kv_full[s], static_cast<uint32_t>(armed[s]));
      }
    } else if ((warp == 1 || warp == 2) && lane == 0) {
      // ------------------------------------------------------------------ MMA issuers
      const int w = warp - 1;
      int slot = 0;
      uint32_t ring_phase = 0;
      int cnt = 0, pvc = 0;  // S and P V products issued for this tile
      int units = 0;         // segments whose last P V was issued (tile present)
      int n = 0;
      const uint64_t q_desc = opaque_u64(sdesc_sw128(smem_u32(sQ + w * Cfg::kTile), 16, 1024));
      const uint64_t p_desc = opaque_u64(sdesc_sw128(smem_u32(sP + w * Cfg::kPBytes), 16, 1024));
      const uint64_t k_desc0 = opaque_u64(sdesc_sw128(smem_u32(sKV), 16, 1024));
      const uint64_t v_desc0 = opaque_u64(sdesc_sw128(smem_u32(sKV), kBox, 1024));
      const uint32_t s_tmem = tmem + w * 128;
      const uint32_t o_tmem = tmem + kOCol + w * 128;
      auto ring_take = [&](int& s_out) -> bool {
        if (!wait_soon(&kv_full[slot], ring_phase, abort_flag, a.err, kErrAttnWait)) return false;
        s_out = slot;
        if (++slot == kRing) {
          slot = 0;
          ring_phase ^= 1u;
        }
        return true;
      };
      auto issue_s = [&](bool here, bool first, bool last) -> bool {
        if (first &&
            !wait_soon(q_full, static_cast<uint32_t>(n) & 1u, abort_flag, a.err, kErrAttnWait))
          return false;
        int ksl;
        if (!ring_take(ksl)) return false;
        if (here) {
          if (cnt >= 1 && !wait_soon(&s_free[w], static_cast<uint32_t>(cnt - 1) & 1u, abort_flag,
                                    a.err, kErrAttnWait))
            return false;
          tc_fence_after();
          const uint64_t k_desc = k_desc0 + static_cast<uint64_t>(ksl) * (Cfg::kTile >> 4);
          if constexpr (HD == 128)
            umma_f16_x8_kk<kBox / 16>(s_tmem, q_desc, k_desc, IDESC_S, 0u);
          else
            umma_f16_x4_kk(s_tmem, q_desc, k_desc, IDESC_S, 0u);
          tc_commit(&s_full[w]);
          ++cnt;
        }
        tc_commit(&kv_empty[ksl]);
        if (last) tc_commit(q_empty);
        return true;
      };
      auto issue_pv = [&](bool here, bool first, bool last) -> bool {
        int vsl;
        if (!ring_take(vsl)) return false;
        if (here) {
          // the tile's previous segment must have read O out before it is overwritten
          if (first && units > 0 &&
              !wait_soon(&o_empty[w], static_cast<uint32_t>(units - 1) & 1u, abort_flag, a.err,
                        kErrAttnWait))
            return false;
          if (!wait_soon(&p_full[w], static_cast<uint32_t>(pvc) & 1u, abort_flag, a.err,
                        kErrAttnWait))
            return false;
          tc_fence_after();
          umma_f16_x8_kmn<kBox / 16>(
              o_tmem, p_desc, v_desc0 + static_cast<uint64_t>(vsl) * (Cfg::kTile >> 4), IDESC_PV,
              first ? 0u : 1u);
          tc_commit(&p_free[w]);
          ++pvc;
          if (last) ++units;
        }
        tc_commit(&kv_empty[vsl]);
        return true;
      };
      Walk wk = first->walk;
      bool ok = true, p_here = false, p_first = false, pending = false;
      while (wk.more && ok) {
        const bool here = w == 0 || wk.u.qb * kBlockQ + 128 < wk.u.len.q;
        if (pending) ok = issue_pv(p_here, p_first, true);
        for (int j = wk.j0; j < wk.j1 && ok; ++j)
          ok = issue_s(here, j == wk.j0, j + 1 == wk.j1) &&
               (j == wk.j0 || issue_pv(here, j - 1 == wk.j0, false));
        pending = true;
        p_here = here;
        p_first = wk.j1 - 1 == wk.j0;
        ++n;
        wk.next(a);
      }
      if (ok && pending) issue_pv(p_here, p_first, true);
      tc_commit(&drain[w]);
      drain_wait(&drain[w], 0);
    }
  } else {
    regs_alloc<200>();
    // ------------------------------------------------------------------ softmax (tile w)
    const int w = (warp - 4) >> 2;
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_addr = tmem + lane_addr + w * 128;
    const uint32_t o_addr = tmem + lane_addr + kOCol + w * 128;
    const float sl2 = a.scale_log2;
    uint4* pbuf = reinterpret_cast<uint4*>(sP + w * Cfg::kPBytes);
    bool ok = true;
    int c = 0;  // steps of this tile so far
    int t = 0;  // steps of this CTA so far (ring position)
    for (Walk wk = first->walk; wk.more && ok; wk.next(a)) {
      const int q0 = wk.u.qb * kBlockQ + w * 128;
      if (w == 1 && q0 >= wk.u.len.q) {
        t += wk.j1 - wk.j0;
        continue;
      }
      // own keys [0, own_end) are seen by this row
      int own_end = wk.u.len.kv;
      if (a.causal) own_end = min(own_end, q0 + row + 1 + wk.u.len.kv - wk.u.len.q);
      float m = -INFINITY, l = 0.f;
      for (int j = wk.j0; j < wk.j1; ++j, ++c, ++t) {
        ok = warp_wait(&s_full[w], static_cast<uint32_t>(c) & 1u, abort_flag,
                                              a.err, kErrAttnWait);
        if (!ok) break;
        tc_fence_after();
        float s[128];
        {
          uint32_t r[128];
          tmem_ld128_sync(s_addr, r);
#pragma unroll
          for (int q = 0; q < 128; ++q) s[q] = __uint_as_float(r[q]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[w]);
        const bool far = j < a.prefix_tiles;
        const int tok = (far ? j : j - a.prefix_tiles) * 128;
        const int lim = (far ? a.n_prefix : own_end) - tok;
        const float alpha = softmax_max(s, lim, sl2, m);
        uint32_t pk[64];
        softmax_exp<T>(s, sl2, m, alpha, l, pk);
        if (c >= 1) {
          // the P tile is free, and O complete, once the tile's previous P V has finished
          ok = warp_wait(&p_free[w], static_cast<uint32_t>(c - 1) & 1u,
                                                abort_flag, a.err, kErrAttnWait);
          if (!ok) break;
        }
#pragma unroll
        for (int c16 = 0; c16 < 16; ++c16)
          pbuf[tile_piece(row, c16)] =
              make_uint4(pk[c16 * 4], pk[c16 * 4 + 1], pk[c16 * 4 + 2], pk[c16 * 4 + 3]);
        if (j > wk.j0 && __any_sync(0xffffffffu, alpha != 1.0f)) {
          tc_fence_after();
#pragma unroll 1
          for (int cc = 0; cc < HD / 32; ++cc) {
            uint32_t r[32];
            tmem_ld32(o_addr + cc * 32, r);
            tmem_wait_ld(r);
#pragma unroll
            for (int q = 0; q < 32; ++q) r[q] = __float_as_uint(__uint_as_float(r[q]) * alpha);
            tmem_st32(o_addr + cc * 32, r);
          }
          tmem_wait_st();
        }
        if (!far && wk.u.len.kv - tok < 128) {
          // the values behind the sequence's end may be anything (0 * NaN is NaN): zeros.  V
          // of step t is the ring's load 2 t + 2, or 2 t + 1 at a segment's last step.
          const int idx = 2 * t + (j + 1 == wk.j1 ? 1 : 2);
          const int vsl = idx % kRing;
          ok = warp_wait(&kv_full[vsl], static_cast<uint32_t>(idx / kRing) & 1u,
                                   abort_flag, a.err, kErrAttnWait);
          if (!ok) break;
          const int from = max(0, wk.u.len.kv - tok);
          uint4* v = reinterpret_cast<uint4*>(sKV + vsl * Cfg::kTile);
          for (int i = row; i < (128 - from) * 8 * Cfg::kNBox; i += 128) {
            const int x = i / ((128 - from) * 8), e = i - x * (128 - from) * 8;
            v[x * (kBox / 16) + from * 8 + e] = make_uint4(0u, 0u, 0u, 0u);
          }
          // all four warps' zeros before any of them releases P: the product reads all rows
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[w]);
      }
      if (!ok) break;
      // ---- end of the segment: O holds every P V product once the last one completes
      ok = warp_wait(&p_free[w], static_cast<uint32_t>(c - 1) & 1u,
                                            abort_flag, a.err, kErrAttnWait);
      if (!ok) break;
      tc_fence_after();
      const int part = static_cast<int>(blockIdx.x) * 2 + w;
      if (wk.j1 < wk.u.steps) {
        // not the unit's end: leave the state for the CTA that has it
        float4* po = a.part_o + size_t(part) * (HD / 4) * 128 + row;
#pragma unroll 1
        for (int cc = 0; cc < HD / 32; ++cc) {
          uint32_t r[32];
          tmem_ld32(o_addr + cc * 32, r);
          tmem_wait_ld(r);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            __stcg(po + size_t(cc * 8 + i) * 128,
                   make_float4(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]),
                               __uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3])));
        }
        __stcg(a.part_ml + size_t(part) * 128 + row, make_float2(m, l));
        __threadfence();
        __syncwarp();
        if (lane == 0) st_release_u64(a.flags + part * 4 + quarter, a.seq);
      } else {
        // the unit's end: join the states that the CTAs lo .. blockIdx.x - 1 left, in order
        const int me = static_cast<int>(blockIdx.x);
        const Cut all = first->cut;
        int lo = me;
        float wb = 1.0f;
        if (wk.j0 > 0) {
          lo = first_cta(wk.u, all, me);
          float top = m;
          for (int from = lo; from < me && ok; ++from) {
            if (!has_piece(wk.u, all, from)) continue;
            ok = __all_sync(0xffffffffu, wait_flag(a.flags + (from * 2 + w) * 4 + quarter, a.seq,
                                                   abort_flag, a.err));
            if (ok) top = fmaxf(top, __ldcg(a.part_ml + size_t(from * 2 + w) * 128 + row).x);
          }
          if (!ok) break;
          wb = weight_of(m, top);
          l *= wb;
          for (int from = lo; from < me; ++from) {
            if (!has_piece(wk.u, all, from)) continue;
            const float2 ml = __ldcg(a.part_ml + size_t(from * 2 + w) * 128 + row);
            l = fmaf(ml.y, weight_of(ml.x, top), l);
          }
          m = top;
        }
        const float inv_l = m == -INFINITY ? 0.0f : 1.0f / l;  // 0: the row sees no key
        constexpr int kVecs = HD / 8;  // 16-byte pieces of a row
#pragma unroll 1
        for (int cc = 0; cc < HD / 32; ++cc) {
          float o[32];
          {
            uint32_t r[32];
            tmem_ld32(o_addr + cc * 32, r);
            tmem_wait_ld(r);
#pragma unroll
            for (int q = 0; q < 32; ++q) o[q] = __uint_as_float(r[q]) * wb;
          }
          for (int from = lo; from < me; ++from) {
            if (!has_piece(wk.u, all, from)) continue;
            const int src = from * 2 + w;
            const float wa = weight_of(__ldcg(a.part_ml + size_t(src) * 128 + row).x, m);
            const float4* po = a.part_o + size_t(src) * (HD / 4) * 128 + row;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 v = __ldcg(po + size_t(cc * 8 + i) * 128);
              o[4 * i + 0] = fmaf(v.x, wa, o[4 * i + 0]);
              o[4 * i + 1] = fmaf(v.y, wa, o[4 * i + 1]);
              o[4 * i + 2] = fmaf(v.z, wa, o[4 * i + 2]);
              o[4 * i + 3] = fmaf(v.w, wa, o[4 * i + 3]);
            }
          }
          // to where this row's P was, 16 bytes at a time.  A warp writes and reads back its own
          // 32 rows of P only: one that is ahead may be storing the next segment's
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint4 u;
            u.x = pack2<T>(o[8 * i + 0] * inv_l, o[8 * i + 1] * inv_l);
            u.y = pack2<T>(o[8 * i + 2] * inv_l, o[8 * i + 3] * inv_l);
            u.z = pack2<T>(o[8 * i + 4] * inv_l, o[8 * i + 5] * inv_l);
            u.w = pack2<T>(o[8 * i + 6] * inv_l, o[8 * i + 7] * inv_l);
            pbuf[tile_piece(row, cc * 4 + i)] = u;
          }
        }
        // and from there whole rows at a time: the warp's own 32, those past q_len left out
        __syncwarp();
        T* dst = static_cast<T*>(a.out.data) + wk.u.b * a.out.batch + wk.u.h * a.out.head;
#pragma unroll 4
        for (int i = 0; i < kVecs; ++i) {
          const int r = quarter * 32 + (i * 32 + lane) / kVecs, v = lane & (kVecs - 1);
          const uint4 u = pbuf[tile_piece(r, v)];
          if (q0 + r < wk.u.len.q)
            *reinterpret_cast<uint4*>(dst + static_cast<long long>(q0 + r) * a.out.token + v * 8) = u;
        }
        // the flags go back at zero, so that a replay of this launch waits for them again
        __syncwarp();
        if (lane == 0)
          for (int from = lo; from < me; ++from)
            if (has_piece(wk.u, all, from)) a.flags[(from * 2 + w) * 4 + quarter] = 0ull;
      }
      // O may now be overwritten by the next segment's first P V
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_empty[w]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ============================================================================ narrow form
// Few queries (decoding, a few drafted tokens): what has to be read is the keys and values,
// each once, and the tensor core's 128 rows are filled with all queries that read the same
// ones.  A unit of the prefix holds the rows of gt query heads of one key head, of every query,
// of bt sequences; a unit of a sequence's own keys the same of that sequence alone.  The units'
// key tiles, laid end to end, are cut into one equal range per CTA, and every part of a unit
// leaves its rows' state (O, m, l) in the workspace; a second kernel joins the states of each
// row, of the prefix and of its own, in a fixed order.
// Within a CTA the steps alternate between two chains, each with its own scores, weights and
// output accumulator: S, softmax and P V of one step take longer than the step's bytes take to
// arrive, two such chains do not.  The weights go to tensor memory over the scores they come
// from (S of the chain's next step is issued behind P V, and the tensor core works in order),
// which leaves the shared memory to the ring of K and V tiles and to two Q tiles.  A slot of the
// ring has a full barrier for each chain: the tiles of one slot go to either chain, and a chain
// that is ahead must not take the barrier's earlier phase, the other chain's, for its own.
// Roles (384 threads): warp 0 loads; warps 1 and 2 issue chain 0 and 1; warpgroups 1 and 2 are
// their softmax (warps without rows only keep the barriers' count).
// TMEM: S0 / P0 [0, 128), S1 / P1 [128, 256), O0 [256, 384), O1 [384, 512).
// Measured on B200, bf16, one query, 24 / 8 heads of 128: 48 sequences of 1 to 2,011 own keys over
// 16,133 shared ones 70 us in a graph, 0.57 of the copy rate (75 to 81 in repeated calls; a step of
// the prefix is bound by its softmax);
// with 2,048 own keys each and next to no prefix 0.93 to 0.95.  Two sequences of 4 heads of 64 over
// 257 keys take 11 us: launch, schedule, cold instructions and the join.  A unit of a single step
// costs its CTA some 2.6 us, which bounds many short own caches (2,048 sequences of about 115 own
// keys over 4,096 shared ones: 530 us, 0.29).

template <int HD>
struct NarrowCfg {
  static constexpr int kNBox = HD / 64;
  static constexpr uint32_t kTile = kNBox * kBox;
  static constexpr int kSlots = HD == 128 ? 5 : 11;  // K or V tiles in flight
  static constexpr size_t kSmem = 1024 + (2 + kSlots) * size_t(kTile) + 1024;
  static_assert(kSmem <= 232448, "above 227 KB");
};

struct NarrowMaps {
  CUtensorMap q_far, q_own, kp, vp, k, v;
};

// Inclusive sum over the lanes.
__device__ __forceinline__ int lane_scan(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// Work of a sequence's own units; 0 behind the batch.
__device__ __forceinline__ int narrow_own_work(const PrefixArgs& a, int b) {
  return b < a.batch ? a.own_units * narrow_work(narrow_steps(lens_of(a, b))) : 0;
}

// The CTA's first segment.  All lanes of a warp.
__device__ inline NarrowWalk narrow_first(const PrefixArgs& a, int lane, int cta) {
  const int far = narrow_prefix_work(a);
  // a lane has sequence lane, lane + 32, ...
  int total = far;
  Lens l{0, 0};
  int one = 0, end = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    l = Lens{0, 0};
    if (b0 + lane < a.batch) l = lens_of(a, b0 + lane);
    one = narrow_work(narrow_steps(l));
    end = lane_scan(one * a.own_units, lane);
    total += __shfl_sync(0xffffffffu, end, 31);
  }
  const int ctas = narrow_ctas(total, a.ctas);
  NarrowWalk w{};
  if (total == 0 || cta >= ctas) return w;
  const Cut all = cut(total, ctas);
  w.begin = all.begin(cta);
  w.end = all.begin(cta + 1);
  w.more = w.end > w.begin;
  if (w.begin < far) {
    w.u.index = w.begin / narrow_far_work(a);
    w.u.base = w.u.index * narrow_far_work(a);
    w.u.b = -1;
    w.u.steps = a.prefix_tiles;
  } else {
    int base = far;
    for (int b0 = 0; b0 < a.batch; b0 += 32) {
      if (a.batch > 32) {  // else the lanes still hold them
        l = Lens{0, 0};
        if (b0 + lane < a.batch) l = lens_of(a, b0 + lane);
        one = narrow_work(narrow_steps(l));
        end = lane_scan(one * a.own_units, lane);
      }
      const unsigned hit = __ballot_sync(0xffffffffu, one > 0 && base + end > w.begin);
      if (hit) {
        const int src = __ffs(hit) - 1;
        w.u.b = b0 + src;
        w.u.len.q = __shfl_sync(0xffffffffu, l.q, src);
        w.u.len.kv = __shfl_sync(0xffffffffu, l.kv, src);
        w.u.steps = narrow_steps(w.u.len);
        const int each = narrow_work(w.u.steps);
        base += __shfl_sync(0xffffffffu, end, src) - each * a.own_units;
        w.u.in_b = (w.begin - base) / each;
        w.u.base = base + w.u.in_b * each;
        w.u.index = a.prefix_units + w.u.b * a.own_units + w.u.in_b;
        break;
      }
      base += __shfl_sync(0xffffffffu, end, 31);
    }
  }
  w.settle(a);
  return w;
}

// Key head and first query head of a unit, and the first of its sequences.
struct NarrowHeads {
  int kvh, h0, b0, rows;
};
__device__ __forceinline__ NarrowHeads narrow_heads(const PrefixArgs& a, const NarrowUnit& u) {
  NarrowHeads r;
  int hh;
  if (u.b < 0) {
    hh = u.index / a.chunks;
    const int bc = u.index - hh * a.chunks;
    r.b0 = bc * a.bt;
    r.rows = min(a.bt, a.batch - r.b0) * a.gt * a.n_q;
  } else {
    hh = u.in_b;
    r.b0 = u.b;
    r.rows = a.gt * a.n_q;
  }
  r.kvh = hh / a.head_groups;
  r.h0 = r.kvh * a.group + (hh - r.kvh * a.head_groups) * a.gt;
  return r;
}

template <typename T, int HD>
__global__ void __launch_bounds__(384, 1)
    k_prefix_narrow(const __grid_constant__ NarrowMaps tm, const __grid_constant__ PrefixArgs a) {
  using Cfg = NarrowCfg<HD>;
  constexpr bool kF16 = std::is_same_v<T, __half>;
  constexpr int kSlots = Cfg::kSlots;
  constexpr uint32_t IDESC_S = kF16 ? idesc_fp16(128, 128, false) : idesc_bf16(128, 128, false);
  constexpr uint32_t IDESC_PV = kF16 ? idesc_fp16(128, HD, true) : idesc_bf16(128, HD, true);
  constexpr uint32_t kTmemCols = 512;
  constexpr uint32_t kOCol = 256;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;                  // 2 tiles
  uint8_t* sKV = sQ + 2 * Cfg::kTile;  // kSlots tiles
  uint64_t* bars = reinterpret_cast<uint64_t*>(sKV + kSlots * Cfg::kTile);
  uint64_t* q_full = bars + 0;    // [2 tiles]
  uint64_t* q_empty = bars + 2;   // [2]
  uint64_t* s_full = bars + 4;    // [2 chains]
  uint64_t* p_full = bars + 6;    // [2]
  uint64_t* o_full = bars + 8;    // [2]
  uint64_t* drain = bars + 10;    // [2]
  uint64_t* kv_full = bars + 12;  // [2 chains][kSlots]
  uint64_t* kv_empty = kv_full + 2 * kSlots;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(kv_empty + kSlots);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  NarrowWalk* start = reinterpret_cast<NarrowWalk*>(bars + 48);
  static_assert(12 + 3 * kSlots + 1 <= 48 && 48 * 8 + sizeof(NarrowWalk) <= 1024, "barrier area");

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 2);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_full[i], 1);
      mbar_init(&drain[i], 1);
    }
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_full[kSlots + s], 1);
      mbar_init(&kv_empty[s], 1);
    }
    *abort_flag = 0u;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  if (warp == 4) {
    const NarrowWalk w = narrow_first(a, lane, static_cast<int>(blockIdx.x));
    if (lane == 0) *start = w;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < 4) {
    regs_dealloc<104>();
    if (warp == 0 && lane == 0) {
      // ------------------------------------------------------------------ producer
      bool ok = true;
      int slot = 0, n = 0;
      uint32_t ring_phase = 0;
      // for the way out: the slots' fills so far, as (chain, parity), and per chain and slot the
      // parity of the next fill
      int armed[kSlots];
#pragma unroll
      for (int s = 0; s < kSlots; ++s) armed[s] = -1;
      uint32_t fills[2] = {0, 0};
      unsigned t = 0;  // steps so far; step t is chain t & 1's
      int q_armed[2] = {-1, -1};
      auto load = [&](const CUtensorMap* m, int tok, int kvh, int b) -> bool {
        if (!wait_soon(&kv_empty[slot], ring_phase ^ 1u, abort_flag, a.err, kErrAttnWait))
          return false;
        uint64_t* full = &kv_full[(t & 1u) * kSlots + slot];
        mbar_arrive_expect_tx(full, Cfg::kTile);
#pragma unroll
        for (int x = 0; x < Cfg::kNBox; ++x)
          tma_load_4d(sKV + slot * Cfg::kTile + x * kBox, m, full, 64 * x, tok, kvh, b);
        uint32_t& f = (t & 1u) ? fills[1] : fills[0];
#pragma unroll
        for (int s = 0; s < kSlots; ++s)
          if (s == slot) armed[s] = static_cast<int>((t & 1u) * 2 + ((f >> s) & 1u));
        f ^= 1u << slot;
        if (++slot == kSlots) {
          slot = 0;
          ring_phase ^= 1u;
        }
        return true;
      };
      for (NarrowWalk w = *start; w.more && ok; w.next(a), ++n) {
        const bool far = w.u.b < 0;
        const NarrowHeads hd = narrow_heads(a, w.u);
        const int qb = n & 1;
        if (n >= 2 && !wait_soon(&q_empty[qb], static_cast<uint32_t>((n >> 1) - 1) & 1u, abort_flag,
                                a.err, kErrAttnWait)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(&q_full[qb],
                              static_cast<uint32_t>((far ? a.bt : 1) * a.gt * a.n_q) * 128u * Cfg::kNBox);
#pragma unroll
        for (int x = 0; x < Cfg::kNBox; ++x)
          tma_load_4d(sQ + qb * Cfg::kTile + x * kBox, far ? &tm.q_far : &tm.q_own, &q_full[qb],
                      64 * x, 0, hd.h0, hd.b0);
        q_armed[qb] = (n >> 1) & 1;
        for (int j = w.j0; j < w.j1 && ok; ++j, ++t)
          ok = load(far ? &tm.kp : &tm.k, j * 128, hd.kvh, far ? 0 : w.u.b) &&
               load(far ? &tm.vp : &tm.v, j * 128, hd.kvh, far ? 0 : w.u.b);
      }
      if (!ok) {
        for (int i = 0; i < 2; ++i)
          if (q_armed[i] >= 0) drain_wait(&q_full[i], static_cast<uint32_t>(q_armed[i]));
#pragma unroll
        for (int s = 0; s < kSlots; ++s)
          if (armed[s] >= 0)
            drain_wait(&kv_full[(armed[s] >> 1) * kSlots + s], static_cast<uint32_t>(armed[s] & 1));
      }
    } else if ((warp == 1 || warp == 2) && lane == 0) {
      // ------------------------------------------------------------------ MMA issuers
      const int c = warp - 1;
      const uint64_t q_desc0 = opaque_u64(sdesc_sw128(smem_u32(sQ), 16, 1024));
      const uint64_t k_desc0 = opaque_u64(sdesc_sw128(smem_u32(sKV), 16, 1024));
      const uint64_t v_desc0 = opaque_u64(sdesc_sw128(smem_u32(sKV), kBox, 1024));
      const uint32_t s_tmem = tmem + c * 128;
      const uint32_t o_tmem = tmem + kOCol + c * 128;
      bool ok = true;
      unsigned t = 0;        // steps of this CTA so far; step t is chain t & 1's
      uint32_t mine = 0;     // this chain's
      uint32_t phases = 0;   // parity of this chain's next fill of each slot
      int n = 0;
      for (NarrowWalk w = *start; w.more && ok; w.next(a), ++n) {
        const int qb = n & 1;
        const int count = w.j1 - w.j0;
        const unsigned t_end = t + count;
        bool first = true;
        if (!wait_soon(&q_full[qb], static_cast<uint32_t>(n >> 1) & 1u, abort_flag, a.err,
                      kErrAttnWait))
          break;
        for (unsigned x = t + ((t ^ c) & 1u); x < t_end; x += 2, ++mine) {
          const unsigned ik = 2 * x, iv = 2 * x + 1;
          const int ks = ik % kSlots, vs = iv % kSlots;
          if (!wait_soon(&kv_full[c * kSlots + ks], (phases >> ks) & 1u, abort_flag, a.err,
                        kErrAttnWait)) {
            ok = false;
            break;
          }
          phases ^= 1u << ks;
          tc_fence_after();
          const uint64_t q_desc = q_desc0 + static_cast<uint64_t>(qb) * (Cfg::kTile >> 4);
          const uint64_t k_desc = k_desc0 + static_cast<uint64_t>(ks) * (Cfg::kTile >> 4);
          if constexpr (HD == 128)
            umma_f16_x8_kk<kBox / 16>(s_tmem, q_desc, k_desc, IDESC_S, 0u);
          else
            umma_f16_x4_kk(s_tmem, q_desc, k_desc, IDESC_S, 0u);
          tc_commit(&s_full[c]);
          tc_commit(&kv_empty[ks]);
          if (x + 2 >= t_end) tc_commit(&q_empty[qb]);
          if (!wait_soon(&p_full[c], mine & 1u, abort_flag, a.err, kErrAttnWait) ||
              !wait_soon(&kv_full[c * kSlots + vs], (phases >> vs) & 1u, abort_flag, a.err,
                        kErrAttnWait)) {
            ok = false;
            break;
          }
          phases ^= 1u << vs;
          tc_fence_after();
          const uint64_t v_desc = v_desc0 + static_cast<uint64_t>(vs) * (Cfg::kTile >> 4);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_f16_ts(o_tmem, s_tmem + kk * 8, v_desc + kk * 128, IDESC_PV,
                        (first && kk == 0) ? 0u : 1u);
          first = false;
          tc_commit(&kv_empty[vs]);
          if (x + 2 >= t_end) tc_commit(&o_full[c]);
        }
        if (ok && first) mbar_arrive(&q_empty[qb]);  // a segment of one step, the other chain's
        t = t_end;
      }
      tc_commit(&drain[c]);
      drain_wait(&drain[c], 0);
    }
  } else {
    regs_alloc<200>();
    // ------------------------------------------------------------------ softmax (chain c)
    const int c = (warp - 4) >> 2;
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_addr = tmem + lane_addr + c * 128;
    const uint32_t o_addr = tmem + lane_addr + kOCol + c * 128;
    const float sl2 = a.scale_log2;
    bool ok = true;
    unsigned t = 0;
    uint32_t mine = 0, ends = 0, phases = 0;
    for (NarrowWalk w = *start; w.more && ok; w.next(a)) {
      const bool far = w.u.b < 0;
      const NarrowHeads hd = narrow_heads(a, w.u);
      const bool warp_on = quarter * 32 < hd.rows;
      int own_end = w.u.len.kv;
      if (!far && a.causal) own_end = min(own_end, row % a.n_q + 1 + w.u.len.kv - w.u.len.q);
      const unsigned t_end = t + (w.j1 - w.j0);
      float m = -INFINITY, l = 0.f;
      bool first = true;
      for (unsigned x = t + ((t ^ c) & 1u); x < t_end; x += 2, ++mine) {
        const int tok = (w.j0 + static_cast<int>(x - t)) * 128;
        ok = warp_wait(&s_full[c], mine & 1u, abort_flag, a.err, kErrAttnWait);
        if (!ok) break;
        if (warp_on) {
          tc_fence_after();
          float s[128];
          {
            uint32_t r[128];
            tmem_ld128_sync(s_addr, r);
#pragma unroll
            for (int q = 0; q < 128; ++q) s[q] = __uint_as_float(r[q]);
          }
          const float alpha = softmax_max(s, (far ? a.n_prefix : own_end) - tok, sl2, m);
          uint32_t pk[64];
          softmax_exp<T>(s, sl2, m, alpha, l, pk);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t r[32];
#pragma unroll
            for (int q = 0; q < 32; ++q) r[q] = pk[half * 32 + q];
            tmem_st32(s_addr + half * 32, r);
          }
          // O holds the chain's earlier products: S of this step was issued behind them
          if (!first && __any_sync(0xffffffffu, alpha != 1.0f)) {
#pragma unroll 1
            for (int cc = 0; cc < HD / 32; ++cc) {
              uint32_t r[32];
              tmem_ld32(o_addr + cc * 32, r);
              tmem_wait_ld(r);
#pragma unroll
              for (int q = 0; q < 32; ++q) r[q] = __float_as_uint(__uint_as_float(r[q]) * alpha);
              tmem_st32(o_addr + cc * 32, r);
            }
          }
          tmem_wait_st();
        }
        first = false;
        const unsigned iv = 2 * x + 1;
        phases ^= 1u << ((2 * x) % kSlots);
        if (!far && w.u.len.kv - tok < 128) {
          // the values behind the sequence's end may be anything (0 * NaN is NaN): zeros
          const int vs = iv % kSlots;
          ok = warp_wait(&kv_full[c * kSlots + vs], (phases >> vs) & 1u,
                                                abort_flag, a.err, kErrAttnWait);
          if (!ok) break;
          const int from = max(0, w.u.len.kv - tok);
          uint4* v = reinterpret_cast<uint4*>(sKV + vs * Cfg::kTile);
          for (int i = row; i < (128 - from) * 8 * Cfg::kNBox; i += 128) {
            const int b = i / ((128 - from) * 8), e = i - b * (128 - from) * 8;
            v[b * (kBox / 16) + from * 8 + e] = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        phases ^= 1u << (iv % kSlots);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[c]);
      }
      if (!ok) break;
      // ---- end of the segment: this chain's state of every row
      const size_t at = narrow_row(a, far, w.u.index, static_cast<int>(blockIdx.x), c) + row;
      if (!first) {
        ok = warp_wait(&o_full[c], ends & 1u, abort_flag, a.err, kErrAttnWait);
        if (!ok) break;
        ++ends;
        if (warp_on) {
          tc_fence_after();
#pragma unroll 1
          for (int cc = 0; cc < HD / 32; ++cc) {
            uint32_t r[32];
            tmem_ld32(o_addr + cc * 32, r);
            tmem_wait_ld(r);
            if (row < hd.rows) {
              float4* d = reinterpret_cast<float4*>(a.part_rows + at * HD + cc * 32);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                d[i] = make_float4(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]),
                                   __uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3]));
            }
          }
          tc_fence_before();
        }
      }
      if (row < hd.rows) a.part_sums[at] = make_float2(m, l);
      t = t_end;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the states of a row of the output: WARPS warps per (sequence, query, head), each with
// its share of the channels, lanes over those and over the states.  Launched while k_prefix_narrow runs: the
// first rows' schedule is worked out before the wait for it, only the states' two loads come
// after.  A block takes 4 / WARPS rows at a time of a range of rows, which is that many where
// rows are few; where they are many it is longer, so that the whole batch's lengths are not
// summed for every row.
template <typename T, int HD, int WARPS>
__global__ void __launch_bounds__(128) k_prefix_join(const __grid_constant__ PrefixArgs a, int per) {
  constexpr int kRows = 4 / WARPS;              // rows of a block at a time
  constexpr int kLanes = HD / (4 * WARPS);      // lanes that have a state's channels, 4 each
  constexpr int kStates = 32 / kLanes;          // states at a time
  __shared__ int s_sum[2][4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int in_block = warp / WARPS, sub = warp % WARPS;
  const int far = narrow_prefix_work(a);
  const int per_b = a.n_q * a.heads, rows = a.batch * per_b;
  const int times = (rows + kRows - 1) / kRows;
  const int time0 = blockIdx.x * per, time1 = min(times, time0 + per);
  const int mine = lane / kLanes;                                    // states mine, mine + kStates ..
  const int chan = (sub * kLanes + lane % kLanes) * 4;
  // the work in front of the block's first sequence, and all of it
  int at_b = time0 * kRows / per_b, at_base, total;
  {
    int before = 0, sum = 0;
#pragma unroll 4
    for (int b = threadIdx.x; b < a.batch; b += 128) {
      const int own = narrow_own_work(a, b);
      sum += own;
      if (b < at_b) before += own;
    }
    before = __reduce_add_sync(0xffffffffu, before);
    sum = __reduce_add_sync(0xffffffffu, sum);
    if (lane == 0) {
      s_sum[0][warp] = before;
      s_sum[1][warp] = sum;
    }
    __syncthreads();
    at_base = far + s_sum[0][0] + s_sum[0][1] + s_sum[0][2] + s_sum[0][3];
    total = far + s_sum[1][0] + s_sum[1][1] + s_sum[1][2] + s_sum[1][3];
  }
  for (int time = time0; time < time1; ++time) {
    const int row = time * kRows + in_block;
    const int b = row / per_b, in_b = row - b * per_b;
    const int tok = in_b / a.heads, h = in_b - tok * a.heads;
    while (at_b < b) at_base += narrow_own_work(a, at_b++);
    Lens len{0, 0};
    if (b < a.batch) len = lens_of(a, b);
    const bool on = b < a.batch && tok < len.q;
    Side side[2];
    side[0].n = side[1].n = 0;
    if (on && total > 0) {
      const Cut all = cut(total, narrow_ctas(total, a.ctas));
      const int kvh = h / a.group, hg = (h - kvh * a.group) / a.gt;
      const int g = h - kvh * a.group - hg * a.gt, hh = kvh * a.head_groups + hg;
      if (a.prefix_units > 0) {
        const int chunk = b / a.bt, index = hh * a.chunks + chunk;
        side[0] = narrow_side(a, all, true, index, index * narrow_far_work(a), a.prefix_tiles,
                              ((b - chunk * a.bt) * a.gt + g) * a.n_q + tok);
      }
      const int steps = narrow_steps(len);
      if (steps > 0)
        side[1] = narrow_side(a, all, false, a.prefix_units + b * a.own_units + hh,
                              at_base + hh * narrow_work(steps), steps, g * a.n_q + tok);
    }
    if (time == time0) asm volatile("griddepcontrol.wait;" ::: "memory");
    // (max, sum) of the first 32 states of each side, a lane each; more are read again
    auto state = [&](const Side& s, int i) -> float2 {
      if (i >= s.n) return make_float2(-INFINITY, 0.f);
      return __ldcg(a.part_sums + s.row + (i >> 1) * s.step + (i & 1) * s.chain);
    };
    float2 ml[2];
#pragma unroll
    for (int d = 0; d < 2; ++d) ml[d] = state(side[d], lane);
    float top = fmaxf(ml[0].x, ml[1].x);
#pragma unroll
    for (int d = 0; d < 2; ++d)
      for (int i = lane + 32; i < side[d].n; i += 32) top = fmaxf(top, state(side[d], i).x);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
    float l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      for (int i0 = 0; i0 < side[d].n; i0 += 32) {
        const float2 one = i0 == 0 ? ml[d] : state(side[d], i0 + lane);
        const float wt = weight_of(one.x, top);
        l = fmaf(one.y, wt, l);
        const int n = min(32, side[d].n - i0);
#pragma unroll 4
        for (int i1 = 0; i1 < n; i1 += kStates) {
          const int i = i1 + mine;
          const float w = __shfl_sync(0xffffffffu, wt, i & 31);
          // 0: a chain without steps, or a state that no longer counts
          if (i >= n || w == 0.f) continue;
          const float4 v = __ldcg(reinterpret_cast<const float4*>(
              a.part_rows +
              (side[d].row + ((i0 + i) >> 1) * side[d].step + (i & 1) * side[d].chain) * HD + chan));
          o[0] = fmaf(v.x, w, o[0]);
          o[1] = fmaf(v.y, w, o[1]);
          o[2] = fmaf(v.z, w, o[2]);
          o[3] = fmaf(v.w, w, o[3]);
        }
      }
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
#pragma unroll
    for (int s = 16; s >= kLanes; s >>= 1)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] += __shfl_xor_sync(0xffffffffu, o[e], s);
    if (!on || mine != 0) continue;
    const float inv_l = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
    T* dst = static_cast<T*>(a.out.data) + b * a.out.batch + tok * a.out.token + h * a.out.head + chan;
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<T>(o[0] * inv_l, o[1] * inv_l),
                                                pack2<T>(o[2] * inv_l, o[3] * inv_l));
  }
}

// A [batch, tokens, heads, HD] view as a TMA map whose box is 64 channels of box_tokens tokens
// of box_heads heads of box_batch sequences.
bool view_map(CUtensorMap* map, const HeadView& v, bool fp16, int batch, int tokens, int heads,
              int hd, int box_tokens = 128, int box_heads = 1, int box_batch = 1) {
  const cuuint64_t dims[4] = {cuuint64_t(hd), cuuint64_t(tokens), cuuint64_t(heads),
                              cuuint64_t(batch)};
  // (a dimension of size 1 has stride 0 here, which is any valid stride's worth)
  auto bytes = [&](long long st) { return cuuint64_t(st > 0 ? st * 2 : hd * 2); };
  const cuuint64_t strides[3] = {bytes(v.token), bytes(v.head), bytes(v.batch)};
  const cuuint32_t box[4] = {64, cuuint32_t(box_tokens), cuuint32_t(box_heads),
                             cuuint32_t(box_batch)};
  return make_tmap_16bit(map, v.data, fp16, 4, dims, strides, box);
}

// The maps of the prefix's and of the sequences' keys and values.
template <typename M>
bool key_maps(M& tm, const PrefixArgs& a, bool f16, int hd) {
  bool ok = true;
  if (a.n_prefix > 0)
    ok = ok && view_map(&tm.kp, a.kp, f16, 1, a.n_prefix, a.kv_heads, hd) &&
         view_map(&tm.vp, a.vp, f16, 1, a.n_prefix, a.kv_heads, hd);
  if (a.n_kv > 0)
    ok = ok && view_map(&tm.k, a.k, f16, a.batch, a.n_kv, a.kv_heads, hd) &&
         view_map(&tm.v, a.v, f16, a.batch, a.n_kv, a.kv_heads, hd);
  // without own keys (or without a prefix) that pair of maps is never used
  if (a.n_prefix == 0) { tm.kp = tm.k; tm.vp = tm.v; }
  if (a.n_kv == 0) { tm.k = tm.kp; tm.v = tm.vp; }
  return ok;
}

// Dynamic shared memory above 48 KB has to be asked for, once per device.
template <typename K>
int allow_smem(const DevCtx& ctx, K kernel, size_t bytes, std::atomic<uint64_t>& done) {
  const uint64_t bit = 1ull << (ctx.device & 63);
  if (done.load() & bit) return 0;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(bytes));
  if (e != cudaSuccess)
    return set_error(-3, "attention_prefix: cudaFuncSetAttribute: %s", cudaGetErrorString(e));
  done.fetch_or(bit);
  return 0;
}

template <typename T, int HD>
int launch_wide(const DevCtx& ctx, PrefixArgs a, cudaStream_t stream) {
  using Cfg = WideCfg<HD>;
  constexpr bool f16 = std::is_same_v<T, __half>;
  Maps tm;
  if (!view_map(&tm.q, a.q, f16, a.batch, a.n_q, a.heads, HD) || !key_maps(tm, a, f16, HD))
    return set_error(-3, "attention_prefix: cuTensorMapEncodeTiled failed");
  auto kernel = k_prefix_wide<T, HD>;
  static std::atomic<uint64_t> done{0};
  if (int rc = allow_smem(ctx, kernel, Cfg::kSmem, done)) return rc;
  const int grid = wide_ctas(a, std::min(ctx.num_sms, kMaxSkCtas));
  a.seq = next_scratch_seq();
  kernel<<<grid, 384, Cfg::kSmem, stream>>>(tm, a);
  return check_launch("attention_prefix");
}

// Blocks of the join an SM gets at most; a block sums the batch's lengths once, for all its rows.
// 2,048 sequences of 24 heads: 600 us when it came, with a block for every four rows 819.
constexpr long long kJoinBlocks = 16;

template <typename T, int HD>
int launch_narrow(const DevCtx& ctx, const PrefixArgs& a, cudaStream_t stream) {
  using Cfg = NarrowCfg<HD>;
  constexpr bool f16 = std::is_same_v<T, __half>;
  NarrowMaps tm;
  if (!view_map(&tm.q_own, a.q, f16, a.batch, a.n_q, a.heads, HD, a.n_q, a.gt, 1) ||
      !view_map(&tm.q_far, a.q, f16, a.batch, a.n_q, a.heads, HD, a.n_q, a.gt, a.bt) ||
      !key_maps(tm, a, f16, HD))
    return set_error(-3, "attention_prefix: cuTensorMapEncodeTiled failed");
  auto kernel = k_prefix_narrow<T, HD>;
  static std::atomic<uint64_t> done{0};
  if (int rc = allow_smem(ctx, kernel, Cfg::kSmem, done)) return rc;
  kernel<<<a.ctas, 384, Cfg::kSmem, stream>>>(tm, a);
  if (int rc = check_launch("attention_prefix")) return rc;
  // launched while the first kernel runs; it waits for it before it reads.  A unit of the prefix
  // is spread over about ctas / prefix_units CTAs, two states each: from eight states on four
  // warps share a row.
  const long long rows = 1ll * a.batch * a.n_q * a.heads;
  const bool many = a.prefix_units > 0 && 2 * a.ctas >= 8 * a.prefix_units;
  cudaLaunchConfig_t cfg = {};
  const long long times = many ? rows : (rows + 3) / 4;
  const int per = static_cast<int>((times + kJoinBlocks * a.ctas - 1) / (kJoinBlocks * a.ctas));
  cfg.gridDim = dim3(static_cast<unsigned>((times + per - 1) / per));
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (many) cudaLaunchKernelEx(&cfg, k_prefix_join<T, HD, 4>, a, per);
  else cudaLaunchKernelEx(&cfg, k_prefix_join<T, HD, 1>, a, per);
  return check_launch("attention_prefix join");
}

template <typename T, int HD>
int launch_form(const DevCtx& ctx, const PrefixArgs& a, bool narrow, cudaStream_t stream) {
  return narrow ? launch_narrow<T, HD>(ctx, a, stream) : launch_wide<T, HD>(ctx, a, stream);
}

}  // namespace

size_t prefix_workspace_bytes(PrefixArgs a, int head_dim) {
  a.group = a.heads / a.kv_heads;
  if (a.batch == 0 || a.n_q == 0) return 16;
  if (use_narrow(a)) {
    narrow_units(a);
    return narrow_rows(a) * (head_dim * 4 + 8);
  }
  if (wide_work_cap(a) * 2 > kMaxWork) return 0;
  return size_t(kMaxSkCtas) * 2 * 128 * (head_dim * 4 + 8) + size_t(kMaxSkCtas) * 2 * 4 * 8;
}

int launch_attention_prefix(const DevCtx& ctx, bool fp16, int head_dim, PrefixArgs a, void* ws,
                            cudaStream_t stream) {
  a.err = ctx.err_flag;
  a.prefix_tiles = (a.n_prefix + 127) / 128;
  a.group = a.heads / a.kv_heads;
  a.ctas = std::min(ctx.num_sms, kMaxSkCtas);
  const bool narrow = use_narrow(a);
  uint8_t* p = static_cast<uint8_t*>(ws);
  if (narrow) {
    narrow_units(a);
    const size_t rows = narrow_rows(a);
    a.part_rows = reinterpret_cast<float*>(p);
    a.part_sums = reinterpret_cast<float2*>(p + rows * head_dim * 4);
  } else {
    a.part_o = reinterpret_cast<float4*>(p);
    p += size_t(kMaxSkCtas) * 2 * 128 * head_dim * 4;
    a.part_ml = reinterpret_cast<float2*>(p);
    p += size_t(kMaxSkCtas) * 2 * 128 * 8;
    a.flags = reinterpret_cast<unsigned long long*>(p);
  }
  if (head_dim == 128)
    return fp16 ? launch_form<__half, 128>(ctx, a, narrow, stream)
                : launch_form<bf16, 128>(ctx, a, narrow, stream);
  return fp16 ? launch_form<__half, 64>(ctx, a, narrow, stream)
              : launch_form<bf16, 64>(ctx, a, narrow, stream);
}

}  // namespace h3b
