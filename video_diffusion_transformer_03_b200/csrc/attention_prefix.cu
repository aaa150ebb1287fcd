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
constexpr int kMaxPieces = 8;  // CTAs that share a unit, on average, at most

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
__device__ inline long long total_work(const PrefixArgs& a, int lane) {
  long long sum = 0;
  for (int b = lane; b < a.batch; b += 32) sum += a.heads * head_work(a, lens_of(a, b));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

__device__ inline void unit_at(const PrefixArgs& a, long long pos, int lane, Unit& u) {
  long long base = 0;
  for (int b0 = 0;; b0 += 32) {
    const int b = b0 + lane;
    Lens l{0, 0};
    long long w = 0;
    if (b < a.batch) {
      l = lens_of(a, b);
      w = a.heads * head_work(a, l);
    }
    long long end = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += v;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, w > 0 && base + end >= pos);
    if (hit) {
      const int src = __ffs(hit) - 1;
      u.b = b0 + src;
      u.len.q = __shfl_sync(0xffffffffu, l.q, src);
      u.len.kv = __shfl_sync(0xffffffffu, l.kv, src);
      const long long hw = __shfl_sync(0xffffffffu, w, src) / a.heads;
      base += __shfl_sync(0xffffffffu, end - w, src);
      u.h = static_cast<int>((pos - base - 1) / hw);
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
  while (u.qb < last && u.base + kWorkUnit + static_cast<long long>(u.steps) * u.step_work < pos) {
    u.base += kWorkUnit + static_cast<long long>(u.steps) * u.step_work;
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
  long long total;
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

// Softmax of a row's 128 scores s against the running maximum m (base 2): P to the row of
// the P tile at pbuf is left to the caller; s becomes P, l the new running sum.  Returns the
// factor by which O has to be multiplied (1 where the maximum stays).
__device__ __forceinline__ float softmax_row(float (&s)[128], int lim, float sl2, float& m,
                                             float& l) {
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
  const float base = m == -INFINITY ? 0.0f : -m;
  const uint64_t sl2x2 = pack_f32x2(sl2, sl2), base2 = pack_f32x2(base, base);
  uint64_t sum[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
  for (int q = 0; q < 128; q += 2) {
    float x0, x1;
    unpack_f32x2(fma_f32x2(pack_f32x2(s[q], s[q + 1]), sl2x2, base2), x0, x1);
    s[q] = ex2_approx(x0);
    s[q + 1] = ex2_approx(x1);
    sum[(q >> 1) & 3] = add_f32x2(sum[(q >> 1) & 3], pack_f32x2(s[q], s[q + 1]));
  }
  float a, b;
  unpack_f32x2(add_f32x2(add_f32x2(sum[0], sum[1]), add_f32x2(sum[2], sum[3])), a, b);
  l = fmaf(l, alpha, a + b);
  return alpha;
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
    const long long total = total_work(a, lane);
    Walk w{};
    w.begin = range_begin(total, blockIdx.x, gridDim.x);
    w.end = range_begin(total, blockIdx.x + 1, gridDim.x);
    w.more = w.end > w.begin;
    if (w.more) {
      unit_at(a, w.end, lane, w.u);
      w.settle(a);
    }
    if (lane == 0) *first = FirstWalk{w, total};
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
        if (!wait_bar(&kv_empty[slot], ring_phase ^ 1u, abort_flag, a.err, kErrAttnWait))
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
            if (n > 0 && !wait_bar(q_empty, static_cast<uint32_t>(n - 1) & 1u, abort_flag, a.err,
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
        if (!wait_bar(&kv_full[slot], ring_phase, abort_flag, a.err, kErrAttnWait)) return false;
        s_out = slot;
        if (++slot == kRing) {
          slot = 0;
          ring_phase ^= 1u;
        }
        return true;
      };
      auto issue_s = [&](bool here, bool first, bool last) -> bool {
        if (first &&
            !wait_bar(q_full, static_cast<uint32_t>(n) & 1u, abort_flag, a.err, kErrAttnWait))
          return false;
        int ksl;
        if (!ring_take(ksl)) return false;
        if (here) {
          if (cnt >= 1 && !wait_bar(&s_free[w], static_cast<uint32_t>(cnt - 1) & 1u, abort_flag,
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
              !wait_bar(&o_empty[w], static_cast<uint32_t>(units - 1) & 1u, abort_flag, a.err,
                        kErrAttnWait))
            return false;
          if (!wait_bar(&p_full[w], static_cast<uint32_t>(pvc) & 1u, abort_flag, a.err,
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
    uint8_t* pbuf = sP + w * Cfg::kPBytes + row * 128;
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
        ok = __all_sync(0xffffffffu, wait_bar(&s_full[w], static_cast<uint32_t>(c) & 1u, abort_flag,
                                              a.err, kErrAttnWait));
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
        const float alpha = softmax_row(s, lim, sl2, m, l);
        if (c >= 1) {
          // the P tile is free, and O complete, once the tile's previous P V has finished
          ok = __all_sync(0xffffffffu, wait_bar(&p_free[w], static_cast<uint32_t>(c - 1) & 1u,
                                                abort_flag, a.err, kErrAttnWait));
          if (!ok) break;
        }
#pragma unroll
        for (int c16 = 0; c16 < 16; ++c16) {
          uint4 u;
          u.x = pack2<T>(s[c16 * 8 + 0], s[c16 * 8 + 1]);
          u.y = pack2<T>(s[c16 * 8 + 2], s[c16 * 8 + 3]);
          u.z = pack2<T>(s[c16 * 8 + 4], s[c16 * 8 + 5]);
          u.w = pack2<T>(s[c16 * 8 + 6], s[c16 * 8 + 7]);
          const int chunk = (c16 & 7) ^ (row & 7);
          *reinterpret_cast<uint4*>(pbuf + (c16 >> 3) * kBox + chunk * 16) = u;
        }
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
          ok = __all_sync(0xffffffffu,
                          wait_bar(&kv_full[vsl], static_cast<uint32_t>(idx / kRing) & 1u,
                                   abort_flag, a.err, kErrAttnWait));
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
      ok = __all_sync(0xffffffffu, wait_bar(&p_free[w], static_cast<uint32_t>(c - 1) & 1u,
                                            abort_flag, a.err, kErrAttnWait));
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
        int lo = me;
        float wb = 1.0f;
        if (wk.j0 > 0) {
          while (lo > 0 && range_begin(first->total, lo, gridDim.x) > wk.u.base) --lo;
          float top = m;
          for (int from = lo; from < me && ok; ++from) {
            if (!has_piece(wk.u, first->total, from, gridDim.x)) continue;
            ok = __all_sync(0xffffffffu, wait_flag(a.flags + (from * 2 + w) * 4 + quarter, a.seq,
                                                   abort_flag, a.err));
            if (ok) top = fmaxf(top, __ldcg(a.part_ml + size_t(from * 2 + w) * 128 + row).x);
          }
          if (!ok) break;
          wb = weight_of(m, top);
          l *= wb;
          for (int from = lo; from < me; ++from) {
            if (!has_piece(wk.u, first->total, from, gridDim.x)) continue;
            const float2 ml = __ldcg(a.part_ml + size_t(from * 2 + w) * 128 + row);
            l = fmaf(ml.y, weight_of(ml.x, top), l);
          }
          m = top;
        }
        const float inv_l = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);  // NaN stays NaN
        const int token = q0 + row;
        T* dst = static_cast<T*>(a.out.data) + wk.u.b * a.out.batch +
                 static_cast<long long>(token) * a.out.token + wk.u.h * a.out.head;
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
            if (!has_piece(wk.u, first->total, from, gridDim.x)) continue;
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
          if (token < wk.u.len.q) {
            uint4* d = reinterpret_cast<uint4*>(dst + cc * 32);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint4 u;
              u.x = pack2<T>(o[8 * i + 0] * inv_l, o[8 * i + 1] * inv_l);
              u.y = pack2<T>(o[8 * i + 2] * inv_l, o[8 * i + 3] * inv_l);
              u.z = pack2<T>(o[8 * i + 4] * inv_l, o[8 * i + 5] * inv_l);
              u.w = pack2<T>(o[8 * i + 6] * inv_l, o[8 * i + 7] * inv_l);
              d[i] = u;
            }
          }
        }
        // the flags go back at zero, so that a replay of this launch waits for them again
        __syncwarp();
        if (lane == 0)
          for (int from = lo; from < me; ++from)
            if (has_piece(wk.u, first->total, from, gridDim.x)) a.flags[(from * 2 + w) * 4 + quarter] = 0ull;
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

// A [batch, tokens, heads, HD] view as a TMA map whose box is 128 tokens by 64 channels.
bool view_map(CUtensorMap* map, const HeadView& v, bool fp16, int batch, int tokens, int heads,
              int hd) {
  const cuuint64_t dims[4] = {cuuint64_t(hd), cuuint64_t(tokens), cuuint64_t(heads),
                              cuuint64_t(batch)};
  // (a dimension of size 1 has stride 0 here, which is any valid stride's worth)
  auto bytes = [&](long long st) { return cuuint64_t(st > 0 ? st * 2 : hd * 2); };
  const cuuint64_t strides[3] = {bytes(v.token), bytes(v.head), bytes(v.batch)};
  const cuuint32_t box[4] = {64, 128, 1, 1};
  return make_tmap_16bit(map, v.data, fp16, 4, dims, strides, box);
}

template <typename T, int HD>
int launch_wide(const DevCtx& ctx, PrefixArgs a, cudaStream_t stream) {
  using Cfg = WideCfg<HD>;
  constexpr bool f16 = std::is_same_v<T, __half>;
  Maps tm;
  bool ok = view_map(&tm.q, a.q, f16, a.batch, a.n_q, a.heads, HD);
  if (a.n_prefix > 0)
    ok = ok && view_map(&tm.kp, a.kp, f16, 1, a.n_prefix, a.kv_heads, HD) &&
         view_map(&tm.vp, a.vp, f16, 1, a.n_prefix, a.kv_heads, HD);
  if (a.n_kv > 0)
    ok = ok && view_map(&tm.k, a.k, f16, a.batch, a.n_kv, a.kv_heads, HD) &&
         view_map(&tm.v, a.v, f16, a.batch, a.n_kv, a.kv_heads, HD);
  if (!ok) return set_error(-3, "attention_prefix: cuTensorMapEncodeTiled failed");
  // without own keys (or without a prefix) that pair of maps is never used
  if (a.n_prefix == 0) { tm.kp = tm.k; tm.vp = tm.v; }
  if (a.n_kv == 0) { tm.k = tm.kp; tm.v = tm.vp; }
  auto kernel = k_prefix_wide<T, HD>;
  static std::atomic<uint64_t> attr_done{0};
  const uint64_t bit = 1ull << (ctx.device & 63);
  if (!(attr_done.load() & bit)) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(Cfg::kSmem));
    if (e != cudaSuccess)
      return set_error(-3, "attention_prefix: cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    attr_done.fetch_or(bit);
  }
  const long long units = 1ll * a.batch * a.heads * ((a.n_q + kBlockQ - 1) / kBlockQ);
  const int grid = static_cast<int>(
      std::min<long long>(units * kMaxPieces, std::min(ctx.num_sms, kMaxSkCtas)));
  a.seq = next_scratch_seq();
  kernel<<<grid, 384, Cfg::kSmem, stream>>>(tm, a);
  return check_launch("attention_prefix");
}

}  // namespace

size_t prefix_workspace_bytes(int head_dim) {
  return size_t(kMaxSkCtas) * 2 * 128 * (head_dim * 4 + 8) + size_t(kMaxSkCtas) * 2 * 4 * 8;
}

int launch_attention_prefix(const DevCtx& ctx, bool fp16, int head_dim, PrefixArgs a, void* ws,
                            cudaStream_t stream) {
  uint8_t* p = static_cast<uint8_t*>(ws);
  a.part_o = reinterpret_cast<float4*>(p);
  p += size_t(kMaxSkCtas) * 2 * 128 * head_dim * 4;
  a.part_ml = reinterpret_cast<float2*>(p);
  p += size_t(kMaxSkCtas) * 2 * 128 * 8;
  a.flags = reinterpret_cast<unsigned long long*>(p);
  a.err = ctx.err_flag;
  a.prefix_tiles = (a.n_prefix + 127) / 128;
  a.group = a.heads / a.kv_heads;
  if (head_dim == 128)
    return fp16 ? launch_wide<__half, 128>(ctx, a, stream) : launch_wide<bf16, 128>(ctx, a, stream);
  return fp16 ? launch_wide<__half, 64>(ctx, a, stream) : launch_wide<bf16, 64>(ctx, a, stream);
}

}  // namespace h3b
