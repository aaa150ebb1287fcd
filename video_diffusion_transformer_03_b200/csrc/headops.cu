// Row operators on the heads of q and k: rotary positions with several axes at explicit
// positions (h3b_rope_axes), and the per-head RMS norm with that rotation in the same pass,
// forward and backward (h3b_qk_norm_rope, h3b_qk_norm_rope_backward).
//
// Mathematics.  Pair p of a head turns by the angle pos[axis(p)] * freq(p).  The angle is
// taken in revolutions: r = pos * (freq / 2 pi) in 64 bits, r minus its nearest integer is
// exact, and sin / cos of 2 pi times that remainder come from sincospif in 32 bits, so a
// position of 10^5 costs no accuracy (in 32 bits its angle alone would be off by 4e-3).
//   forward   y = R (n * g),  n = x * rstd,  rstd = 1 / sqrt(mean(x^2) + eps)
//   backward  z = R^T gy;  dg = sum over tokens and heads of z * n;  w = z * g;
//             dx = rstd * (w - n * mean(w * n))
// Everything between the load and the store is in 32 bits; one rounding, at the store.
//
// What bounds it: HBM.  Forward reads and writes every head once, backward reads x and gy
// and writes dx.  So a warp takes a token and walks over its heads of q or of k (a block has
// one or the other, which keeps one set of gains and sums in registers): each lane owns 16 or 8
// channels of a head (the pairs C/2 s .. C/2 s + C/2 - 1 of its slot s, in both pairings), so the
// angles of a token are computed once for all heads of the warp's item, pairs never cross
// lanes, and the only shuffles are those of the norm's sums and the angles'.  A group of heads is
// loaded while the one before it is worked on, from one item into the next.
//
// Measured on B200 (CUDA graphs, inputs past the L2 or rotated), heads of 128, against the copy
// rate of 6,555 GB/s:
//   rotation, fp16, 2 x 11,344 tokens of 24 heads               48 us  0.89
//   norm + rotation, bf16, 3 x 11,341 tokens of 24 + 8 heads   107 us  0.79
//   its backward, fp16, 2 x 11,343 tokens of 24 + 8 heads      106 us  0.80
//   in 32 bits, norm + rotation of 11,341 tokens of 24 + 8      67 us  0.85, its backward 95, 0.90
//   at 1,600 tokens, bf16: rotation of 24 heads 7.0 us, norm + rotation of 24 + 24 13.5, backward
//   18.7 (0.43 to 0.48)
// (The first three in calls from Python: 50, 110 and 109 to 113 us.)  Large calls wait for HBM: the
// largest stall is the loads' (0.55 to 0.63 instructions issued a cycle), and registers limit how
// many are in flight.  At 1,600 tokens a warp has three or so items, and launch, ladder and first
// loads are 4 us of the time.
#include "kernels.h"
#include "ptx.cuh"

#include <algorithm>
#include <cuda_fp16.h>
#include <type_traits>

namespace h3b {

namespace {

constexpr int kWarps = 4;  // warps of a block

enum Mode : int { kModeRope = 0, kModeNorm = 1, kModeNormBwd = 2 };

// A lane's C channels (C / 2 pairs): chunk c0 .. c0 + C/2 - 1 and chunk c1 .. c1 + C/2 - 1.
// Adjacent pairing: c1 = c0 + C/2 and pair i is channels (2 i, 2 i + 1) of the two laid end to
// end.  Half-split pairing: c1 = c0 + rot / 2 and pair i is (c0 + i, c1 + i); behind the rotated
// width c1 = c0 + C/2.  C = 16 (16-bit types, widths that are multiples of 16) makes both chunks
// 16-byte accesses and halves the shuffles, roots and addresses per byte; C = 8 is for the rest.
template <typename T, int C>
struct Raw {
  uint32_t w[C * sizeof(T) / 4];
};

template <typename T, int C, bool HALVES>
__device__ __forceinline__ void load_raw(const T* p, int c0, int c1, Raw<T, C>& r) {
  if constexpr (C * sizeof(T) == 32) {  // two chunks of 16 bytes
    const uint4 a = *reinterpret_cast<const uint4*>(p + c0);
    const uint4 b = *reinterpret_cast<const uint4*>(p + c1);
    r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
    r.w[4] = b.x; r.w[5] = b.y; r.w[6] = b.z; r.w[7] = b.w;
  } else if constexpr (HALVES) {
    const uint2 a = *reinterpret_cast<const uint2*>(p + c0);
    const uint2 b = *reinterpret_cast<const uint2*>(p + c1);
    r.w[0] = a.x; r.w[1] = a.y; r.w[2] = b.x; r.w[3] = b.y;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(p + c0);
    r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
  }
}

template <typename T, int C, bool HALVES>
__device__ __forceinline__ void store_raw(T* p, int c0, int c1, const Raw<T, C>& r) {
  if constexpr (C * sizeof(T) == 32) {
    *reinterpret_cast<uint4*>(p + c0) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    *reinterpret_cast<uint4*>(p + c1) = make_uint4(r.w[4], r.w[5], r.w[6], r.w[7]);
  } else if constexpr (HALVES) {
    *reinterpret_cast<uint2*>(p + c0) = make_uint2(r.w[0], r.w[1]);
    *reinterpret_cast<uint2*>(p + c1) = make_uint2(r.w[2], r.w[3]);
  } else {
    *reinterpret_cast<uint4*>(p + c0) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
  }
}

// The pairs of a lane, members a and b apart, as packed fp32: a[0] holds pairs 0 and 1.
// Packed arithmetic does two of them in one issue slot, which is what these kernels run out of
// first once enough loads are in flight.
template <int C>
struct Pairs {
  uint64_t a[C / 4], b[C / 4];
};

template <typename T>
__device__ __forceinline__ float2 two(uint32_t u) {
  if constexpr (std::is_same_v<T, __half>) return __half22float2(*reinterpret_cast<const __half2*>(&u));
  else return unpack_bf16x2(u);
}

template <typename T>
__device__ __forceinline__ uint32_t two(float x, float y) {
  if constexpr (std::is_same_v<T, __half>) return pack_f16x2(x, y);
  else return pack_bf16x2(x, y);
}

template <typename T, int C, bool HALVES>
__device__ __forceinline__ Pairs<C> widen(const Raw<T, C>& r) {
  Pairs<C> p;
#pragma unroll
  for (int i = 0; i < C / 4; ++i) {
    if constexpr (std::is_same_v<T, float>) {
      const float f0 = __uint_as_float(r.w[HALVES ? 2 * i : 4 * i]);
      const float f1 = __uint_as_float(r.w[HALVES ? 2 * i + 1 : 4 * i + 1]);
      const float f2 = __uint_as_float(r.w[HALVES ? C / 2 + 2 * i : 4 * i + 2]);
      const float f3 = __uint_as_float(r.w[HALVES ? C / 2 + 1 + 2 * i : 4 * i + 3]);
      p.a[i] = HALVES ? pack_f32x2(f0, f1) : pack_f32x2(f0, f2);
      p.b[i] = HALVES ? pack_f32x2(f2, f3) : pack_f32x2(f1, f3);
    } else {
      const float2 u = two<T>(r.w[HALVES ? i : 2 * i]);
      const float2 v = two<T>(r.w[HALVES ? C / 4 + i : 2 * i + 1]);
      p.a[i] = HALVES ? pack_f32x2(u.x, u.y) : pack_f32x2(u.x, v.x);
      p.b[i] = HALVES ? pack_f32x2(v.x, v.y) : pack_f32x2(u.y, v.y);
    }
  }
  return p;
}

template <typename T, int C, bool HALVES>
__device__ __forceinline__ Raw<T, C> narrow(const Pairs<C>& p) {
  Raw<T, C> r;
#pragma unroll
  for (int i = 0; i < C / 4; ++i) {
    float a0, a1, b0, b1;
    unpack_f32x2(p.a[i], a0, a1);
    unpack_f32x2(p.b[i], b0, b1);
    if constexpr (std::is_same_v<T, float>) {
      r.w[HALVES ? 2 * i : 4 * i] = __float_as_uint(a0);
      r.w[HALVES ? 2 * i + 1 : 4 * i + 2] = __float_as_uint(a1);
      r.w[HALVES ? C / 2 + 2 * i : 4 * i + 1] = __float_as_uint(b0);
      r.w[HALVES ? C / 2 + 1 + 2 * i : 4 * i + 3] = __float_as_uint(b1);
    } else {
      r.w[HALVES ? i : 2 * i] = HALVES ? two<T>(a0, a1) : two<T>(a0, b0);
      r.w[HALVES ? C / 4 + i : 2 * i + 1] = HALVES ? two<T>(b0, b1) : two<T>(a1, b1);
    }
  }
  return r;
}

template <int C>
__device__ __forceinline__ Pairs<C> mul(const Pairs<C>& p, uint64_t f) {
  Pairs<C> r;
#pragma unroll
  for (int i = 0; i < C / 4; ++i) {
    r.a[i] = mul_f32x2(p.a[i], f);
    r.b[i] = mul_f32x2(p.b[i], f);
  }
  return r;
}
// sum of the products of the channels
template <int C>
__device__ __forceinline__ float dot(const Pairs<C>& p, const Pairs<C>& q) {
  uint64_t x = mul_f32x2(p.a[0], q.a[0]), y = mul_f32x2(p.b[0], q.b[0]);
#pragma unroll
  for (int i = 1; i < C / 4; ++i) {
    x = fma_f32x2(p.a[i], q.a[i], x);
    y = fma_f32x2(p.b[i], q.b[i], y);
  }
  float lo, hi;
  unpack_f32x2(add_f32x2(x, y), lo, hi);
  return lo + hi;
}

// sin and cos of 2 pi t.  Adding 1.5 * 2^52 rounds t to the nearest integer.
__device__ __forceinline__ void sincos_turns(double t, float& s, float& c) {
  const double magic = 6755399441055744.0;
  const double n = (t + magic) - magic;
  sincospif(2.0f * static_cast<float>(t - n), &s, &c);
}

// A turn, with a factor on each member before it (the gains): a -> a ac - b bs, b -> a as + b bc.
template <int C>
struct Turn {
  uint64_t ac[C / 4], nbs[C / 4], as[C / 4], bc[C / 4];  // nbs = -bs
};

// Kept in shared memory, 16 bytes of every lane side by side: in registers the turn would cost
// a quarter of the warps (norm + rotation of 3 x 11,341 tokens: 106 us, in registers 134).
template <int C>
__device__ __forceinline__ void put(uint4* at, int part, const uint64_t (&v)[C / 4]) {
#pragma unroll
  for (int i = 0; i < C / 8; ++i)
    *reinterpret_cast<ulonglong2*>(at + (part * (C / 8) + i) * kWarps * 32) =
        make_ulonglong2(v[2 * i], v[2 * i + 1]);
}
template <int C>
__device__ __forceinline__ void get(const uint4* at, int part, uint64_t (&v)[C / 4]) {
#pragma unroll
  for (int i = 0; i < C / 8; ++i) {
    const ulonglong2 u =
        *reinterpret_cast<const ulonglong2*>(at + (part * (C / 8) + i) * kWarps * 32);
    v[2 * i] = u.x;
    v[2 * i + 1] = u.y;
  }
}
template <int C>
__device__ __forceinline__ Turn<C> load_turn(const uint4* at) {
  Turn<C> t;
  get<C>(at, 0, t.ac);
  get<C>(at, 1, t.nbs);
  get<C>(at, 2, t.as);
  get<C>(at, 3, t.bc);
  return t;
}

// Of two packed pairs the first n from x, the others from y.
__device__ __forceinline__ uint64_t first_pairs(uint64_t x, uint64_t y, int n) {
  float x0, x1, y0, y1;
  unpack_f32x2(x, x0, x1);
  unpack_f32x2(y, y0, y1);
  return pack_f32x2(n > 0 ? x0 : y0, n > 1 ? x1 : y1);
}

// The lane's pairs, of which the first n turn (WHOLE: all of every lane's).  The others only take
// their factors: a sine of 0 times an infinity or a NaN would carry a channel that passes through
// into the one beside it.  Whole heads have kernels of their own, which the choice costs nothing;
// heads turned in part take 1% longer for it (norm + rotation of 3 x 11,341 tokens, 64 of 128
// channels: 109.5 us, 109.0 without).
template <int C, bool WHOLE>
__device__ __forceinline__ Pairs<C> rotate(const Pairs<C>& p, const Turn<C>& t, int n) {
  Pairs<C> r;
#pragma unroll
  for (int i = 0; i < C / 4; ++i) {
    const uint64_t b = mul_f32x2(p.b[i], t.bc[i]);
    r.a[i] = fma_f32x2(p.a[i], t.ac[i], mul_f32x2(p.b[i], t.nbs[i]));
    r.b[i] = fma_f32x2(p.a[i], t.as[i], b);
    if constexpr (!WHOLE) {
      r.a[i] = first_pairs(r.a[i], mul_f32x2(p.a[i], t.ac[i]), n - 2 * i);
      r.b[i] = first_pairs(r.b[i], b, n - 2 * i);
    }
  }
  return r;
}

// Sum over the LPH lanes of a head.
template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = LPH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Channel of pair i's members behind the first of a lane's contiguous ones.
template <int C, bool HALVES>
__device__ __forceinline__ constexpr int member_a(int i) {
  return HALVES ? i : 2 * i;
}
template <int C, bool HALVES>
__device__ __forceinline__ constexpr int member_b(int i) {
  return HALVES ? C / 2 + i : 2 * i + 1;
}

// A group is kPass passes of 32 / LPH heads.  An item is one token, or (parts > 1, where
// tokens are few) an equal share of its groups.
template <typename T, int C, int MODE>
constexpr int pass_count() {
  return (MODE == kModeNormBwd || C * sizeof(T) == 32) ? 1 : 2;
}

// What an item costs beside its groups of heads (its angles), in groups; 1, 2 and 3 measured
// within 3% of one another.
constexpr int kItemCost = 1;

// Blocks that are on an SM at a time; the grid is that many a SM at most.  As many as registers
// allow without spills: loads in flight are what hides HBM here.
constexpr int blocks_per_sm(int mode, int C) {
  if (mode == kModeRope) return 8;
  if (mode == kModeNorm) return C == 16 ? 5 : 6;
  return C == 16 ? 4 : 5;
}
// (the caller's workspace has a row for each of the backward pass's blocks)
static_assert(blocks_per_sm(kModeNormBwd, 8) <= kHeadRowsBwdPerSm &&
                  blocks_per_sm(kModeNormBwd, 16) <= kHeadRowsBwdPerSm,
              "backward workspace");

template <typename T, int C, bool HALVES, int LPH, int MODE, bool WHOLE>
__global__ void __launch_bounds__(kWarps * 32, blocks_per_sm(MODE, C)) k_head_rows(const __grid_constant__ HeadRows a) {
  constexpr int kPass = pass_count<T, C, MODE>();
  constexpr int kHeads = 32 / LPH;
  constexpr int kGroup = kPass * kHeads;
  constexpr bool kBwd = MODE == kModeNormBwd;
  // (the backward pass's second kernel may be launched; it waits for this one's end)
  if constexpr (kBwd) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int slot = lane % LPH, sub = lane / LPH;
  constexpr int kPairs = C / 2;
  const bool live = slot * C < a.head_dim;
  const bool turned = slot * kPairs < a.n_pairs;
  const bool half_slot = HALVES && turned;
  // pairs of this lane that turn, or more (half-split: all of them or none)
  const int n_turned = HALVES ? (turned ? kPairs : 0) : a.n_pairs - slot * kPairs;
  const int c0 = half_slot ? slot * kPairs : slot * C;
  const int c1 = half_slot ? a.n_pairs + slot * kPairs : slot * C + kPairs;

  const int w = static_cast<int>(blockIdx.x) >= a.q_blocks;
  const unsigned block = w ? blockIdx.x - a.q_blocks : blockIdx.x;
  const unsigned blocks = w ? gridDim.x - a.q_blocks : static_cast<unsigned>(a.q_blocks);
  const HeadView in = a.in[w], out = a.out[w];
  const int heads = a.heads[w], parts = a.parts[w];
  const int groups = (heads + kGroup - 1) / kGroup;
  const unsigned n_items = static_cast<unsigned>(a.rows) * parts;

  // this lane computes kOwn of its slot's angles; lanes of the other heads the others
  constexpr int kOwn = kPairs / kHeads > 0 ? kPairs / kHeads : 1;
  double turns[kOwn];
  uint64_t axes = 0;  // a byte a pair
  Pairs<C> acc;
  bool have_lane = false;
  const float inv_hd = 1.0f / static_cast<float>(a.head_dim);
#pragma unroll
  for (int i = 0; i < kOwn; ++i) turns[i] = 0.0;
#pragma unroll
  for (int i = 0; i < C / 4; ++i) acc.a[i] = acc.b[i] = 0ull;

  __shared__ uint4 s_turn[(MODE == kModeRope ? 4 : 6) * (C / 8) * kWarps * 32];
  uint4* my_turn = s_turn + threadIdx.x;
  // The ladder is a kernel argument, which lanes read one by one: once a block, not once a warp.
  __shared__ double s_turns[128];
  __shared__ __align__(8) uint8_t s_axis[128];
  const long long in_step = kHeads * in.head, out_step = kHeads * out.head;
  long long grd_step = 0;
  if constexpr (kBwd) grd_step = kHeads * a.grad[w].head;

  // the item at hand: its token, its groups and the heads from this lane's first on
  unsigned item = block * kWarps + (threadIdx.x >> 5), b = 0, t = 0;
  int n_groups = 0, left = 0;
  // this lane's channels of the next head to be loaded
  const T* src = nullptr;
  const T* grd = nullptr;
  Raw<T, C> x[kPass], gy[kPass];
  auto load = [&](int n) {
#pragma unroll
    for (int i = 0; i < kPass; ++i) {
      const bool on = live && i * kHeads < n;
      x[i] = Raw<T, C>{};
      if (on) load_raw<T, C, HALVES>(src, c0, c1, x[i]);
      src += in_step;
      if constexpr (kBwd) {
        gy[i] = Raw<T, C>{};
        if (on) load_raw<T, C, HALVES>(grd, c0, c1, gy[i]);
        grd += grd_step;
      }
    }
  };
  auto open = [&]() {
    unsigned row = item;
    int g0 = 0, g1 = groups;
    if (parts > 1) {
      row = item / parts;
      const int part = static_cast<int>(item - row * parts);
      const int each = (groups + parts - 1) / parts;  // (the last item may have fewer)
      g0 = part * each;
      g1 = min(groups, g0 + each);
    }
    t = row;
    if (a.rows != a.tokens) {
      b = row / static_cast<unsigned>(a.tokens);
      t = row - b * static_cast<unsigned>(a.tokens);
    }
    n_groups = g1 - g0;
    const int first = g0 * kGroup + sub;
    left = heads - first;
    src = static_cast<const T*>(in.data) + b * in.batch + t * in.token + first * in.head;
    if constexpr (kBwd)
      grd = static_cast<const T*>(a.grad[w].data) + b * a.grad[w].batch + t * a.grad[w].token +
            first * a.grad[w].head;
    load(left);
  };
  bool more = item < n_items;
  if (more) open();
  if (a.n_pairs > 0) {
    const int i = threadIdx.x;  // kWarps * 32 = 128 of them
    s_turns[i] = i < a.n_pairs ? a.turns[i] : 0.0;
    s_axis[i] = i < a.n_pairs ? a.axis[i] : uint8_t(0);
    __syncthreads();
  }
  while (more) {
    T* dst = static_cast<T*>(out.data) + b * out.batch + t * out.token + (heads - left) * out.head;
    if (!have_lane) {
      // this lane's constants, behind its first loads
      have_lane = true;
      if (turned) {
#pragma unroll
        for (int i = 0; i < kOwn; ++i) turns[i] = s_turns[slot * kPairs + (sub * kOwn + i) % kPairs];
        if constexpr (C == 16) axes = *reinterpret_cast<const uint64_t*>(s_axis + slot * kPairs);
        else axes = *reinterpret_cast<const uint32_t*>(s_axis + slot * kPairs);
      }
      if constexpr (MODE != kModeRope) {
        const float* g = w ? a.k_gain : a.q_gain;
        Pairs<C> gain;
        float ga[kPairs], gb[kPairs];
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          const bool on = g != nullptr && live;
          ga[i] = on ? __ldg(g + (HALVES && turned ? c0 + i : slot * C + member_a<C, HALVES>(i))) : 1.f;
          gb[i] = on ? __ldg(g + (HALVES && turned ? c1 + i : slot * C + member_b<C, HALVES>(i))) : 1.f;
        }
#pragma unroll
        for (int i = 0; i < C / 4; ++i) {
          gain.a[i] = pack_f32x2(ga[2 * i], ga[2 * i + 1]);
          gain.b[i] = pack_f32x2(gb[2 * i], gb[2 * i + 1]);
        }
        put<C>(my_turn, 4, gain.a);
        put<C>(my_turn, 5, gain.b);
      }
    }
    {
      Turn<C> turn;
      Pairs<C> gain;
      if constexpr (MODE == kModeNorm) {
        get<C>(my_turn, 4, gain.a);
        get<C>(my_turn, 5, gain.b);
      }
      float cs[kPairs], sn[kPairs];
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        cs[i] = 1.f;
        sn[i] = 0.f;
      }
      if (a.n_pairs > 0) {
        const float* pos = a.pos + b * a.pos_batch + static_cast<size_t>(t) * a.n_axes;
        float oc[kOwn], os[kOwn];
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
          // (a pair past the rotated width has turns 0: it stays)
          const int p = (sub * kOwn + i) % kPairs;
          sincos_turns(static_cast<double>(__ldg(pos + static_cast<int>((axes >> (8 * p)) & 0xffu))) * turns[i], os[i],
                       oc[i]);
          if (kBwd || (MODE == kModeRope && a.inverse)) os[i] = -os[i];
        }
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          if constexpr (kOwn == kPairs) {
            cs[i] = oc[i];
            sn[i] = os[i];
          } else {
            cs[i] = __shfl_sync(0xffffffffu, oc[i % kOwn], slot + (i / kOwn) * LPH);
            sn[i] = __shfl_sync(0xffffffffu, os[i % kOwn], slot + (i / kOwn) * LPH);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < C / 4; ++i) {
        const uint64_t c = pack_f32x2(cs[2 * i], cs[2 * i + 1]), s = pack_f32x2(sn[2 * i], sn[2 * i + 1]);
        const uint64_t n = pack_f32x2(-sn[2 * i], -sn[2 * i + 1]);
        const bool folded = MODE == kModeNorm;  // y = rstd R(g x): the gains go into the turn
        turn.ac[i] = folded ? mul_f32x2(gain.a[i], c) : c;
        turn.nbs[i] = folded ? mul_f32x2(gain.b[i], n) : n;
        turn.as[i] = folded ? mul_f32x2(gain.a[i], s) : s;
        turn.bc[i] = folded ? mul_f32x2(gain.b[i], c) : c;
      }
      put<C>(my_turn, 0, turn.ac);
      put<C>(my_turn, 1, turn.nbs);
      put<C>(my_turn, 2, turn.as);
      put<C>(my_turn, 3, turn.bc);
    }
    const int groups_here = n_groups;
    int left_here = left;
    for (int g = 0; g < groups_here; ++g) {
      Raw<T, C> xc[kPass], gc[kPass];
#pragma unroll
      for (int i = 0; i < kPass; ++i) {
        xc[i] = x[i];
        if constexpr (kBwd) gc[i] = gy[i];
      }
      // the next group's loads, or the next item's first
      if (g + 1 < groups_here) {
        load(left_here - kGroup);
      } else {
        item += blocks * kWarps;
        more = item < n_items;
        if (more) open();
      }
#pragma unroll
      for (int i = 0; i < kPass; ++i) {
        Pairs<C> f = widen<T, C, HALVES>(xc[i]);
        if constexpr (MODE != kModeRope) {
          const float rstd = rsqrtf(head_sum<LPH>(dot(f, f)) * inv_hd + a.eps);
          const uint64_t r2 = pack_f32x2(rstd, rstd);
          if constexpr (!kBwd) {
            f = mul(f, r2);
          } else {
            Pairs<C> gain;
            get<C>(my_turn, 4, gain.a);
            get<C>(my_turn, 5, gain.b);
            Pairs<C> z = rotate<C, WHOLE>(widen<T, C, HALVES>(gc[i]), load_turn<C>(my_turn), n_turned);
            f = mul(f, r2);
#pragma unroll
            for (int k = 0; k < C / 4; ++k) {
              acc.a[k] = fma_f32x2(z.a[k], f.a[k], acc.a[k]);
              acc.b[k] = fma_f32x2(z.b[k], f.b[k], acc.b[k]);
              z.a[k] = mul_f32x2(z.a[k], gain.a[k]);
              z.b[k] = mul_f32x2(z.b[k], gain.b[k]);
            }
            const float zn = -head_sum<LPH>(dot(z, f)) * inv_hd;
            const uint64_t d2 = pack_f32x2(zn, zn);
#pragma unroll
            for (int k = 0; k < C / 4; ++k) {
              f.a[k] = fma_f32x2(f.a[k], d2, z.a[k]);
              f.b[k] = fma_f32x2(f.b[k], d2, z.b[k]);
            }
            f = mul(f, r2);
          }
        }
        if constexpr (!kBwd) f = rotate<C, WHOLE>(f, load_turn<C>(my_turn), n_turned);
        if (live && i * kHeads < left_here) store_raw<T, C, HALVES>(dst, c0, c1, narrow<T, C, HALVES>(f));
        dst += out_step;
      }
      left_here -= kGroup;
    }
  }
  if constexpr (kBwd) {
    // the block's share of the gain's gradient: lanes of the same slot, then its warps in
    // order, then one row [head_dim] of the workspace
    __shared__ float red[kWarps][LPH * C];
    float va[kPairs], vb[kPairs];
#pragma unroll
    for (int i = 0; i < C / 4; ++i) {
      unpack_f32x2(acc.a[i], va[2 * i], va[2 * i + 1]);
      unpack_f32x2(acc.b[i], vb[2 * i], vb[2 * i + 1]);
    }
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
#pragma unroll
      for (int o = LPH; o < 32; o <<= 1) {
        va[i] += __shfl_xor_sync(0xffffffffu, va[i], o);
        vb[i] += __shfl_xor_sync(0xffffffffu, vb[i], o);
      }
      if (sub == 0 && live) {
        float* r = red[threadIdx.x >> 5];
        r[HALVES && turned ? c0 + i : slot * C + member_a<C, HALVES>(i)] = va[i];
        r[HALVES && turned ? c1 + i : slot * C + member_b<C, HALVES>(i)] = vb[i];
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < a.head_dim; c += kWarps * 32) {
      float v = 0.f;
#pragma unroll
      for (int j = 0; j < kWarps; ++j) v += red[j][c];
      a.part[static_cast<size_t>(blockIdx.x) * a.head_dim + c] = v;
    }
  }
}

// Gains' gradients from the blocks' rows, in a fixed order: a block per 32 columns of one
// gain (blockIdx.y: q or k), warp j takes rows j, j + 32, ..., then the 32 sums are added.  It is
// launched while the first kernel runs and waits for its end: 0.8 to 1.1 us less of every call.
__global__ void __launch_bounds__(1024) k_gain_reduce(const float* part, int q_rows,
                                                      int k_rows, int head_dim,
                                                      float* __restrict__ dq_gain,
                                                      float* __restrict__ dk_gain) {
  __shared__ float red[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  const int rows = blockIdx.y ? k_rows : q_rows;
  if (blockIdx.y) part += static_cast<size_t>(q_rows) * head_dim;
  float* out = blockIdx.y ? dk_gain : dq_gain;
  if (out == nullptr) return;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float v = 0.f;
  if (col < head_dim)
#pragma unroll 4
    for (int r = warp; r < rows; r += 32) v += part[static_cast<size_t>(r) * head_dim + col];
  red[warp][lane] = v;
  __syncthreads();
  v = red[lane][warp];  // warp c adds the 32 sums of column c
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane == 0 && blockIdx.x * 32 + warp < head_dim) out[blockIdx.x * 32 + warp] = v;
}

template <typename T, int C, bool HALVES, int LPH, int MODE, bool WHOLE>
int launch(const DevCtx& ctx, HeadRows& a, cudaStream_t stream) {
  constexpr int kGroup = pass_count<T, C, MODE>() * (32 / LPH);
  const int sms = std::min(ctx.num_sms, kMaxSkCtas);
  const long long most = 1ll * blocks_per_sm(MODE, C) * sms;
  // An item is a token's heads (of q, or of k).  Where tokens are too few to keep the SMs busy
  // that way, it is `per` groups of them: of 1 to 8, 16, 32, ... the number for which the warps that
  // fit would be done first, each going through its share of the items one after the other, every
  // item computing its token's angles again.  At 300 tokens of 24 + 24 heads norm + rotation takes 4.8 us instead
  // of 6.0; at 3 x 11,341 tokens, where whole tokens are kept, the same choice costs 126 instead
  // of 106.
  int groups[2];
  for (int w = 0; w < 2; ++w) {
    groups[w] = (a.heads[w] + kGroup - 1) / kGroup;
    a.parts[w] = 1;
  }
  if (a.rows < 16ll * sms) {
    long long best = -1;
    for (int per = 1; per <= std::max(groups[0], groups[1]); per = per < 8 ? per + 1 : 2 * per) {
      const long long n = a.rows * ((groups[0] + per - 1) / per + (groups[1] + per - 1) / per);
      const long long time = (n + most * kWarps - 1) / (most * kWarps) * (per + kItemCost);
      if (best >= 0 && time >= best) continue;
      best = time;
      for (int w = 0; w < 2; ++w) a.parts[w] = std::max(1, (groups[w] + per - 1) / per);
    }
  }
  long long items[2], cost[2];
  for (int w = 0; w < 2; ++w) {
    items[w] = groups[w] > 0 ? a.rows * a.parts[w] : 0;
    cost[w] = items[w] * kItemCost + (groups[w] > 0 ? a.rows * groups[w] : 0);
  }
  // q's share of the blocks is its share of the work
  long long blocks[2];
  for (int w = 0; w < 2; ++w) {
    const long long share = items[w] > 0 ? most * cost[w] / (cost[0] + cost[1]) : 0;
    blocks[w] = std::min<long long>((items[w] + kWarps - 1) / kWarps, std::max<long long>(share, 1));
  }
  a.q_blocks = static_cast<int>(blocks[0]);
  if (blocks[0] + blocks[1] > 0) {
    k_head_rows<T, C, HALVES, LPH, MODE, WHOLE>
        <<<static_cast<unsigned>(blocks[0] + blocks[1]), kWarps * 32, 0, stream>>>(a);
    if (int rc = check_launch("head rows")) return rc;
  }
  if (MODE != kModeNormBwd || (!a.dq_gain && !a.dk_gain)) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.head_dim + 31) / 32, 2);
  cfg.blockDim = dim3(1024);
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, k_gain_reduce, static_cast<const float*>(a.part),
                     static_cast<int>(blocks[0]), static_cast<int>(blocks[1]), a.head_dim, a.dq_gain,
                     a.dk_gain);
  return check_launch("gain reduce");
}

template <typename T, int C, bool HALVES, int LPH, bool WHOLE>
int launch_mode(const DevCtx& ctx, int mode, HeadRows& a, cudaStream_t stream) {
  if constexpr (C == 8)
    if (mode == kModeRope) return launch<T, C, HALVES, LPH, kModeRope, WHOLE>(ctx, a, stream);
  if (mode == kModeNorm) return launch<T, C, HALVES, LPH, kModeNorm, WHOLE>(ctx, a, stream);
  return launch<T, C, HALVES, LPH, kModeNormBwd, WHOLE>(ctx, a, stream);
}

template <typename T, int C, bool HALVES, bool WHOLE>
int launch_width(const DevCtx& ctx, int mode, HeadRows& a, cudaStream_t stream) {
  if (a.head_dim <= 64) return launch_mode<T, C, HALVES, 64 / C, WHOLE>(ctx, mode, a, stream);
  if (a.head_dim <= 128) return launch_mode<T, C, HALVES, 128 / C, WHOLE>(ctx, mode, a, stream);
  return launch_mode<T, C, HALVES, 256 / C, WHOLE>(ctx, mode, a, stream);
}

template <typename T, int C, bool HALVES>
int launch_turned(const DevCtx& ctx, int mode, HeadRows& a, cudaStream_t stream) {
  return 2 * a.n_pairs == a.head_dim ? launch_width<T, C, HALVES, true>(ctx, mode, a, stream)
                                     : launch_width<T, C, HALVES, false>(ctx, mode, a, stream);
}

template <typename T>
int launch_type(const DevCtx& ctx, int mode, HeadRows& a, bool halves, cudaStream_t stream) {
  // (the rotation alone has nothing to gain: 47 us against 51 at 2 x 11,344 tokens)
  if constexpr (sizeof(T) == 2) {
    if (mode != kModeRope && a.head_dim % 16 == 0 && (!halves || a.n_pairs % 8 == 0))
      return halves ? launch_turned<T, 16, true>(ctx, mode, a, stream)
                    : launch_turned<T, 16, false>(ctx, mode, a, stream);
  }
  return halves ? launch_turned<T, 8, true>(ctx, mode, a, stream)
                : launch_turned<T, 8, false>(ctx, mode, a, stream);
}

}  // namespace

int launch_head_rows(const DevCtx& ctx, int dtype, int mode, HeadRows a, bool halves,
                     cudaStream_t stream) {
  if (dtype == 0) return launch_type<bf16>(ctx, mode, a, halves, stream);
  if (dtype == 1) return launch_type<__half>(ctx, mode, a, halves, stream);
  return launch_type<float>(ctx, mode, a, halves, stream);
}

}  // namespace h3b
