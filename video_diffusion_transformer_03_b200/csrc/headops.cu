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
// one or the other, which keeps one set of gains and sums in registers): each lane owns eight
// channels of a head (the four pairs 4 s .. 4 s + 3 of its slot s, in both pairings), so the
// angles of a token are computed once for all heads of the warp's item, pairs never cross
// lanes, and the only shuffles are those of the norm's sums.  An item's first loads are issued
// before its angles are computed, later ones while the heads before them are worked on.
#include "kernels.h"
#include "ptx.cuh"

#include <algorithm>
#include <cuda_fp16.h>
#include <type_traits>

namespace h3b {

namespace {

constexpr int kWarps = 4;  // warps of a block

enum Mode : int { kModeRope = 0, kModeNorm = 1, kModeNormBwd = 2 };

// A lane's eight channels: chunk c0 .. c0 + 3 and chunk c1 .. c1 + 3.  Adjacent pairing:
// c1 = c0 + 4 and pair i is (f[2 i], f[2 i + 1]).  Half-split pairing: c1 = c0 + rot / 2 and
// pair i is (f[i], f[4 + i]); behind the rotated width c1 = c0 + 4.
template <typename T>
struct Raw {
  uint32_t w[2 * sizeof(T)];
};

template <typename T, bool HALVES>
__device__ __forceinline__ void load_raw(const T* p, int c0, int c1, Raw<T>& r) {
  if constexpr (sizeof(T) == 4) {
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

template <typename T, bool HALVES>
__device__ __forceinline__ void store_raw(T* p, int c0, int c1, const Raw<T>& r) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<uint4*>(p + c0) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    *reinterpret_cast<uint4*>(p + c1) = make_uint4(r.w[4], r.w[5], r.w[6], r.w[7]);
  } else if constexpr (HALVES) {
    *reinterpret_cast<uint2*>(p + c0) = make_uint2(r.w[0], r.w[1]);
    *reinterpret_cast<uint2*>(p + c1) = make_uint2(r.w[2], r.w[3]);
  } else {
    *reinterpret_cast<uint4*>(p + c0) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
  }
}

template <typename T>
__device__ __forceinline__ void widen(const Raw<T>& r, float (&f)[8]) {
  if constexpr (std::is_same_v<T, float>) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(r.w[i]);
  } else if constexpr (std::is_same_v<T, __half>) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&r.w[i]));
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = unpack_bf16x2(r.w[i]);
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  }
}

template <typename T>
__device__ __forceinline__ void narrow(const float (&f)[8], Raw<T>& r) {
  if constexpr (std::is_same_v<T, float>) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i] = __float_as_uint(f[i]);
  } else if constexpr (std::is_same_v<T, __half>) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 v = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      r.w[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
  }
}

// sin and cos of 2 pi t.  Adding 1.5 * 2^52 rounds t to the nearest integer.
__device__ __forceinline__ void sincos_turns(double t, float& s, float& c) {
  const double magic = 6755399441055744.0;
  const double n = (t + magic) - magic;
  sincospif(2.0f * static_cast<float>(t - n), &s, &c);
}

// The pairs of f turned by (c, s).
template <bool HALVES>
__device__ __forceinline__ void rotate(float (&f)[8], const float (&c)[4], const float (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int ia = HALVES ? i : 2 * i, ib = HALVES ? 4 + i : 2 * i + 1;
    const float a = f[ia], b = f[ib];
    f[ia] = fmaf(a, c[i], -(b * s[i]));
    f[ib] = fmaf(a, s[i], b * c[i]);
  }
}

// Sum over the LPH lanes of a head.
template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = LPH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A group is kPass passes of 32 / LPH heads.  An item is one token, or (parts > 1, where
// tokens are few) an equal share of its groups.
template <typename T, int MODE>
constexpr int pass_count() {
  return (MODE == kModeNormBwd || sizeof(T) == 4) ? 1 : 2;
}

// Blocks that are on an SM at a time (their registers: 64, 80 and 128 a thread); the grid is
// that many a SM at most.
constexpr int blocks_per_sm(int mode) {
  return mode == kModeNormBwd ? kHeadRowsBwdPerSm : mode == kModeNorm ? 6 : 8;
}

template <typename T, bool HALVES, int LPH, int MODE>
__global__ void __launch_bounds__(kWarps * 32, blocks_per_sm(MODE)) k_head_rows(const __grid_constant__ HeadRows a) {
  constexpr int kPass = pass_count<T, MODE>();
  constexpr int kHeads = 32 / LPH;
  constexpr int kGroup = kPass * kHeads;
  constexpr bool kBwd = MODE == kModeNormBwd;
  const int lane = threadIdx.x & 31;
  const int slot = lane % LPH, sub = lane / LPH;
  const bool live = slot * 8 < a.head_dim;
  const bool turned = slot * 4 < a.n_pairs;
  const bool half_slot = HALVES && turned;
  const int c0 = half_slot ? slot * 4 : slot * 8;
  const int c1 = half_slot ? a.n_pairs + slot * 4 : slot * 8 + 4;

  const int w = static_cast<int>(blockIdx.x) >= a.q_blocks;
  const unsigned block = w ? blockIdx.x - a.q_blocks : blockIdx.x;
  const unsigned blocks = w ? gridDim.x - a.q_blocks : static_cast<unsigned>(a.q_blocks);
  const HeadView in = a.in[w], out = a.out[w];
  const int heads = a.heads[w], parts = a.parts[w];
  const int groups = (heads + kGroup - 1) / kGroup;
  const unsigned n_items = static_cast<unsigned>(a.rows) * parts;

  double turns[4] = {0.0, 0.0, 0.0, 0.0};
  uint32_t axes = 0;
  float gain[8];
  float acc[8];
  bool have_lane = false;
  const float inv_hd = 1.0f / static_cast<float>(a.head_dim);
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;

  for (unsigned item = block * kWarps + (threadIdx.x >> 5); item < n_items;
       item += blocks * kWarps) {
    unsigned row = item, b = 0;
    int g0 = 0, g1 = groups;
    if (parts > 1) {
      row = item / parts;
      const int part = static_cast<int>(item - row * parts);
      g0 = groups * part / parts;
      g1 = groups * (part + 1) / parts;
    }
    unsigned t = row;
    if (a.rows != a.tokens) {
      b = row / static_cast<unsigned>(a.tokens);
      t = row - b * static_cast<unsigned>(a.tokens);
    }
    const T* src = static_cast<const T*>(in.data) + b * in.batch + t * in.token;
    const T* grd = nullptr;
    if constexpr (kBwd)
      grd = static_cast<const T*>(a.grad[w].data) + b * a.grad[w].batch + t * a.grad[w].token;
    T* dst = static_cast<T*>(out.data) + b * out.batch + t * out.token;

    Raw<T> x[kPass], gy[kPass];
    auto load = [&](int g) {
#pragma unroll
      for (int i = 0; i < kPass; ++i) {
        const int h = g * kGroup + i * kHeads + sub;
        const bool on = live && h < heads;
        x[i] = Raw<T>{};
        if (on) load_raw<T, HALVES>(src + h * in.head, c0, c1, x[i]);
        if constexpr (kBwd) {
          gy[i] = Raw<T>{};
          if (on) load_raw<T, HALVES>(grd + h * a.grad[w].head, c0, c1, gy[i]);
        }
      }
    };
    load(g0);
    if (!have_lane) {
      // this lane's constants, behind its first loads
      have_lane = true;
      if (turned) {
        const double2 t0 = *reinterpret_cast<const double2*>(a.turns + slot * 4);
        const double2 t1 = *reinterpret_cast<const double2*>(a.turns + slot * 4 + 2);
        turns[0] = t0.x; turns[1] = t0.y; turns[2] = t1.x; turns[3] = t1.y;
        axes = *reinterpret_cast<const uint32_t*>(a.axis + slot * 4);
      }
      if constexpr (MODE != kModeRope) {
        const float* g = w ? a.k_gain : a.q_gain;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          gain[i] = (g != nullptr && live) ? __ldg(g + (i < 4 ? c0 + i : c1 + i - 4)) : 1.f;
      }
    }
    float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
    if (turned) {
      // pairs past the rotated width have turns 0: they stay
      const float* pos = a.pos + b * a.pos_batch + static_cast<size_t>(t) * a.n_axes;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (slot * 4 + i < a.n_pairs)
          sincos_turns(static_cast<double>(__ldg(pos + ((axes >> (8 * i)) & 0xffu))) * turns[i],
                       sn[i], cs[i]);
        if (kBwd || (MODE == kModeRope && a.inverse)) sn[i] = -sn[i];
      }
    }
    for (int g = g0; g < g1; ++g) {
      Raw<T> xc[kPass], gc[kPass];
#pragma unroll
      for (int i = 0; i < kPass; ++i) {
        xc[i] = x[i];
        if constexpr (kBwd) gc[i] = gy[i];
      }
      if (g + 1 < g1) load(g + 1);
#pragma unroll
      for (int i = 0; i < kPass; ++i) {
        const int h = g * kGroup + i * kHeads + sub;
        float f[8];
        widen<T>(xc[i], f);
        if constexpr (MODE != kModeRope) {
          float ss = 0.f;
#pragma unroll
          for (int c = 0; c < 8; ++c) ss = fmaf(f[c], f[c], ss);
          const float rstd = rsqrtf(head_sum<LPH>(ss) * inv_hd + a.eps);
          if constexpr (!kBwd) {
#pragma unroll
            for (int c = 0; c < 8; ++c) f[c] *= rstd * gain[c];
          } else {
            float z[8];
            widen<T>(gc[i], z);
            rotate<HALVES>(z, cs, sn);
            float dot = 0.f;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              f[c] *= rstd;
              acc[c] = fmaf(z[c], f[c], acc[c]);
              z[c] *= gain[c];
              dot = fmaf(z[c], f[c], dot);
            }
            dot = head_sum<LPH>(dot) * inv_hd;
#pragma unroll
            for (int c = 0; c < 8; ++c) f[c] = rstd * fmaf(-f[c], dot, z[c]);
          }
        }
        if constexpr (!kBwd) rotate<HALVES>(f, cs, sn);
        if (live && h < heads) {
          Raw<T> y;
          narrow<T>(f, y);
          store_raw<T, HALVES>(dst + h * out.head, c0, c1, y);
        }
      }
    }
  }
  if constexpr (kBwd) {
    // the block's share of the gain's gradient: lanes of the same slot, then its warps in
    // order, then one row [head_dim] of the workspace
    __shared__ float red[kWarps][LPH * 8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      float v = acc[c];
#pragma unroll
      for (int o = LPH; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (sub == 0 && live) red[threadIdx.x >> 5][c < 4 ? c0 + c : c1 + c - 4] = v;
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
// gain (blockIdx.y: q or k), warp j takes rows j, j + 32, ..., then the 32 sums are added.
__global__ void __launch_bounds__(1024) k_gain_reduce(const float* __restrict__ part, int q_rows,
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

template <typename T, bool HALVES, int LPH, int MODE>
int launch(const DevCtx& ctx, HeadRows& a, cudaStream_t stream) {
  constexpr int kGroup = pass_count<T, MODE>() * (32 / LPH);
  const int sms = std::min(ctx.num_sms, kMaxSkCtas);
  const long long most = 1ll * blocks_per_sm(MODE) * sms;
  // Tokens alone keep an SM busy from about 24 of its warps on; with fewer, a token's groups
  // of heads are dealt to several warps, each of which computes the token's angles again.
  long long items[2], total = 0;
  for (int w = 0; w < 2; ++w) {
    const int groups = (a.heads[w] + kGroup - 1) / kGroup;
    const long long want = a.rows > 0 ? (24ll * sms + a.rows - 1) / a.rows : 1;
    a.parts[w] = static_cast<int>(std::max<long long>(1, std::min<long long>(groups, want)));
    items[w] = groups > 0 ? a.rows * a.parts[w] : 0;
    total += items[w] * groups / a.parts[w];
  }
  // q's share of the blocks is its share of the work
  long long blocks[2];
  for (int w = 0; w < 2; ++w) {
    const int groups = (a.heads[w] + kGroup - 1) / kGroup;
    const long long share = total > 0 ? (most * items[w] * groups / a.parts[w]) / total : 0;
    blocks[w] = std::min<long long>((items[w] + kWarps - 1) / kWarps, std::max<long long>(share, 1));
  }
  a.q_blocks = static_cast<int>(blocks[0]);
  if (blocks[0] + blocks[1] > 0) {
    k_head_rows<T, HALVES, LPH, MODE>
        <<<static_cast<unsigned>(blocks[0] + blocks[1]), kWarps * 32, 0, stream>>>(a);
    if (int rc = check_launch("head rows")) return rc;
  }
  if (MODE != kModeNormBwd || (!a.dq_gain && !a.dk_gain)) return 0;
  k_gain_reduce<<<dim3((a.head_dim + 31) / 32, 2), 1024, 0, stream>>>(
      a.part, static_cast<int>(blocks[0]), static_cast<int>(blocks[1]), a.head_dim, a.dq_gain,
      a.dk_gain);
  return check_launch("gain reduce");
}

template <typename T, bool HALVES, int LPH>
int launch_mode(const DevCtx& ctx, int mode, HeadRows& a, cudaStream_t stream) {
  if (mode == kModeRope) return launch<T, HALVES, LPH, kModeRope>(ctx, a, stream);
  if (mode == kModeNorm) return launch<T, HALVES, LPH, kModeNorm>(ctx, a, stream);
  return launch<T, HALVES, LPH, kModeNormBwd>(ctx, a, stream);
}

template <typename T>
int launch_type(const DevCtx& ctx, int mode, HeadRows& a, bool halves, cudaStream_t stream) {
  const int hd = a.head_dim;
  if (halves)
    return hd <= 64    ? launch_mode<T, true, 8>(ctx, mode, a, stream)
           : hd <= 128 ? launch_mode<T, true, 16>(ctx, mode, a, stream)
                       : launch_mode<T, true, 32>(ctx, mode, a, stream);
  return hd <= 64    ? launch_mode<T, false, 8>(ctx, mode, a, stream)
         : hd <= 128 ? launch_mode<T, false, 16>(ctx, mode, a, stream)
                     : launch_mode<T, false, 32>(ctx, mode, a, stream);
}

}  // namespace

int launch_head_rows(const DevCtx& ctx, int dtype, int mode, HeadRows a, bool halves,
                     cudaStream_t stream) {
  if (dtype == 0) return launch_type<bf16>(ctx, mode, a, halves, stream);
  if (dtype == 1) return launch_type<__half>(ctx, mode, a, halves, stream);
  return launch_type<float>(ctx, mode, a, halves, stream);
}

}  // namespace h3b
