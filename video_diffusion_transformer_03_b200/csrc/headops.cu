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
// and writes dx.  So a warp takes a token and walks over its heads: each lane owns eight
// channels of a head (the four pairs 4 s .. 4 s + 3 of its slot s, in both pairings), so the
// angles of a token are computed once for all heads of the warp's item, pairs never cross
// lanes, and the only shuffles are those of the norm's sum.  Loads of kPass groups of heads
// are issued before the first use.
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

// Item = one token, or one chunk of kPass * (32 / LPH) heads of it where tokens are few
// (split_heads).  Chunks hold heads of q or of k, never both.
template <typename T, bool HALVES, int LPH, int MODE>
__global__ void __launch_bounds__(kWarps * 32) k_head_rows(const __grid_constant__ HeadRows a) {
  constexpr int kPass = (MODE == kModeNormBwd || sizeof(T) == 4) ? 2 : 4;
  constexpr int kHeads = 32 / LPH;           // heads of one pass
  constexpr int kChunk = kPass * kHeads;     // heads of a chunk
  const int lane = threadIdx.x & 31;
  const int slot = lane % LPH, sub = lane / LPH;
  const bool live = slot * 8 < a.head_dim;
  const bool turned = slot * 4 < a.n_pairs;
  const bool half_slot = HALVES && turned;
  const int c0 = half_slot ? slot * 4 : slot * 8;
  const int c1 = half_slot ? a.n_pairs + slot * 4 : slot * 8 + 4;

  double turns[4];
  int axis[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int p = slot * 4 + i;
    const bool in = p < a.n_pairs;
    turns[i] = in ? a.turns[in ? p : 0] : 0.0;
    axis[i] = in ? a.axis[in ? p : 0] : 0;
  }
  float gain[2][8];
  float acc[2][8];
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      acc[w][i] = 0.f;
      gain[w][i] = 1.f;
      if constexpr (MODE != kModeRope) {
        const float* g = w ? a.k_gain : a.q_gain;
        if (g != nullptr && live) gain[w][i] = __ldg(g + (i < 4 ? c0 + i : c1 + i - 4));
      }
    }
  const float inv_hd = 1.0f / static_cast<float>(a.head_dim);

  const int q_chunks = (a.heads[0] + kChunk - 1) / kChunk;
  const int k_chunks = (a.heads[1] + kChunk - 1) / kChunk;
  const int chunks = q_chunks + k_chunks;
  const long long n_items = a.split_heads ? a.rows * chunks : a.rows;
  const long long stride = static_cast<long long>(gridDim.x) * kWarps;
  for (long long item = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
       item < n_items; item += stride) {
    const long long row = a.split_heads ? item / chunks : item;
    const int first = a.split_heads ? static_cast<int>(item - row * chunks) : 0;
    const int last = a.split_heads ? first + 1 : chunks;
    const long long b = row / a.tokens, t = row - b * a.tokens;
    float cs[4], sn[4];
    if (a.n_pairs > 0) {
      const float* pos = a.pos + b * a.pos_batch + t * a.n_axes;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        cs[i] = 1.f;
        sn[i] = 0.f;
        if (slot * 4 + i < a.n_pairs)
          sincos_turns(static_cast<double>(__ldg(pos + axis[i])) * turns[i], sn[i], cs[i]);
        if (MODE == kModeNormBwd || (MODE == kModeRope && a.inverse)) sn[i] = -sn[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        cs[i] = 1.f;
        sn[i] = 0.f;
      }
    }
    for (int ch = first; ch < last; ++ch) {
      const int w = ch >= q_chunks;
      const int h0 = (w ? ch - q_chunks : ch) * kChunk + sub;
      const HeadView& in = a.in[w];
      const HeadView& out = a.out[w];
      const T* src = static_cast<const T*>(in.data) + b * in.batch + t * in.token;
      T* dst = static_cast<T*>(out.data) + b * out.batch + t * out.token;
      Raw<T> x[kPass], gy[kPass];
#pragma unroll
      for (int i = 0; i < kPass; ++i) {
        const int h = h0 + i * kHeads;
        const bool on = live && h < a.heads[w];
        x[i] = Raw<T>{};
        if (on) load_raw<T, HALVES>(src + h * in.head, c0, c1, x[i]);
        if constexpr (MODE == kModeNormBwd) {
          const HeadView& gv = a.grad[w];
          const T* g = static_cast<const T*>(gv.data) + b * gv.batch + t * gv.token;
          gy[i] = Raw<T>{};
          if (on) load_raw<T, HALVES>(g + h * gv.head, c0, c1, gy[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < kPass; ++i) {
        const int h = h0 + i * kHeads;
        float f[8];
        widen<T>(x[i], f);
        if constexpr (MODE != kModeRope) {
          float ss = 0.f;
#pragma unroll
          for (int c = 0; c < 8; ++c) ss = fmaf(f[c], f[c], ss);
          const float rstd = rsqrtf(head_sum<LPH>(ss) * inv_hd + a.eps);
          if constexpr (MODE == kModeNorm) {
#pragma unroll
            for (int c = 0; c < 8; ++c) f[c] *= rstd * (w ? gain[1][c] : gain[0][c]);
          } else {
            float z[8];
            widen<T>(gy[i], z);
            rotate<HALVES>(z, cs, sn);
            float dot = 0.f;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              f[c] *= rstd;
              const float zn = z[c] * f[c];
              if (w) acc[1][c] += zn;
              else acc[0][c] += zn;
              z[c] *= w ? gain[1][c] : gain[0][c];
              dot = fmaf(z[c], f[c], dot);
            }
            dot = head_sum<LPH>(dot) * inv_hd;
#pragma unroll
            for (int c = 0; c < 8; ++c) f[c] = rstd * fmaf(-f[c], dot, z[c]);
          }
        }
        if constexpr (MODE != kModeNormBwd) rotate<HALVES>(f, cs, sn);
        if (live && h < a.heads[w]) {
          Raw<T> y;
          narrow<T>(f, y);
          store_raw<T, HALVES>(dst + h * out.head, c0, c1, y);
        }
      }
    }
  }
  if constexpr (MODE == kModeNormBwd) {
    // the block's share of the gains' gradients: lanes of the same slot, then its warps in
    // order, then one row [2][head_dim] of the workspace
    __shared__ float red[kWarps][2][LPH * 8];
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        float v = acc[w][c];
#pragma unroll
        for (int o = LPH; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (sub == 0 && live) red[threadIdx.x >> 5][w][c < 4 ? c0 + c : c1 + c - 4] = v;
      }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.head_dim; i += kWarps * 32) {
      const int w = i >= a.head_dim, c = w ? i - a.head_dim : i;
      float v = 0.f;
#pragma unroll
      for (int j = 0; j < kWarps; ++j) v += red[j][w][c];
      a.part[static_cast<size_t>(blockIdx.x) * 2 * a.head_dim + i] = v;
    }
  }
}

// Gains' gradients from the blocks' rows, in a fixed order: a block per 32 columns, warp j
// takes rows j, j + 32, ..., then the 32 sums are added in order.
__global__ void __launch_bounds__(1024) k_gain_reduce(const float* __restrict__ part, int rows,
                                                      int head_dim, float* __restrict__ dq_gain,
                                                      float* __restrict__ dk_gain) {
  __shared__ float red[32][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (col < 2 * head_dim)
    for (int r = warp; r < rows; r += 32) v += part[static_cast<size_t>(r) * 2 * head_dim + col];
  red[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && col < 2 * head_dim) {
#pragma unroll
    for (int j = 1; j < 32; ++j) v += red[j][lane];
    float* out = col < head_dim ? dq_gain : dk_gain;
    if (out != nullptr) out[col < head_dim ? col : col - head_dim] = v;
  }
}

template <typename T, bool HALVES, int LPH, int MODE>
int launch(const DevCtx& ctx, HeadRows& a, cudaStream_t stream) {
  constexpr int kPass = (MODE == kModeNormBwd || sizeof(T) == 4) ? 2 : 4;
  constexpr int kChunk = kPass * (32 / LPH);
  const int chunks = (a.heads[0] + kChunk - 1) / kChunk + (a.heads[1] + kChunk - 1) / kChunk;
  // Tokens alone keep every SM's warps busy from 16 a SM on; with fewer a token's heads are
  // dealt to several warps, each of which computes the token's angles again.
  a.split_heads = a.rows < 16ll * ctx.num_sms;
  const long long items = a.split_heads ? a.rows * chunks : a.rows;
  const long long most = 1ll * (MODE == kModeNormBwd ? kHeadRowsBwdPerSm : kHeadRowsPerSm) *
                         std::min(ctx.num_sms, kMaxSkCtas);
  const long long blocks = std::min<long long>((items + kWarps - 1) / kWarps, most);
  if (blocks > 0) {
    k_head_rows<T, HALVES, LPH, MODE>
        <<<static_cast<unsigned>(blocks), kWarps * 32, 0, stream>>>(a);
    if (int rc = check_launch("head rows")) return rc;
  }
  if (MODE != kModeNormBwd) return 0;
  k_gain_reduce<<<(2 * a.head_dim + 31) / 32, 1024, 0, stream>>>(
      a.part, static_cast<int>(blocks), a.head_dim, a.dq_gain, a.dk_gain);
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
