// The wide attention's schedule: how the work of a batch is cut into one range per CTA, and
// the walk over a range.  Host and device, so that it can be enumerated without a GPU.
#pragma once

#include "kernels.h"

namespace h3b {

constexpr int kBlockQ = 256;

__host__ __device__ inline int clamp_len(int v, int top) { return v < 0 ? 0 : v > top ? top : v; }

struct Lens {
  int q, kv;
};

__host__ __device__ inline Lens lens_of(const PrefixArgs& a, int b) {
  Lens l;
  l.kv = a.kv_len ? clamp_len(a.kv_len[b], a.n_kv) : a.n_kv;
  l.q = a.q_len ? clamp_len(a.q_len[b], a.n_q) : a.n_q;
  return l;
}

// A unit, and where its work starts in the batch's.
struct Unit {
  int b, h, qb;
  Lens len;
  int steps;        // key tiles (at least one, so that rows without keys are written)
  int step_work;    // cost of a step
  long long base;
};

// Cost of a step with two query tiles and of one whose second tile is empty, and of a unit's
// start and end (the first S, the normalise and store of O), in the same measure.
constexpr int kWorkTwo = 8, kWorkOne = 5, kWorkUnit = 12;

__host__ __device__ inline int blocks_of(const Lens& l) { return (l.q + kBlockQ - 1) / kBlockQ; }

__host__ __device__ inline void unit_cost(const PrefixArgs& a, const Lens& l, int qb, int& steps,
                                          int& step_work) {
  int own = l.kv;
  if (a.causal) {
    const int last = qb * kBlockQ + kBlockQ < l.q ? qb * kBlockQ + kBlockQ : l.q;
    own = clamp_len(last + l.kv - l.q, l.kv);
  }
  steps = a.prefix_tiles + (own + 127) / 128;
  if (steps < 1) steps = 1;
  step_work = qb * kBlockQ + 128 < l.q ? kWorkTwo : kWorkOne;
}

// Work of one head of a sequence.
__host__ __device__ inline long long head_work(const PrefixArgs& a, const Lens& l) {
  const int nb = blocks_of(l);
  if (nb == 0) return 0;
  long long sum = 0;
  int steps, w;
  if (a.causal) {
    for (int qb = 0; qb < nb; ++qb) {
      unit_cost(a, l, qb, steps, w);
      sum += kWorkUnit + static_cast<long long>(steps) * w;
    }
    return sum;
  }
  unit_cost(a, l, nb - 1, steps, w);
  sum = kWorkUnit + static_cast<long long>(steps) * w;
  return sum + (nb - 1ll) * (kWorkUnit + static_cast<long long>(steps) * kWorkTwo);
}

// The first step of the unit at or after position pos (steps where there is none).
__host__ __device__ inline int step_at(const Unit& u, long long pos) {
  const long long r = pos - u.base - kWorkUnit;
  if (r <= 0) return 0;
  const long long j = (r + u.step_work - 1) / u.step_work;
  return j < u.steps ? static_cast<int>(j) : u.steps;
}

__host__ __device__ inline void unit_set(const PrefixArgs& a, Unit& u) {
  unit_cost(a, u.len, u.qb, u.steps, u.step_work);
}

// The unit before u (base known); false at the batch's start.
__host__ __device__ inline bool unit_prev(const PrefixArgs& a, Unit& u) {
  if (u.qb > 0) {
    --u.qb;
  } else {
    if (u.h > 0) {
      --u.h;
    } else {
      do {
        if (u.b == 0) return false;
        --u.b;
        u.len = lens_of(a, u.b);
      } while (u.len.q == 0);
      u.h = a.heads - 1;
    }
    u.qb = blocks_of(u.len) - 1;
  }
  unit_set(a, u);
  u.base -= kWorkUnit + static_cast<long long>(u.steps) * u.step_work;
  return true;
}

__host__ __device__ inline long long range_begin(long long total, int cta, int ctas) {
  return total * cta / ctas;
}

// Whether CTA `cta` holds steps of the unit.
__host__ __device__ inline bool has_piece(const Unit& u, long long total, int cta, int ctas) {
  return step_at(u, range_begin(total, cta, ctas)) < step_at(u, range_begin(total, cta + 1, ctas));
}

// A CTA's range [begin, end) of positions, walked from its end; one segment is the part of a
// unit that lies in it, steps [j0, j1).
struct Walk {
  Unit u;
  long long begin, end;
  int j0, j1;
  bool more;

  __host__ __device__ inline void clip() {
    j0 = step_at(u, begin);
    j1 = step_at(u, end);
  }
  __host__ __device__ inline void settle(const PrefixArgs& a) {
    while (more) {
      clip();
      if (j0 < j1) return;
      more = u.base > begin && unit_prev(a, u);
    }
  }
  __host__ __device__ inline void next(const PrefixArgs& a) {
    more = u.base > begin && unit_prev(a, u);
    settle(a);
  }
};

}  // namespace h3b
