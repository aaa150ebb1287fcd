// The schedules of the shared-prefix attention: how the work of a batch is cut into one range
// per CTA, and the walk over a range, of its wide and of its narrow form; and where the rows of a
// swizzled tile lie.  Host and device, so that they can be enumerated without a GPU.
#pragma once

#include "kernels.h"

#include <algorithm>

namespace h3b {

constexpr int kBlockQ = 256;
// Work is counted in 32 bits: calls of more than this are refused (at 2^31, some 10^8 tiles).
constexpr long long kMaxWork = (1ll << 31) - 1;

__host__ __device__ inline int clamp_len(int v, int top) { return v < 0 ? 0 : v > top ? top : v; }

// Where the 16-byte piece `piece` of row `row` lies in a tile of 128 rows in boxes of 128 bytes a
// row, swizzled as the tensor core reads them; in pieces.
__host__ __device__ inline int tile_piece(int row, int piece) {
  return (piece >> 3) * (128 * 8) + row * 8 + ((piece & 7) ^ (row & 7));
}

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
  int base;
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
__host__ __device__ inline int head_work(const PrefixArgs& a, const Lens& l) {
  const int nb = blocks_of(l);
  if (nb == 0) return 0;
  int sum = 0;
  int steps, w;
  if (a.causal) {
    for (int qb = 0; qb < nb; ++qb) {
      unit_cost(a, l, qb, steps, w);
      sum += kWorkUnit + steps * w;
    }
    return sum;
  }
  unit_cost(a, l, nb - 1, steps, w);
  sum = kWorkUnit + steps * w;
  return sum + (nb - 1) * (kWorkUnit + steps * kWorkTwo);
}

// The first step of the unit at or after position pos (steps where there is none).
__host__ __device__ inline int step_at(const Unit& u, int pos) {
  const int r = pos - u.base - kWorkUnit;
  if (r <= 0) return 0;
  // (constant divisors: a shift and a multiplication)
  const int j = u.step_work == kWorkTwo ? (r + kWorkTwo - 1) / kWorkTwo : (r + kWorkOne - 1) / kWorkOne;
  return j < u.steps ? j : u.steps;
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
  u.base -= kWorkUnit + u.steps * u.step_work;
  return true;
}

// The cut of `total` into equal ranges: the first `more` of them are `each` + 1 long, the
// others `each`.
struct Cut {
  int each, more;
  __host__ __device__ inline int begin(int cta) const {
    return each * cta + (cta < more ? cta : more);
  }
  // the range that holds position pos
  __host__ __device__ inline int cta_of(int pos) const {
    const int head = more * (each + 1);
    return pos < head ? pos / (each + 1) : more + (pos - head) / each;
  }
};
__host__ __device__ inline Cut cut(int total, int ctas) { return Cut{total / ctas, total % ctas}; }

// Whether CTA `cta` holds steps of the unit.
__host__ __device__ inline bool has_piece(const Unit& u, const Cut& c, int cta) {
  return step_at(u, c.begin(cta)) < step_at(u, c.begin(cta + 1));
}

// A CTA's range [begin, end) of positions, walked from its end; one segment is the part of a
// unit that lies in it, steps [j0, j1).
struct Walk {
  Unit u;
  int begin, end;
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

// The first CTA that may hold steps of the unit, whose last step is `me`'s.
__host__ __device__ inline int first_cta(const Unit& u, const Cut& c, int me) {
  while (me > 0 && c.begin(me) > u.base) --me;
  return me;
}

// CTAs that share a unit, on average, at most: the one that joins the states reads them one after
// the other.  With 8, 4 and 3, us: one sequence of 12 heads and 127 queries over 2,712 keys 34, 27
// and 27; 512 queries of 6 heads over 4,096 45, 41 and 44; two of 100 over 8,000 45, 41 and 47.
constexpr int kMaxPieces = 4;
inline int wide_ctas(const PrefixArgs& a, int most) {
  const long long units = 1ll * a.batch * a.heads * ((a.n_q + kBlockQ - 1) / kBlockQ);
  return static_cast<int>(std::min<long long>(units * kMaxPieces, most));
}

// The most work a call of these sizes can have (in 64 bits the largest would not fit).
inline double wide_work_cap(const PrefixArgs& a) {
  const double tiles = (a.n_prefix + 127) / 128 + (a.n_kv + 127) / 128;
  return 1.0 * a.batch * a.heads * ((a.n_q + kBlockQ - 1) / kBlockQ) * (kWorkUnit + (tiles + 1) * kWorkTwo);
}

// ------------------------------------------------------------------------- narrow form
// Units: the prefix's first, (key head, group of gt query heads, chunk of bt sequences), then
// every sequence's own, (sequence, key head, group of query heads).  A unit's rows are its
// sequences' queries of those heads; its steps the 128-key tiles of the prefix or of the
// sequence.  Units without keys or queries have no work.
// Cost of a step and of a unit's start and end, and of a step of the prefix where its rows take
// all four quarters of tensor memory.  Measured, us (unit, full step): 512 sequences of 24 / 8
// heads with one step each over 4,096 shared keys (126 rows) 180 (16, 8), 163 (12, 8), 146 (12, 10),
// 150 (12, 13); 48 with 1 to 16 steps over 16,133 (72 rows) 69 with a unit of 12 or 16, 76 with 6.
constexpr int kOwnStep = 8, kNarrowUnit = 12;
constexpr int kFarFull = 10;
inline int narrow_far_step(int rows) { return rows > 96 ? kFarFull : kOwnStep; }

struct NarrowUnit {
  int index;        // prefix units, then batch x own units
  int b;            // sequence; -1: of the prefix
  int in_b;         // own: index inside the sequence
  Lens len;
  int steps;
  int base;
};

__host__ __device__ inline int narrow_work(int steps) {
  return steps > 0 ? kNarrowUnit + steps * kOwnStep : 0;
}
__host__ __device__ inline int narrow_far_work(const PrefixArgs& a) {
  return kNarrowUnit + a.prefix_tiles * a.far_step;
}
__host__ __device__ inline int narrow_work(const PrefixArgs& a, const NarrowUnit& u) {
  return u.b < 0 ? narrow_far_work(a) : narrow_work(u.steps);
}
__host__ __device__ inline int narrow_steps(const Lens& l) {
  return l.q > 0 ? (l.kv + 127) / 128 : 0;
}
__host__ __device__ inline int narrow_prefix_work(const PrefixArgs& a) {
  return a.prefix_units * narrow_far_work(a);
}

__host__ __device__ inline int narrow_step_at(const PrefixArgs& a, const NarrowUnit& u, int pos) {
  const int r = pos - u.base - kNarrowUnit;
  if (r <= 0) return 0;
  // (either divisor a constant: a shift or a multiplication)
  const bool full = u.b < 0 && a.far_step == kFarFull;
  const int j = full ? (r + kFarFull - 1) / kFarFull : (r + kOwnStep - 1) / kOwnStep;
  return j < u.steps ? j : u.steps;
}

// The first of a sequence's units at or after sequence b that has work.
__host__ __device__ inline bool narrow_own(const PrefixArgs& a, NarrowUnit& u, int b) {
  for (; b < a.batch; ++b) {
    u.len = lens_of(a, b);
    u.steps = narrow_steps(u.len);
    if (u.steps == 0) continue;
    u.b = b;
    u.in_b = 0;
    u.index = a.prefix_units + b * a.own_units;
    return true;
  }
  return false;
}

__host__ __device__ inline bool narrow_next(const PrefixArgs& a, NarrowUnit& u) {
  u.base += narrow_work(a, u);
  if (u.b < 0) {
    if (++u.index < a.prefix_units) return true;
    return narrow_own(a, u, 0);
  }
  if (++u.in_b < a.own_units) {
    ++u.index;
    return true;
  }
  return narrow_own(a, u, u.b + 1);
}

// CTAs that get a range: as many as there are, but at least kMinRange for each.
constexpr int kMinRange = 2 * kOwnStep + kNarrowUnit;
// A range longer than a unit's start and a step: at each end of a unit at most one CTA has some of
// the unit's range and none of its steps (narrow_side leaves it out).
static_assert(kMinRange > kNarrowUnit + kOwnStep && kMinRange > kNarrowUnit + kFarFull,
              "range too short");
__host__ __device__ inline int narrow_ctas(int total, int most) {
  const int n = total / kMinRange;
  return n < 1 ? 1 : n < most ? n : most;
}

struct NarrowWalk {
  NarrowUnit u;
  int begin, end;
  int j0, j1;
  bool more;

  __host__ __device__ inline void settle(const PrefixArgs& a) {
    while (more) {
      j0 = narrow_step_at(a, u, begin);
      j1 = narrow_step_at(a, u, end);
      if (j0 < j1) return;
      more = u.base + narrow_work(a, u) < end && narrow_next(a, u);
    }
  }
  __host__ __device__ inline void next(const PrefixArgs& a) {
    more = u.base + narrow_work(a, u) < end && narrow_next(a, u);
    settle(a);
  }
};

inline long long narrow_work_cap(const PrefixArgs& a) {
  const long long far = (a.n_prefix + 127) / 128, own = (a.n_kv + 127) / 128;
  return a.prefix_units * (kNarrowUnit + far * a.far_step) +
         1ll * a.batch * a.own_units * (kNarrowUnit + own * kOwnStep);
}

// Where a segment's state goes: slots of the prefix hold bt * gt * n_q rows, own ones gt * n_q;
// CTA + unit is different for every segment.
__host__ __device__ inline size_t narrow_row(const PrefixArgs& a, bool far, int index, int cta,
                                             int chain) {
  const size_t own_rows = size_t(a.gt) * a.n_q, far_rows = own_rows * a.bt;
  const size_t far_slots = a.prefix_units > 0 ? size_t(a.prefix_units) + a.ctas : 0;
  if (far) return (size_t(index + cta) * 2 + chain) * far_rows;
  return far_slots * 2 * far_rows + (size_t(index - a.prefix_units + cta) * 2 + chain) * own_rows;
}

// The states of one side (the prefix, the own keys) of a row: CTAs c0 .. c1 hold the unit's
// steps, two chains each; state i is chain i & 1 of CTA c0 + (i >> 1).
struct Side {
  int c0, n;         // n states
  size_t row, step;  // row of state 0 in the workspace, and from one CTA's to the next
  size_t chain;      // from chain 0's to chain 1's
};

__host__ __device__ inline Side narrow_side(const PrefixArgs& a, const Cut& all, bool far, int index,
                                            int base, int steps, int in_unit) {
  Side s;
  NarrowUnit u;
  u.b = far ? -1 : 0;
  u.base = base;
  u.steps = steps;
  // a CTA at either end may hold some of the unit's range but no step of it
  s.c0 = all.cta_of(base);
  int c1 = all.cta_of(base + narrow_work(a, u) - 1);
  if (narrow_step_at(a, u, all.begin(s.c0 + 1)) == 0) ++s.c0;
  if (narrow_step_at(a, u, all.begin(c1)) == steps) --c1;
  s.n = 2 * (c1 - s.c0 + 1);
  s.row = narrow_row(a, far, index, s.c0, 0) + in_unit;
  s.chain = size_t(a.gt) * a.n_q * (far ? a.bt : 1);
  s.step = 2 * s.chain;
  return s;
}

// The narrow form's units.
inline void narrow_units(PrefixArgs& a) {
  a.gt = std::min(a.group, 128 / a.n_q);
  a.head_groups = (a.group + a.gt - 1) / a.gt;
  a.gt = (a.group + a.head_groups - 1) / a.head_groups;
  a.bt = a.n_prefix > 0 ? std::min(a.batch, 128 / (a.gt * a.n_q)) : 1;
  a.chunks = (a.batch + a.bt - 1) / a.bt;
  a.bt = (a.batch + a.chunks - 1) / a.chunks;
  a.own_units = a.kv_heads * a.head_groups;
  a.far_step = narrow_far_step(a.bt * a.gt * a.n_q);
  a.prefix_units = a.n_prefix > 0 ? a.own_units * a.chunks : 0;
}

// Rows of the narrow form's workspace.
inline size_t narrow_rows(const PrefixArgs& a) {
  const size_t own = size_t(a.gt) * a.n_q;
  size_t rows = 2 * (size_t(a.batch) * a.own_units + kMaxSkCtas) * own;
  if (a.prefix_units > 0) rows += 2 * (size_t(a.prefix_units) + kMaxSkCtas) * own * a.bt;
  return rows;
}

// The narrow form, for at most this many queries a sequence.  Narrow and wide, in us, 8 sequences
// over 4,096 shared keys and 1,000 of their own: 24 / 8 heads 22 and 94 with one query, 50 and 94
// with 32, 90 and 94 with 64, 115 and 95 with 96; 24 / 24 heads 77 and 97 with 64, 116 and 97 with
// 96.  The narrow form's states, 8 * (HD / 2 + 1) bytes a row, side and chain, are written and read
// back, so its cost and its workspace grow with the batch; over 4,096 shared and 256 own keys, heads
// of 128, 16, 32 and 64 queries, narrow, and wide (which they hardly change):
//   24 / 8 heads, 64 sequences 152, 362, 956 and 573; 256: 584, 1,392, 3,775 and 2,247
//   24 / 24 heads, 64 sequences 152, 281, 590 and 579; 256: 560, 1,052, 2,312 and 2,260
// With 33 to 64 queries of shared key heads the wide form would be the faster one; the rule has no
// part for that yet.  The workspace there is 1.1 GB for 256 sequences of 64 queries.  The second
// limit bounds the schedule's integers, not the workspace.
constexpr int kNarrowQueries = 64;

inline bool use_narrow(PrefixArgs a) {
  if (a.n_q > kNarrowQueries || 1ll * a.batch * a.heads > (1 << 20)) return false;
  narrow_units(a);
  return narrow_work_cap(a) * 2 <= kMaxWork;
}

}  // namespace h3b
