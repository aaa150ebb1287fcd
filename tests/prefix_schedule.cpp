// The host side of csrc/prefix_sched.h as C functions, for tests/test_prefix_schedule.py.  The
// kernels find a range's first unit with a warp; here it is found by walking over the units.
#include "prefix_sched.h"

#include <vector>

using namespace h3b;

namespace {

PrefixArgs args_of(const int* sizes, const int* kv_len, const int* q_len) {
  PrefixArgs a;
  a.batch = sizes[0];
  a.n_q = sizes[1];
  a.heads = sizes[2];
  a.kv_heads = sizes[3];
  a.n_prefix = sizes[4];
  a.n_kv = sizes[5];
  a.causal = sizes[6];
  a.ctas = sizes[7];
  a.kv_len = kv_len;
  a.q_len = q_len;
  a.group = a.heads / a.kv_heads;
  a.prefix_tiles = (a.n_prefix + 127) / 128;
  return a;
}

}  // namespace

extern "C" {

int t_tile_piece(int row, int piece) { return tile_piece(row, piece); }

// Wide form.  out: rows of 8, (cta, b, h, qb, j0, j1, steps, first CTA of the unit) in the order of
// the walks.  Returns their number, grid[0] the CTAs.
long long t_wide(const int* sizes, const int* kv_len, const int* q_len, int* out, int* grid,
                 long long* all_work) {
  const PrefixArgs a = args_of(sizes, kv_len, q_len);
  std::vector<Unit> units;
  int total = 0;
  long long exact = 0;
  for (int b = 0; b < a.batch; ++b)
    for (int h = 0; h < a.heads; ++h) {
      const Lens l = lens_of(a, b);
      const int before = total;
      for (int qb = 0; qb < blocks_of(l); ++qb) {
        Unit u{};
        u.b = b;
        u.h = h;
        u.qb = qb;
        u.len = l;
        unit_set(a, u);
        u.base = total;
        total += kWorkUnit + u.steps * u.step_work;
        exact += kWorkUnit + 1ll * u.steps * u.step_work;
        units.push_back(u);
      }
      if (total - before != head_work(a, l)) return -1;
    }
  *all_work = exact;
  grid[0] = wide_ctas(a, a.ctas);
  const Cut c = cut(total, grid[0]);
  long long n = 0;
  for (int cta = 0; cta < grid[0]; ++cta) {
    Walk w{};
    w.begin = c.begin(cta);
    w.end = c.begin(cta + 1);
    w.more = w.end > w.begin;
    if (!w.more) continue;
    size_t at = 0;
    while (units[at].base + kWorkUnit + units[at].steps * units[at].step_work < w.end) ++at;
    w.u = units[at];
    w.settle(a);
    for (; w.more; w.next(a)) {
      const int row[8] = {cta, w.u.b, w.u.h, w.u.qb, w.j0, w.j1, w.u.steps, 0};
      for (int i = 0; i < 8; ++i) out[8 * n + i] = row[i];
      if (w.j1 == w.u.steps) {
        int first = first_cta(w.u, c, cta), joined = 0;
        if (w.j0 == 0) first = cta;
        for (int from = first; from < cta; ++from) joined += has_piece(w.u, c, from) ? 1 : 0;
        out[8 * n + 7] = joined;
      }
      ++n;
    }
  }
  return n;
}

// Narrow form.  dims: gt, head_groups, bt, chunks, own_units, prefix_units, CTAs used.
// out: rows of 8, (cta, index, b, in_b, j0, j1, steps, 0); slots: rows of the workspace at which
// chains 0 and 1 of the segment start, and their number.
long long t_narrow(const int* sizes, const int* kv_len, const int* q_len, int* out, long long* slots,
                   int* dims, long long* rows) {
  PrefixArgs a = args_of(sizes, kv_len, q_len);
  if (!use_narrow(a)) return -2;
  narrow_units(a);
  std::vector<NarrowUnit> units;
  int total = 0;
  for (int i = 0; i < a.prefix_units; ++i) {
    NarrowUnit u{};
    u.index = i;
    u.b = -1;
    u.steps = a.prefix_tiles;
    u.base = total;
    total += narrow_work(a, u);
    units.push_back(u);
  }
  if (total != narrow_prefix_work(a)) return -1;
  for (int b = 0; b < a.batch; ++b)
    for (int i = 0; i < a.own_units; ++i) {
      NarrowUnit u{};
      u.index = a.prefix_units + b * a.own_units + i;
      u.b = b;
      u.in_b = i;
      u.len = lens_of(a, b);
      u.steps = narrow_steps(u.len);
      u.base = total;
      if (u.steps > 0) units.push_back(u);
      total += narrow_work(a, u);
    }
  const int ctas = total > 0 ? narrow_ctas(total, a.ctas) : 0;
  const int d[7] = {a.gt, a.head_groups, a.bt, a.chunks, a.own_units, a.prefix_units, ctas};
  for (int i = 0; i < 7; ++i) dims[i] = d[i];
  *rows = static_cast<long long>(narrow_rows(a));
  long long n = 0;
  if (total == 0) return 0;
  const Cut c = cut(total, ctas);
  for (int cta = 0; cta < ctas; ++cta) {
    NarrowWalk w{};
    w.begin = c.begin(cta);
    w.end = c.begin(cta + 1);
    w.more = w.end > w.begin;
    size_t at = 0;
    while (units[at].base + narrow_work(a, units[at]) <= w.begin) ++at;
    w.u = units[at];
    w.settle(a);
    for (; w.more; w.next(a)) {
      const int row[8] = {cta, w.u.index, w.u.b, w.u.in_b, w.j0, w.j1, w.u.steps, 0};
      for (int i = 0; i < 8; ++i) out[8 * n + i] = row[i];
      const bool far = w.u.b < 0;
      slots[3 * n] = static_cast<long long>(narrow_row(a, far, w.u.index, cta, 0));
      slots[3 * n + 1] = static_cast<long long>(narrow_row(a, far, w.u.index, cta, 1));
      slots[3 * n + 2] = 1ll * a.gt * a.n_q * (far ? a.bt : 1);
      // what the join takes this unit's states to be
      const Side s = narrow_side(a, c, far, w.u.index, w.u.base, w.u.steps, 0);
      const long long i = cta - s.c0;
      if (i < 0 || 2 * i + 1 >= s.n || static_cast<long long>(s.row + i * s.step) != slots[3 * n] ||
          static_cast<long long>(s.row + i * s.step + s.chain) != slots[3 * n + 1])
        return -3;
      out[8 * n + 7] = s.n / 2;
      ++n;
    }
  }
  return n;
}

}
