"""The shared-prefix attention's tile layout and schedules, enumerated on the host by the functions
its kernels run (csrc/prefix_sched.h, compiled here with the C++ compiler), against what the
kernels rely on: every step of every unit is one CTA's; a unit's steps lie in consecutive CTAs; of
the wide form a CTA leaves one state at most, the first of its walk, and the CTA of a unit's last
step joins exactly those of the unit's other CTAs; of the narrow form no two states share rows of
the workspace and the join reads exactly those that were written.  No GPU."""
import collections
import ctypes
import os
import random
import subprocess

import pytest

from video_diffusion_transformer_03_b200 import build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("prefix") / "sched.so")
    cuda = os.path.join(os.path.dirname(os.path.dirname(build.nvcc())), "include")
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", build.CSRC, "-I", cuda,
                    os.path.join(HERE, "prefix_schedule.cpp"), "-o", so], check=True)
    lib = ctypes.CDLL(so)
    lib.t_wide.restype = lib.t_narrow.restype = ctypes.c_longlong
    return lib


@pytest.mark.parametrize("head_dim", [64, 128])
def test_staged_rows_stay_in_their_warp_of_the_weights(lib, head_dim):
    """A warp stages its 32 output rows over its own rows of the weights' tile, no others: nothing
    orders the four warps of a tile between a unit's end and the next one's first weights."""
    weights = [{lib.t_tile_piece(r, p) for r in range(32 * w, 32 * w + 32) for p in range(16)}
               for w in range(4)]
    staged = [{lib.t_tile_piece(r, p) for r in range(32 * w, 32 * w + 32)
               for p in range(head_dim // 8)} for w in range(4)]
    assert set().union(*weights) == set(range(2048)) and all(len(s) == 512 for s in weights)
    for w in range(4):
        assert len(staged[w]) == 32 * head_dim // 8 and staged[w] <= weights[w]
    # rows laid end to end, a head's width apart, would not do for heads of 128
    ends = [{r * (head_dim // 8) + p for r in range(32 * w, 32 * w + 32)
             for p in range(head_dim // 8)} for w in range(4)]
    assert all(e <= x for e, x in zip(ends, weights)) == (head_dim == 64)


def test_tile_layout_is_the_swizzle_of_128_bytes(lib):
    # 16-byte pieces of a 128-byte row, exclusive-or-ed with the row modulo 8; boxes of 128 rows
    for row in range(128):
        for piece in range(16):
            byte = (piece // 8) * 128 * 128 + row * 128 + (((piece % 8) ^ (row % 8)) * 16)
            assert lib.t_tile_piece(row, piece) * 16 == byte


# ------------------------------------------------------------------------------- schedules
def ints(x):
    return None if x is None else (ctypes.c_int * len(x))(*x)


def case(rng, batch, n_q, n_prefix, n_kv):
    """Sizes as the C functions take them, and lengths (some out of range, as a caller's may be)."""
    kv = rng.randint(1, 6)
    group = rng.randint(1, 7)
    if n_prefix == 0 and n_kv == 0:
        n_kv = 1
    sms = rng.choice((148, 148, 132, 160, rng.randint(1, 20)))
    sizes = [batch, n_q, kv * group, kv, n_prefix, n_kv, rng.randint(0, 1), sms]

    def lens(top):
        if rng.random() < 0.25:
            return None
        pool = [rng.randint(-1, top + 2), rng.randint(0, top), 0, 1, top]
        return [rng.choice(pool + [rng.randint(0, top)]) for _ in range(batch)]
    return sizes, lens(n_kv), lens(n_q)


def clamped(x, top, batch):
    return [top] * batch if x is None else [min(max(v, 0), top) for v in x]


def wide_cases():
    rng = random.Random(11)
    for i in range(300):
        n_q = rng.choice((rng.randint(1, 300), rng.randint(65, 2000), 128, 129, 256, 257))
        yield case(rng, rng.randint(1, rng.choice((2, 9, 70))), n_q, rng.choice((0, 1, 128, rng.randint(1, 5000))),
                   rng.choice((0, 1, 129, rng.randint(1, 3000))))
    # the clips of the tests and of the benchmark's file: more units than SMs
    yield [6, 1600, 24, 24, 1024, 1600, 0, 148], [1600, 1460, 1320, 1180, 1040, 900], [1600, 1460, 1320, 1180, 1040, 900]
    yield [6, 300, 24, 24, 130, 300, 1, 148], [300, 20, 0, 5, 7, 299], [300, 128, 70, 257, 0, 1]


def test_wide_schedule(lib):
    went_on = 0
    for sizes, kv_len, q_len in wide_cases():
        batch, n_q, heads, _, n_prefix, n_kv, causal, sms = sizes
        kv, q = clamped(kv_len, n_kv, batch), clamped(q_len, n_q, batch)
        want = {}
        for b in range(batch):
            for qb in range(-(-q[b] // 256)):
                # keys that the block's last query sees
                own = min(kv[b], min(q[b], 256 * qb + 256) + kv[b] - q[b]) if causal else kv[b]
                steps = max(1, -(-n_prefix // 128) + -(-max(own, 0) // 128))
                for h in range(heads):
                    want[b, h, qb] = steps
        out = (ctypes.c_int * (8 * (sum(want.values()) + 1)))()
        grid, work = (ctypes.c_int * 1)(), (ctypes.c_longlong * 1)()
        n = lib.t_wide(ints(sizes), ints(kv_len), ints(q_len), out, grid, work)
        assert n >= 0 and 0 <= grid[0] <= sms and work[0] < 2 ** 30
        parts, joined, walks = collections.defaultdict(list), {}, collections.defaultdict(list)
        for i in range(n):
            cta, b, h, qb, j0, j1, steps, join = out[8 * i:8 * i + 8]
            assert steps == want[b, h, qb] and 0 <= j0 < j1 <= steps
            parts[b, h, qb].append((j0, j1, cta))
            walks[cta].append(j1 == steps)
            if j1 == steps:
                assert (b, h, qb) not in joined
                joined[b, h, qb] = join
        assert set(parts) == set(want)
        for unit, steps in want.items():
            at = 0
            for j0, j1, cta in sorted(parts[unit]):
                assert j0 == at
                at = j1
            assert at == steps and joined[unit] == len(parts[unit]) - 1
            ctas = [p[2] for p in sorted(parts[unit])]
            assert ctas == sorted(set(ctas))
        for ends in walks.values():
            assert all(ends[1:])                       # only the first may leave a state
        went_on = max(went_on, max((len(e) for e in walks.values()), default=0))
    assert went_on > 3


def narrow_cases():
    rng = random.Random(12)
    for i in range(300):
        n_q = rng.choice((1, 1, rng.randint(1, 8), rng.randint(1, 64)))
        yield case(rng, rng.randint(1, rng.choice((3, 40, 200))), n_q, rng.choice((0, 1, 129, rng.randint(1, 16000))),
                   rng.choice((0, 1, 128, rng.randint(1, 4000))))


def test_narrow_schedule(lib):
    for sizes, kv_len, q_len in narrow_cases():
        batch, n_q, heads, kv_heads, n_prefix, n_kv, _, sms = sizes
        kv, q = clamped(kv_len, n_kv, batch), clamped(q_len, n_q, batch)
        most = 8 * (heads * batch * (n_prefix // 128 + n_kv // 128 + 4) + 400)
        out, slots = (ctypes.c_int * most)(), (ctypes.c_longlong * most)()
        dims, rows = (ctypes.c_int * 7)(), (ctypes.c_longlong * 1)()
        n = lib.t_narrow(ints(sizes), ints(kv_len), ints(q_len), out, slots, dims, rows)
        assert n >= 0, n
        gt, head_groups, bt, chunks, own_units, prefix_units, ctas = dims
        group = heads // kv_heads
        # rows: sequences, heads and queries of a unit fit a tile and cover all of them
        assert 1 <= gt * n_q * bt <= 128 and gt * head_groups >= group and bt * chunks >= batch
        assert own_units == kv_heads * head_groups and ctas <= sms
        assert prefix_units == (own_units * chunks if n_prefix else 0)
        want = {i: -(-n_prefix // 128) for i in range(prefix_units)}
        for b in range(batch):
            if q[b] and kv[b]:
                for i in range(own_units):
                    want[prefix_units + b * own_units + i] = -(-kv[b] // 128)
        parts, taken = collections.defaultdict(list), []
        for i in range(n):
            cta, index, b, in_b, j0, j1, steps, states = out[8 * i:8 * i + 8]
            assert 0 <= j0 < j1 <= steps == want[index]
            assert (b == -1) == (index < prefix_units)
            if b >= 0:
                assert index == prefix_units + b * own_units + in_b
            parts[index].append((j0, j1, cta, states))
            r0, r1, count = slots[3 * i:3 * i + 3]
            taken += [(r0, r0 + count), (r1, r1 + count)]
        assert set(parts) == set(want)
        for index, steps in want.items():
            at, first = 0, parts[index][0][2]
            for i, (j0, j1, cta, states) in enumerate(parts[index]):
                # consecutive CTAs, as many as the join takes them to be
                assert j0 == at and cta == first + i and states == len(parts[index])
                at = j1
            assert at == steps
        taken.sort()
        assert all(a[1] <= b[0] for a, b in zip(taken, taken[1:]))
        assert not taken or (taken[0][0] >= 0 and taken[-1][1] <= rows[0])
