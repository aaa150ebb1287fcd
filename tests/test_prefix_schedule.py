"""The shared-prefix attention's tile layout, enumerated on the host by the functions its kernels
run (csrc/prefix_sched.h, compiled here with the C++ compiler).  No GPU."""
import ctypes
import os
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
    return ctypes.CDLL(so)


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
