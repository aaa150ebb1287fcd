"""Infinities, NaN and signed zeros in the channels that the rotation passes through: they stay
in their channel, as in the formulas (oracle/heads.py)."""
import numpy as np
import pytest
import torch

from oracle import heads as OH
from tests.helpers import np64, rnd
from tests.test_gpu_heads import BF, DEV, EPS, F32, HF, h3b, positions

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
# head_dim, split: whole lanes pass, a lane is turned in part, an odd count of pairs in a head
WIDTHS = [(128, (16, 16)), (64, (6, 4)), (96, (2,)), (8, (2,)), (256, (16, 24, 24))]


def same(got, want):
    """Equal values, signed zeros and infinities included; NaN where the other has one."""
    got, want = np64(got), np64(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), np.argwhere(np.isnan(got) != np.isnan(want))[:4]
    ok = np.isnan(want) | ((got == want) & (np.signbit(got) == np.signbit(want)))
    assert ok.all(), np.argwhere(~ok)[:4]


def setup(hd, split, halves, dtype):
    if halves and sum(split) % 8:
        pytest.skip("half-split pairs need a width that is a multiple of 8")
    t, h = 5, 3
    x = rnd((t, h, hd), 1.0, seed=1, dtype=dtype)
    return h3b.make_rope_axes(split, pairing=int(halves)), positions(1, t, len(split))[0], x, sum(split)


@pytest.mark.parametrize("dtype", [BF, HF, F32], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("halves", [False, True], ids=["adjacent", "halves"])
@pytest.mark.parametrize("hd,split", WIDTHS)
def test_rotation_passes_channels_through(hd, split, halves, dtype):
    plan, pos, x, rot = setup(hd, split, halves, dtype)
    x[0, 0, rot] = INF
    x[1, 1, hd - 1] = NAN
    x[2, :, rot] = -0.0
    x[2, :, rot + 1] = -1.0
    x[3, 2, rot:] = torch.finfo(dtype).min
    for inverse in (False, True):
        out = torch.empty_like(x, device=DEV)
        h3b.rope_axes(plan, x.to(DEV), pos.to(DEV), out, inverse=inverse)
        h3b.sync_status()
        same(out[..., rot:], x[..., rot:])
        assert torch.isfinite(out[..., :rot]).all()


@pytest.mark.parametrize("dtype", [BF, HF, F32], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("halves", [False, True], ids=["adjacent", "halves"])
@pytest.mark.parametrize("hd,split", WIDTHS + [(128, None), (72, None)])
def test_norm_and_its_gradients_mix_turned_channels_only(hd, split, halves, dtype):
    if split is None and halves:
        pytest.skip("no rotation")
    plan, pos, x, rot = setup(hd, split or (2,), halves, dtype)
    if split is None:
        plan, pos, rot = None, None, 0
    kw = {} if plan is None else dict(pos=np64(pos), split=split, halves=halves)
    gain = 1.0 + rnd((hd,), 0.1, seed=3, dtype=F32)
    pd = None if pos is None else pos.to(DEV)
    # an infinite channel: it becomes NaN, its head's others 0
    y = x.clone()
    y[1, 1, rot + 1] = INF
    out = torch.empty_like(y, device=DEV)
    h3b.qk_norm_rope(plan, y.to(DEV), None, gain.to(DEV), None, EPS, pd, out, None)
    h3b.sync_status()
    with np.errstate(invalid="ignore"):
        want = OH.norm_rope(np64(y), np64(gain), EPS, **kw)
    assert np.array_equal(np.isnan(np64(out)), np.isnan(want))
    # an infinite gradient of one: its gain's gradient is, the others' are not
    g = rnd(tuple(x.shape), 1.0, seed=4, dtype=dtype)
    g[1, 1, rot + 1] = INF
    dx, dg = torch.empty_like(x, device=DEV), torch.empty(hd, device=DEV)
    h3b.qk_norm_rope_backward(plan, x.to(DEV), None, gain.to(DEV), None, EPS, pd, g.to(DEV), None, dx,
                              None, dg, None,
                              h3b.workspace(h3b.qk_norm_rope_backward_workspace_size(hd)))
    h3b.sync_status()
    with np.errstate(invalid="ignore"):
        _, want = OH.norm_rope_backward(np64(x), np64(gain), EPS, np64(g), **kw)
    finite = np.ones(hd, bool)
    finite[rot + 1] = False
    assert np.array_equal(np.isfinite(want), finite)
    assert np.array_equal(np.isfinite(np64(dg)), finite)
