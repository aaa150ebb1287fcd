"""The operators on heads without a GPU: the oracle against closed forms and differences, the
plan of the axes, and the refusals of the C entry points (nothing is launched)."""
import ctypes
import math

import numpy as np
import pytest

from oracle import heads as OH
from oracle import oracle as O
from video_diffusion_transformer_03_b200 import h3b

L = h3b.lib
P = 4096                       # aligned, never dereferenced: the checks come first


def refused(rc, word):
    assert rc == h3b.H3B_EINVAL and word in L.h3b_last_error().decode(), L.h3b_last_error()


# ------------------------------------------------------------------------------- oracle
def test_oracle_rotation_is_the_grid_rotation():
    # two separately written rotations: that of the block (adjacent pairs, three axes) and this
    split, n = (4, 6, 6), 7
    rng = np.random.default_rng(0)
    x = rng.standard_normal((n, 2, 16))
    pos = rng.integers(0, 9, (n, 3)).astype(float)
    assert np.allclose(OH.rope_axes(x, pos, split), O.rope_rotate(x, pos, split, 10000.0))


@pytest.mark.parametrize("halves", [False, True])
def test_oracle_rotation_turns_back_and_depends_on_differences(halves):
    split = (8, 8)
    rng = np.random.default_rng(1)
    x, y = rng.standard_normal((2, 5, 3, 24))
    pos = rng.integers(0, 50, (5, 2)).astype(float)
    kw = dict(halves=halves, shared_freq=halves)
    turned = OH.rope_axes(x, pos, split, **kw)
    assert np.allclose(OH.rope_axes(turned, pos, split, inverse=True, **kw), x)
    assert np.array_equal(turned[..., 16:], x[..., 16:])
    moved = [OH.rope_axes(t, pos + 13.0, split, **kw) for t in (x, y)]
    assert np.allclose((turned * OH.rope_axes(y, pos, split, **kw)).sum(-1),
                       (moved[0] * moved[1]).sum(-1))


def test_oracle_gradients_against_differences():
    rng = np.random.default_rng(2)
    x, g = rng.standard_normal((2, 2, 3, 2, 16))
    gain = 1 + 0.1 * rng.standard_normal(16)
    pos = rng.integers(0, 9, (3, 2)).astype(float)
    kw = dict(pos=pos, split=(8, 8), halves=True)

    def loss(xv, gv):
        return (OH.norm_rope(xv, gv, 1e-6, **kw) * g).sum()

    dx, dg = OH.norm_rope_backward(x, gain, 1e-6, g, **kw)
    e = 1e-6
    for _ in range(5):
        u, v = rng.standard_normal(x.shape), rng.standard_normal(16)
        slope = (loss(x + e * u, gain + e * v) - loss(x - e * u, gain - e * v)) / (2 * e)
        assert abs(slope - (dx * u).sum() - (dg * v).sum()) < 1e-7


def test_oracle_shared_prefix_is_attention_over_the_joined_keys():
    rng = np.random.default_rng(3)
    q = rng.standard_normal((2, 5, 4, 8))
    kp, vp = rng.standard_normal((2, 3, 2, 8))
    k, v = rng.standard_normal((2, 2, 6, 2, 8))
    out = OH.attention_prefix(q, kp, vp, k, v, kv_len=[6, 2], q_len=[5, 3])
    s = q[1, 2, 3] @ np.concatenate((kp[:, 1], k[1, :2, 1])).T / math.sqrt(8)
    p = np.exp(s) / np.exp(s).sum()
    assert np.allclose(out[1, 2, 3], p @ np.concatenate((vp[:, 1], v[1, :2, 1])))
    assert np.isnan(out[1, 3:]).all() and np.isfinite(out[0]).all()
    # causal: query i of 5 sees the prefix and own keys 0 .. 1 + i of 6; without keys: zero
    causal = OH.attention_prefix(q, kp, vp, k, v, causal=True)
    one = OH.attention_prefix(q[:, 2:3], kp, vp, k[:, :4], v[:, :4])
    assert np.allclose(causal[:, 2], one[:, 0])
    none = OH.attention_prefix(q, kp[:0], vp[:0], k, v, kv_len=[0, 3], causal=True)
    assert not none[0].any() and not none[1, :2].any() and none[1, 2:].any()


# ------------------------------------------------------------------------------- plan
def test_plan_holds_the_ladder():
    for split, halves, shared in (((16, 24, 24), 0, False), ((32, 48, 48), 1, True), ((6, 0, 4), 0, False)):
        plan = h3b.make_rope_axes(split, theta=10000.0, pairing=halves, shared_freq=shared)
        axis, freq = OH.ladder(split, 10000.0, shared)
        n = len(axis)
        assert plan.n_pairs == n and plan.n_axes == len(split) and plan.pairing == halves
        assert list(plan.axis[:n]) == list(axis)
        assert np.allclose(np.array(plan.turns[:n]) * 2 * math.pi, freq, rtol=1e-15)


@pytest.mark.parametrize("split,theta,pairing,word", [
    ((), 1e4, 0, "n_axes"), ((2,) * 5, 1e4, 0, "n_axes"), ((3, 5), 1e4, 0, "split"),
    ((-2, 4), 1e4, 0, "split"), ((258,), 1e4, 0, "split"), ((0, 0), 1e4, 0, "width"),
    ((200, 200), 1e4, 0, "width"), ((6, 6), 1e4, 1, "half-split"), ((8,), 0.0, 0, "theta"),
    ((8,), float("nan"), 0, "theta"), ((8,), float("inf"), 0, "theta"), ((8,), 1e4, 2, "pairing")])
def test_plan_refusals(split, theta, pairing, word):
    with pytest.raises(h3b.H3BError, match=word):
        h3b.make_rope_axes(split, theta=theta, pairing=pairing)


# ------------------------------------------------------------------------------- refusals
def hv(ptr=P, b=8192, t=512, h=128):
    return h3b.HeadView(ptr, b, t, h)


def rope(plan="ok", dtype=0, x=None, batch=2, tokens=16, heads=4, hd=128, pos=P, ps=0, out=None):
    plan = h3b.make_rope_axes((32, 48, 48)) if plan == "ok" else plan
    return L.h3b_rope_axes(plan, dtype, x or hv(), batch, tokens, heads, hd, pos, ps, 0, out or hv(),
                           None)


def test_rope_axes_refusals():
    refused(rope(plan=None), "plan is NULL")
    refused(rope(plan=h3b.RopePlan()), "not made by")
    odd = h3b.make_rope_axes((16, 16), pairing=h3b.ROPE_HALVES)
    odd.n_pairs = 6
    refused(rope(plan=odd), "not made by")
    refused(rope(dtype=3), "dtype")
    refused(rope(batch=-1), "sizes")
    refused(rope(tokens=-1), "sizes")
    refused(rope(heads=-1), "sizes")
    refused(rope(hd=132), "head_dim")
    refused(rope(hd=264), "head_dim")
    refused(rope(hd=0), "head_dim")
    refused(rope(hd=64), "rotates 128 channels")
    refused(rope(pos=None), "pos")
    refused(rope(pos=P + 2), "pos")
    refused(rope(ps=-3), "pos_batch_stride")
    refused(rope(x=hv(ptr=None)), "x is NULL")
    refused(rope(x=hv(ptr=P + 8)), "x is NULL or not 16-byte aligned")
    refused(rope(x=hv(t=516)), "x: stride 516")
    refused(rope(x=hv(h=-128)), "x: stride -128")
    refused(rope(out=hv(b=0)), "out has stride 0")
    refused(rope(dtype=2, out=hv(t=514)), "out: stride 514")


def norm(plan=None, dtype=0, q=None, k=None, batch=2, tokens=16, nq=4, nk=4, hd=128, qg=P, kg=P,
         eps=1e-6, qo=None, ko=None):
    return L.h3b_qk_norm_rope(plan, dtype, q or hv(), k or hv(), batch, tokens, nq, nk, hd, qg, kg,
                              eps, None, 0, qo or hv(), ko or hv(), None)


def test_qk_norm_rope_refusals():
    refused(norm(eps=0.0), "eps")
    refused(norm(eps=float("nan")), "eps")
    refused(norm(qg=P + 1), "gains")
    refused(norm(nk=-1), "sizes")
    refused(norm(k=hv(ptr=None)), "k is NULL")
    refused(norm(qo=hv(h=0)), "q_out has stride 0")
    refused(norm(ko=hv(ptr=P + 4)), "k_out is NULL")
    refused(norm(plan=h3b.make_rope_axes((128,))), "pos")


def test_qk_norm_rope_backward_refusals():
    need = h3b.qk_norm_rope_backward_workspace_size(128)

    def back(g=None, d=None, dqg=P, ws=P, nbytes=need, hd=128):
        return L.h3b_qk_norm_rope_backward(None, 0, hv(), hv(), 2, 16, 4, 4, hd, P, P, 1e-6, None, 0,
                                           g or hv(), hv(), d or hv(), hv(), dqg, P, ws, nbytes, None)

    refused(back(g=hv(ptr=None)), "g_q is NULL")
    refused(back(d=hv(t=0)), "dq has stride 0")
    refused(back(dqg=P + 2), "gain gradient")
    for ws, nbytes in ((None, need), (P + 8, need), (P, need - 1)):
        assert back(ws=ws, nbytes=nbytes) == h3b.H3B_EWORKSPACE
    for hd in (0, 12, 264):
        with pytest.raises(h3b.H3BError, match="head_dim"):
            h3b.qk_norm_rope_backward_workspace_size(hd)


def attend(dtype=0, q=None, kp=None, k=None, batch=2, nq=3, heads=4, kv=2, hd=64, prefix=16, nkv=8,
           kv_len=None, q_len=None, scale=0.0, out=None, ws=P, nbytes=1 << 40):
    return L.h3b_attention_prefix(dtype, q or hv(), kp or hv(), hv(), k or hv(), hv(), batch, nq, heads,
                                  kv, hd, prefix, nkv, kv_len, q_len, 0, scale, out or hv(), ws, nbytes,
                                  None)


def test_attention_prefix_refusals():
    refused(attend(dtype=2), "dtype")
    refused(attend(dtype=7), "dtype")
    for kw in (dict(batch=-1), dict(nq=-1), dict(prefix=-1), dict(nkv=-1), dict(batch=1 << 20)):
        refused(attend(**kw), "sizes")
    refused(attend(prefix=0, nkv=0), "no keys")
    for kw in (dict(heads=3), dict(heads=0), dict(kv=0), dict(kv=8)):
        refused(attend(**kw), "n_heads")
    refused(attend(hd=96), "head_dim")
    for s in (-0.5, float("nan"), float("inf")):
        refused(attend(scale=s), "scale")
    refused(attend(q=hv(ptr=None)), "q is NULL")
    refused(attend(kp=hv(ptr=P + 2)), "k_prefix is NULL")
    refused(attend(k=hv(t=0)), "k has stride 0")
    refused(attend(k=hv(h=60)), "k: stride 60")
    refused(attend(out=hv(b=0)), "out has stride 0")
    refused(attend(kv_len=P + 1), "lengths")
    refused(attend(q_len=P + 2), "lengths")
    need = h3b.attention_prefix_workspace_size(2, 3, 4, 2, 64, 16, 8)
    for ws, nbytes in ((None, need), (P + 8, need), (P, need - 1)):
        assert attend(ws=ws, nbytes=nbytes) == h3b.H3B_EWORKSPACE
    with pytest.raises(h3b.H3BError, match="n_heads"):
        h3b.attention_prefix_workspace_size(2, 3, 4, 3, 64, 16, 8)


def test_attention_prefix_refuses_more_work_than_it_counts():
    # 10^9 tiles: the size query and the call say so
    assert h3b.lib.h3b_attention_prefix_workspace_size(1000, 4096, 64, 64, 64, 1 << 25, 0) == 0
    assert "too much work" in h3b.lib.h3b_last_error().decode()
    with pytest.raises(h3b.H3BError, match="too much work"):
        h3b.attention_prefix_workspace_size(60000, 1, 64, 1, 128, 1 << 28, 1 << 20)
    with pytest.raises(h3b.H3BError, match="too much work"):
        h3b.attention_prefix_workspace_size(65535, 1 << 24, 65536, 65536, 64, 1 << 28, 1 << 28)
    assert h3b.attention_prefix_workspace_size(60000, 1, 64, 1, 128, 1000, 1000) > 0
