"""Rotary positions with several axes and the Q/K RMS norm with that rotation, forward and
backward, through the binding, against the float64 oracle (oracle/heads.py).

Tolerances count roundings.  The kernels work in 32 bits and round once at the store:
  * sin, cos: the remainder of the angle in revolutions is rounded once (2^-24 of at most half
    a turn: 1.9e-7 of angle) and sincospif adds at most 2 ulp (1.2e-7 each): below 3.5e-7; the
    two products and the sum of a turned pair add 2^-23 of |a| + |b|.  TURN = 5e-7 covers both.
  * the norm: the sum of at most 256 squares has at most 13 additions in a row (13 * 2^-24,
    half of it in the root), rsqrtf 2 ulp, two products: below 14 * 2^-24.  NORM = 1e-6.
  * the store: half a step of the type, relative, and half its smallest step absolute.
"""
import numpy as np
import pytest
import torch

from oracle import heads as OH
from tests.helpers import np64, rnd

pytestmark = pytest.mark.gpu

h3b = pytest.importorskip("video_diffusion_transformer_03_b200.h3b")

DEV = "cuda"
EPS = 1e-6
TURN, NORM = 5e-7, 1e-6
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def stored(want, err, dtype):
    """Bound on |got - want| after the store, from the bound before it."""
    fi = torch.finfo(dtype)
    return err + fi.eps / 2 * (np.abs(want) + err) + fi.smallest_normal * fi.eps / 2


def within(got, want, tol):
    got = np64(got) if torch.is_tensor(got) else got
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), float(np.nanmax(np.abs(got - want) / tol)))


def pair_sum(x, split, halves):
    """|a| + |b| of the pair every channel belongs to (|x| itself where it is not turned)."""
    n, x = sum(split) // 2, np.abs(x)
    ia = np.arange(n) if halves else 2 * np.arange(n)
    ib = ia + (n if halves else 1)
    s = x.copy()
    s[..., ia] = s[..., ib] = x[..., ia] + x[..., ib]
    return s


def positions(batch, tokens, axes, seed=5, far=0.0):
    g = torch.Generator().manual_seed(seed)
    pos = torch.randint(0, 60, (batch, tokens, axes), generator=g).float()
    pos[..., 0] += far
    pos[..., -1] += 0.5
    return pos


def view(batch, tokens, heads, hd, dtype, seed, layout):
    """The same values in different memory: dense, the q columns of a packed buffer, or
    head-major."""
    x = rnd((batch, tokens, heads, hd), 1.0, seed=seed, dtype=dtype)
    if layout == "packed":
        buf = torch.full((batch, tokens, heads + 3, hd), float("nan"), dtype=dtype, device=DEV)
        buf[:, :, 1:1 + heads] = x.to(DEV)
        return x, buf[:, :, 1:1 + heads]
    if layout == "heads_first":
        return x, x.to(DEV).transpose(1, 2).contiguous().transpose(1, 2)
    return x, x.to(DEV)


# batch, tokens, heads, kv heads, head_dim, split
SHAPES = [(1, 1, 1, 1, 8, (2,)), (2, 7, 3, 1, 64, (16, 24, 24)), (1, 40, 24, 8, 128, (32, 48, 48)),
          (3, 33, 5, 5, 96, (32, 32, 32)), (2, 9, 2, 2, 256, (64, 96, 96)),
          (1, 130, 9, 3, 128, (16, 16)), (1, 19, 2, 1, 80, (8, 24, 24, 8)),
          (2, 1601, 3, 1, 64, (8, 16))]     # the last: tokens enough that heads are not dealt out
FORMS = [(BF, False, False, "packed"), (BF, True, True, "dense"), (HF, False, True, "heads_first"),
         (HF, True, False, "packed"), (F32, False, False, "dense"), (F32, True, False, "packed")]


def usable(split, halves):
    return not halves or sum(split) % 8 == 0


@pytest.mark.parametrize("dtype,halves,shared,layout", FORMS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_rope_axes(shape, dtype, halves, shared, layout):
    b, t, h, _, hd, split = shape
    if not usable(split, halves):
        pytest.skip("half-split pairs need a width that is a multiple of 8")
    plan = h3b.make_rope_axes(split, pairing=int(halves), shared_freq=shared)
    x, xd = view(b, t, h, hd, dtype, 1, layout)
    for far, per_sample, inverse in ((0.0, True, False), (1e5, False, True)):
        pos = positions(b if per_sample else 1, t, len(split), far=far)
        want = OH.rope_axes(np64(x), np64(pos), split, halves=halves, shared_freq=shared,
                            inverse=inverse)
        out = torch.full((b, t, h, hd), float("nan"), dtype=dtype, device=DEV)
        h3b.rope_axes(plan, xd, pos.to(DEV) if per_sample else pos[0].to(DEV), out, inverse=inverse)
        h3b.sync_status()
        within(out, want, stored(want, TURN * pair_sum(np64(x), split, halves), dtype))


@pytest.mark.parametrize("dtype,halves,shared,layout", FORMS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_qk_norm_rope(shape, dtype, halves, shared, layout):
    b, t, h, kv, hd, split = shape
    if not usable(split, halves):
        pytest.skip("half-split pairs need a width that is a multiple of 8")
    plan = h3b.make_rope_axes(split, pairing=int(halves), shared_freq=shared)
    pos = positions(b, t, len(split), far=3e4)
    got = {}
    x, gain = {}, {}
    for name, heads, seed in (("q", h, 1), ("k", kv, 2)):
        x[name], xd = view(b, t, heads, hd, dtype, seed, layout)
        gain[name] = 1.0 + rnd((hd,), 0.1, seed=seed + 10, dtype=F32)
        got[name] = (xd, gain[name].to(DEV),
                     torch.full((b, t, heads, hd), float("nan"), dtype=dtype, device=DEV))
    h3b.qk_norm_rope(plan, got["q"][0], got["k"][0], got["q"][1], got["k"][1], EPS, pos.to(DEV),
                     got["q"][2], got["k"][2])
    h3b.sync_status()
    for name in ("q", "k"):
        n = OH.norm_rope(np64(x[name]), np64(gain[name]), EPS)
        want = OH.rope_axes(n, np64(pos), split, halves=halves, shared_freq=shared)
        within(got[name][2], want,
               stored(want, (TURN + NORM) * pair_sum(n, split, halves), dtype))


def backward_bounds(x, gain, g, pos, split, **kw):
    """Oracle gradients and bounds on their 32-bit errors (before the store)."""
    halves = kw.get("halves", False)
    dx, dgain = OH.norm_rope_backward(x, gain, EPS, g, pos, split, **kw)
    z = g if split is None else OH.rope_axes(g, pos, split, inverse=True, **kw)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + EPS)
    n, w = x * r, z * gain
    ez = TURN * (np.abs(g) if split is None else pair_sum(g, split, halves))
    ew = np.abs(gain) * ez + 2 ** -23 * np.abs(w)
    # mean(w n): its terms' errors, n's (NORM), and at most 13 additions in a row
    edot = (ew * np.abs(n) + (NORM + 14 * 2 ** -24) * np.abs(w * n)).mean(-1, keepdims=True)
    dot = np.abs((w * n).mean(-1, keepdims=True))
    ex = r * (ew + np.abs(n) * edot + (2 * NORM + 2 ** -22) * (np.abs(w) + np.abs(n) * dot))
    # the sum over tokens and heads: no lane adds more than 256 terms here, no reduction after
    # it has more than 64 additions in a row
    zn = np.abs(z * n)
    eg = (ez * np.abs(n) + (NORM + 2 ** -23 + 320 * 2 ** -24) * zn)
    return dx, ex, dgain, eg.reshape(-1, x.shape[-1]).sum(0)


@pytest.mark.parametrize("dtype,halves,shared,layout", FORMS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_qk_norm_rope_backward(shape, dtype, halves, shared, layout):
    b, t, h, kv, hd, split = shape
    if not usable(split, halves):
        pytest.skip("half-split pairs need a width that is a multiple of 8")
    plan = h3b.make_rope_axes(split, pairing=int(halves), shared_freq=shared)
    pos = positions(1, t, len(split))[0]
    ws = h3b.workspace(h3b.qk_norm_rope_backward_workspace_size(hd))
    ws.fill_(255)                            # NaN
    x, g, gain, d = {}, {}, {}, {}
    for name, heads, seed in (("q", h, 1), ("k", kv, 2)):
        x[name], xd = view(b, t, heads, hd, dtype, seed, layout)
        g[name], gd = view(b, t, heads, hd, dtype, seed + 4, layout)
        gain[name] = 1.0 + rnd((hd,), 0.1, seed=seed + 10, dtype=F32)
        d[name] = (xd, gain[name].to(DEV), gd, torch.full_like(xd, float("nan")),
                   torch.full((hd,), float("nan"), device=DEV))
    q, k = d["q"], d["k"]

    def call():
        h3b.qk_norm_rope_backward(plan, q[0], k[0], q[1], k[1], EPS, pos.to(DEV), q[2], k[2], q[3],
                                  k[3], q[4], k[4], ws)
        h3b.sync_status()

    call()
    first = [t.clone() for t in (q[3], k[3], q[4], k[4])]
    for name in ("q", "k"):
        dx, ex, dgain, eg = backward_bounds(np64(x[name]), np64(gain[name]), np64(g[name]),
                                            np64(pos), split, halves=halves, shared_freq=shared)
        within(d[name][3], dx, stored(dx, ex, dtype))
        within(d[name][4], dgain, eg)
    call()
    assert all(torch.equal(a, c) for a, c in zip(first, (q[3], k[3], q[4], k[4])))


def test_backward_against_differences():
    # the gradients against central differences of the oracle's forward, along random directions
    split, b, t, h, hd = (16, 24, 24), 2, 5, 3, 64
    plan = h3b.make_rope_axes(split)
    pos = positions(b, t, 3)
    x, g = (rnd((b, t, h, hd), 1.0, seed=s, dtype=F32) for s in (1, 2))
    gain = 1.0 + rnd((hd,), 0.1, seed=3, dtype=F32)
    dx, dgain = torch.empty_like(x, device=DEV), torch.empty(hd, device=DEV)
    h3b.qk_norm_rope_backward(plan, x.to(DEV), None, gain.to(DEV), None, EPS, pos.to(DEV),
                              g.to(DEV), None, dx, None, dgain, None,
                              h3b.workspace(h3b.qk_norm_rope_backward_workspace_size(hd)))
    h3b.sync_status()

    def loss(xv, gv):
        return (OH.norm_rope(xv, gv, EPS, np64(pos), split) * np64(g)).sum()

    rng = np.random.default_rng(0)
    for _ in range(4):
        u, v, e = rng.standard_normal(x.shape), rng.standard_normal(hd), 1e-5
        slope = (loss(np64(x) + e * u, np64(gain) + e * v)
                 - loss(np64(x) - e * u, np64(gain) - e * v)) / (2 * e)
        got = (np64(dx) * u).sum() + (np64(dgain) * v).sum()
        size = np.abs(np64(dx) * u).sum() + np.abs(np64(dgain) * v).sum()
        # 32-bit gradients: 4e-6 of the sum of magnitudes; differences: e^2 and 2^-53 / e
        assert abs(got - slope) <= 4e-6 * size + 1e-7 * size


def test_in_place_and_broadcast_inputs():
    split, b, t, h, hd = (32, 48, 48), 3, 21, 4, 128
    plan = h3b.make_rope_axes(split, pairing=h3b.ROPE_HALVES)
    pos = positions(1, t, 3)[0].to(DEV)
    one = rnd((1, t, h, hd), 1.0, seed=1).to(DEV)
    x = one.expand(b, t, h, hd)                       # stride 0 over the batch
    out = torch.empty(b, t, h, hd, dtype=BF, device=DEV)
    h3b.rope_axes(plan, x, pos, out)
    same = one.clone()
    h3b.rope_axes(plan, same, pos, same)              # in place
    assert torch.equal(out, same.expand_as(out))
    # positions expanded over the batch equal shared ones
    again = torch.empty_like(out)
    h3b.rope_axes(plan, x, pos[None].expand(b, t, 3), again)
    assert torch.equal(out, again)
    # [tokens, heads, head_dim]
    flat = torch.empty_like(one[0])
    h3b.rope_axes(plan, one[0], pos, flat)
    assert torch.equal(flat, same[0])
    # the norm in place, inside a packed buffer whose other columns stay
    buf = rnd((b, t, 3 * h, hd), 1.0, seed=2).to(DEV)
    kept = buf.clone()
    q, k = buf[:, :, :h], buf[:, :, h:2 * h]
    gain = torch.ones(hd, device=DEV)
    qo, ko = torch.empty_like(out), torch.empty_like(out)
    h3b.qk_norm_rope(plan, q, k, gain, None, EPS, pos, qo, ko)
    h3b.qk_norm_rope(plan, q, k, None, gain, EPS, pos, q, k)
    assert torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(buf[:, :, 2 * h:], kept[:, :, 2 * h:])
    # gradients written over g
    g = rnd((b, t, h, hd), 1.0, seed=4).to(DEV)
    ws = h3b.workspace(h3b.qk_norm_rope_backward_workspace_size(hd))
    d, dg = torch.empty_like(g), torch.empty(hd, device=DEV)
    src = kept[:, :, :h]
    h3b.qk_norm_rope_backward(plan, src, None, gain, None, EPS, pos, g, None, d, None, dg, None, ws)
    h3b.qk_norm_rope_backward(plan, src, None, gain, None, EPS, pos, g, None, g, None, None, None, ws)
    h3b.sync_status()
    assert torch.equal(d, g)


def test_rotation_agrees_with_the_block_table():
    # the grid's own table (h3b_rope_table) turns the same pairs by the same angles
    split, hd, n_audio = (16, 24, 24), 64, 5
    dims = h3b.make_dims(256, 4, hd, 1024, 256, split)
    grid = h3b.make_grid(3, 4, 6, n_audio)
    n = 3 * 4 * 6 + n_audio
    cs = torch.empty(n, hd // 2, 2, device=DEV)
    h3b.rope_table(dims, grid, False, cs)
    t, y, w = torch.meshgrid(torch.arange(3.), torch.arange(4.), torch.arange(6.), indexing="ij")
    pos = torch.cat((torch.stack((t, y, w), -1).reshape(-1, 3), torch.zeros(n_audio, 3))).to(DEV)
    unit = torch.zeros(n, 1, hd, device=DEV)
    unit[..., 0::2] = 1.0
    out = torch.empty_like(unit)
    h3b.rope_axes(h3b.make_rope_axes(split), unit, pos, out)
    h3b.sync_status()
    # two ways to the same sine and cosine in 32 bits, each within TURN
    assert (out.view(n, hd // 2, 2) - cs).abs().max().item() <= 2 * TURN


def test_norm_only_and_empty_calls():
    b, t, h, hd = 2, 11, 3, 72
    x = rnd((b, t, h, hd), 1.0, seed=1, dtype=F32)
    x[0, 3, 1] = 0.0                                  # a zero head stays zero
    out = torch.empty_like(x, device=DEV)
    h3b.qk_norm_rope(None, x.to(DEV), None, None, None, EPS, None, out, None)
    want = OH.norm_rope(np64(x), 1.0, EPS)
    within(out, want, stored(want, NORM * np.abs(want), F32))
    g = rnd((b, t, h, hd), 1.0, seed=2, dtype=F32)
    dx, dg = torch.empty_like(out), torch.empty(hd, device=DEV)
    ws = h3b.workspace(h3b.qk_norm_rope_backward_workspace_size(hd))
    h3b.qk_norm_rope_backward(None, x.to(DEV), None, None, None, EPS, None, g.to(DEV), None, dx, None,
                              dg, None, ws)
    h3b.sync_status()
    wx, ex, wg, eg = backward_bounds(np64(x), np.ones(hd), np64(g), None, None)
    within(dx, wx, stored(wx, ex, F32))
    within(dg, wg, eg)
    # no tokens: nothing is read, and the gains' gradients are zero
    e = torch.empty(0, h, hd, device=DEV)
    h3b.qk_norm_rope(None, e, e, None, None, EPS, None, e, e)
    plan = h3b.make_rope_axes((8,))
    h3b.rope_axes(plan, e, torch.empty(0, 1, device=DEV), e)
    dg2 = torch.full((hd,), 7.0, device=DEV)
    h3b.qk_norm_rope_backward(None, e, e, None, None, EPS, None, e, e, e, e, dg, dg2, ws)
    h3b.sync_status()
    assert not dg.any() and not dg2.any()


def test_special_values_stay_in_their_head():
    t, h, hd = 6, 4, 128
    plan = h3b.make_rope_axes((32, 48, 48))
    x = rnd((t, h, hd), 1.0, seed=1).to(DEV)
    clean = torch.empty_like(x)
    pos = positions(1, t, 3)[0].to(DEV)
    h3b.qk_norm_rope(plan, x, None, None, None, EPS, pos, clean, None)
    x[2, 1, 5] = float("nan")
    x[4, 3, 9] = float("inf")
    out = torch.empty_like(x)
    h3b.qk_norm_rope(plan, x, None, None, None, EPS, pos, out, None)
    h3b.sync_status()
    assert out[2, 1].isnan().all()
    rest = torch.ones(t, h, dtype=torch.bool, device=DEV)
    rest[2, 1] = rest[4, 3] = False
    assert torch.equal(out[rest], clean[rest])


def test_other_stream_and_captured_graph():
    t, h, kv, hd, split = 300, 6, 2, 128, (32, 48, 48)
    plan = h3b.make_rope_axes(split)
    pos = positions(1, t, 3)[0].to(DEV)
    q, k = rnd((t, h, hd), 1.0, seed=1).to(DEV), rnd((t, kv, hd), 1.0, seed=2).to(DEV)
    gq, gk = rnd((t, h, hd), 1.0, seed=3).to(DEV), rnd((t, kv, hd), 1.0, seed=4).to(DEV)
    gain = torch.ones(hd, device=DEV)
    ws = h3b.workspace(h3b.qk_norm_rope_backward_workspace_size(hd))

    def buffers():
        return [torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(q), torch.zeros_like(k),
                torch.zeros(hd, device=DEV), torch.zeros(hd, device=DEV)]

    def both(o):
        h3b.qk_norm_rope(plan, q, k, gain, gain, EPS, pos, o[0], o[1])
        h3b.qk_norm_rope_backward(plan, q, k, gain, gain, EPS, pos, gq, gk, *o[2:], ws)

    want = buffers()
    both(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = buffers()
    with torch.cuda.stream(side):
        both(got)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    cap = buffers()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(cap)
    q.copy_(rnd((t, h, hd), 1.0, seed=11))
    gk.copy_(rnd((t, kv, hd), 1.0, seed=14))
    want = buffers()
    both(want)
    for _ in range(2):
        graph.replay()
    h3b.sync_status()
    assert all(torch.equal(a, b) for a, b in zip(want, cap))


def test_binding_refuses():
    plan = h3b.make_rope_axes((8,))
    x = torch.zeros(2, 3, 4, 16, dtype=BF, device=DEV)
    pos = torch.zeros(3, 1, device=DEV)
    n = h3b.launch_count()
    with pytest.raises(TypeError):
        h3b.rope_axes(plan, x.cpu(), pos, x)
    with pytest.raises(TypeError):
        h3b.rope_axes(plan, x.double(), pos, x.double())
    with pytest.raises(ValueError):                       # another type
        h3b.rope_axes(plan, x, pos, x.float())
    with pytest.raises(ValueError):                       # another shape
        h3b.rope_axes(plan, x, pos, x[:, :2])
    with pytest.raises(ValueError):                       # head_dim not contiguous
        h3b.rope_axes(plan, x.transpose(2, 3), pos, x.transpose(2, 3))
    with pytest.raises(ValueError):                       # positions of other sizes or types
        h3b.rope_axes(plan, x, pos[:2], x)
    with pytest.raises(ValueError):
        h3b.rope_axes(plan, x, pos.double(), x)
    with pytest.raises(ValueError):                       # gains of another length
        h3b.qk_norm_rope(plan, x, None, torch.ones(8, device=DEV), None, EPS, pos, x, None)
    with pytest.raises(h3b.H3BError):                     # strides of 4 bytes
        y = torch.zeros(2, 3, 4, 18, dtype=BF, device=DEV)[..., :16]
        h3b.rope_axes(plan, y, pos, y)
    with pytest.raises(h3b.H3BError):                     # broadcast output
        h3b.rope_axes(plan, x, pos, x[:1].expand_as(x))
    with pytest.raises(h3b.H3BError) as e:                # workspace too small
        h3b.qk_norm_rope_backward(plan, x, None, None, None, EPS, pos, x, None, x.clone(), None,
                                  None, None, h3b.workspace(1024))
    assert e.value.code == h3b.H3B_EWORKSPACE
    assert h3b.launch_count() == n
