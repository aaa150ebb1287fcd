"""Attention over a shared prefix through the binding, against the float64 oracle
(oracle/heads.py), at the sizes and masks where it can go wrong.

Tolerance, per output: with A = sum p |v| / sum p (the oracle run on |v|), u half a step of the
type, n keys and head width d,
  * the weights are rounded to the type before the product with V: u A;
  * a score is a sum of d products kept in fp32: off by at most d 2^-23 sum |q k| scale (an
    accumulator that truncates loses 2^-23 a step), in the exponent, so in p and in sum p;
  * the sums over n keys: n 2^-23 A in the product, and as much in sum p;
  * the exponential (2^-22 relative, and the rounding of arguments below 64): 1e-5 A;
  * the store: u |out|, and half the type's smallest step.
"""
import math

import numpy as np
import pytest
import torch

from oracle import heads as OH
from oracle import oracle as O
from tests.helpers import np64, rel_l2, rnd

pytestmark = pytest.mark.gpu

h3b = pytest.importorskip("video_diffusion_transformer_03_b200.h3b")

DEV = "cuda"
BF, HF = torch.bfloat16, torch.float16
NAN = float("nan")


def bound(q, kp, vp, k, v, want, dtype, scale=None, **kw):
    fi = torch.finfo(dtype)
    u, hd = fi.eps / 2, q.shape[-1]
    scale = hd ** -0.5 if scale is None else scale
    weight = OH.attention_prefix(q, kp, np.abs(vp), k, np.abs(v), scale=scale, **kw)
    n = len(kp) + k.shape[1]
    keys = np.concatenate((kp.reshape(-1, hd), k.reshape(-1, hd)))
    rows = np.nan_to_num(np.abs(q)).reshape(-1, hd)
    dots = np.nan_to_num(np.abs(keys)).max(0) if len(keys) else np.zeros(hd)
    score = hd * 2.0 ** -23 * (rows @ dots).max(initial=0.0) * scale
    return (u + 2 * score + 2 * n * 2.0 ** -23 + 1e-5) * weight + u * np.abs(want) + \
        fi.smallest_normal * fi.eps


def make(batch, nq, heads, kv, hd, prefix, nkv, dtype, seed=0, kv_len=None, q_len=None, std=1.0,
         grow=0.0):
    """CPU inputs.  What no call may look at (queries past q_len, keys past kv_len) is NaN."""
    q = rnd((batch, nq, heads, hd), std, seed=seed + 1, dtype=dtype)
    kp = rnd((prefix, kv, hd), std, seed=seed + 2, dtype=dtype)
    vp = rnd((prefix, kv, hd), 1.0, seed=seed + 3, dtype=dtype)
    k = rnd((batch, nkv, kv, hd), std, seed=seed + 4, dtype=dtype)
    v = rnd((batch, nkv, kv, hd), 1.0, seed=seed + 5, dtype=dtype)
    if grow:                 # later keys score higher: the running maximum has to move
        ramp = torch.linspace(0.2, grow, prefix + nkv)[:, None, None]
        kp = (kp.float() * ramp[:prefix]).to(dtype)
        k = (k.float() * ramp[prefix:]).to(dtype)
    for b in range(batch):
        if kv_len is not None:
            k[b, max(kv_len[b], 0):] = NAN
            v[b, max(kv_len[b], 0):] = NAN
        if q_len is not None:
            q[b, max(q_len[b], 0):] = NAN
    return q, kp, vp, k, v


def workspace(q, kp, k):
    n = h3b.attention_prefix_workspace_size(q.shape[0], q.shape[1], q.shape[2], k.shape[2],
                                            q.shape[3], len(kp), k.shape[1])
    ws = h3b.workspace(n)
    ws.fill_(255)
    return ws


def ints(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device=DEV)


def call(q, kp, vp, k, v, kv_len=None, q_len=None, fill=7.0, **kw):
    d = [t.to(DEV) for t in (q, kp, vp, k, v)]
    out = torch.full(q.shape, fill, dtype=q.dtype, device=DEV)
    h3b.attention_prefix(*(t if t.numel() or t is d[0] else None for t in d), out,
                         kv_len=ints(kv_len), q_len=ints(q_len), ws=workspace(q, kp, k), **kw)
    h3b.sync_status()
    return out


def check(out, q, kp, vp, k, v, kv_len=None, q_len=None, fill=7.0, **kw):
    n = [np64(t) for t in (q, kp, vp, k, v)]
    n[3], n[4] = np.nan_to_num(n[3]), np.nan_to_num(n[4])
    lens = dict(kv_len=None if kv_len is None else np.clip(kv_len, 0, k.shape[1]),
                q_len=None if q_len is None else np.clip(q_len, 0, q.shape[1]))
    want = OH.attention_prefix(*n, **lens, **kw)
    tol = bound(*n, want, q.dtype, **lens, **kw)
    got = np64(out)
    kept = np.isnan(want)                                # rows that are not written
    assert (got[kept] == fill).all()
    bad = ~(np.abs(got - want) <= tol) & ~kept
    assert not bad.any(), (int(bad.sum()), float(np.nanmax(np.abs(got - want) / tol)),
                           np.argwhere(bad)[:4].tolist())


# batch, queries, heads, kv heads, head_dim, prefix, own keys
SIZES = [
    (1, 1, 1, 1, 64, 1, 1), (2, 1, 4, 4, 64, 257, 64), (3, 1, 6, 2, 128, 130, 33),
    (1, 1, 3, 1, 128, 0, 129), (2, 1, 8, 1, 64, 128, 0), (5, 1, 24, 8, 128, 1000, 300),
    (33, 1, 4, 1, 64, 700, 140), (2, 7, 8, 2, 128, 255, 256), (16, 3, 2, 2, 64, 4097, 127),
    (1, 16, 16, 2, 64, 63, 17), (4, 33, 6, 3, 128, 129, 40), (1, 128, 2, 1, 128, 128, 128),
    (2, 129, 3, 3, 64, 100, 129), (1, 300, 2, 1, 128, 513, 300), (2, 515, 4, 2, 64, 0, 515),
    (1, 1600, 3, 3, 128, 1024, 1600), (70, 2, 3, 3, 64, 20, 9),
    # a key head's query heads in uneven groups
    (3, 48, 6, 2, 64, 140, 130), (2, 20, 7, 1, 128, 129, 70),
    # keys and values past the L2: their tiles arrive in any order
    (40, 1, 12, 12, 128, 6000, 1100),
]


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_full_lengths(size, dtype):
    t = make(*size, dtype)
    check(call(*t), *t)


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("size", [s for s in SIZES if s[6] > 1], ids=str)
def test_ragged_lengths(size, causal):
    batch, nq, nkv = size[0], size[1], size[6]
    rng = np.random.default_rng(batch * 1000 + nq)
    kv_len = [int(x) for x in rng.integers(0, nkv + 1, batch)]
    q_len = [int(x) for x in rng.integers(0, nq + 1, batch)]
    kv_len[0], q_len[0] = nkv, nq
    if batch > 1:
        kv_len[-1], q_len[-1] = 0, min(nq, 1)
    if batch > 2:
        q_len[1], kv_len[2] = 0, 1
    t = make(*size, BF if nq % 2 else HF, seed=3, kv_len=kv_len, q_len=q_len)
    kw = dict(kv_len=kv_len, q_len=q_len, causal=causal)
    check(call(*t, **kw), *t, **kw)


@pytest.mark.parametrize("size", [(1100, 1, 4, 2, 64, 200, 40), (2500, 1, 2, 2, 64, 0, 140),
                                  (700, 5, 2, 1, 128, 130, 9)], ids=str)
def test_many_sequences(size):
    """More sequences than lanes and than blocks; whole stretches of them empty."""
    g = np.random.default_rng(11)
    kv_len = g.integers(0, size[6] + 1, size[0]).tolist()
    kv_len[40:90] = [0] * 50
    q_len = g.integers(0, size[1] + 1, size[0]).tolist()
    q_len[64:128] = [0] * 64
    d = make(*size, BF, seed=12, kv_len=kv_len, q_len=q_len)
    lens = dict(kv_len=kv_len, q_len=q_len)
    check(call(*d, **lens, causal=True), *d, **lens, causal=True)


def test_lengths_are_clamped():
    t = make(3, 5, 2, 1, 64, 40, 30, BF)
    kw = dict(kv_len=[99, -5, 30], q_len=[5, 1000, -1], causal=False)
    check(call(*t, **kw), *t, **kw)


@pytest.mark.parametrize("nq", [1, 4, 200])
def test_queries_without_keys_are_zero(nq):
    # no prefix and an empty sequence, and causal queries before the first own key
    t = make(3, nq, 4, 2, 128, 0, 150, BF, kv_len=[0, nq // 2, 150])
    for causal in (False, True):
        out = call(*t, kv_len=[0, nq // 2, 150], causal=causal)
        check(out, *t, kv_len=[0, nq // 2, 150], causal=causal)
        assert not out[0].any()
        if causal:
            assert not out[1, : nq - nq // 2].any()


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("size", [(2, 1, 4, 2, 64, 600, 300), (1, 300, 2, 2, 128, 500, 300)], ids=str)
def test_running_maximum_moves(size, dtype):
    t = make(*size, dtype, grow=6.0)
    check(call(*t), *t)
    # one key far above the others, in the last tile; then equal scores everywhere
    q, kp, vp, k, v = make(*size, dtype)
    k[:, -1] = (q[:, -1, ::size[2] // size[3]].float() * 3).to(dtype)
    check(call(q, kp, vp, k, v), q, kp, vp, k, v)
    q = torch.zeros_like(q)
    check(call(q, kp, vp, k, v), q, kp, vp, k, v)


def test_scale_and_types_of_view():
    batch, nq, heads, kv, hd, prefix, nkv = 3, 5, 6, 2, 64, 150, 90
    q, kp, vp, k, v = make(batch, nq, heads, kv, hd, prefix, nkv, BF)
    scale = 0.31
    want = call(q, kp, vp, k, v, scale=scale)
    check(want, q, kp, vp, k, v, scale=scale)
    # the same values in a packed projection buffer, in head-major caches, in one [2, ...] cache,
    # with NaN all around
    buf = torch.full((batch, nq, heads + 2 * kv + 1, hd), NAN, dtype=BF, device=DEV)
    qd = buf[:, :, :heads]
    qd.copy_(q)
    cache = torch.full((2, batch, kv, nkv + 5, hd), NAN, dtype=BF, device=DEV)
    kd, vd = (c[:, :, :nkv].transpose(1, 2) for c in cache)
    kd.copy_(k)
    vd.copy_(v)
    pre = torch.full((prefix, 2, kv, hd + 8), NAN, dtype=BF, device=DEV)
    pk, pv = pre[:, 0, :, :hd], pre[:, 1, :, :hd]
    pk.copy_(kp)
    pv.copy_(vp)
    obuf = torch.full((batch, heads, nq, hd + 16), 3.0, dtype=BF, device=DEV)
    out = obuf[..., :hd].transpose(1, 2)
    h3b.attention_prefix(qd, pk, pv, kd, vd, out, scale=scale, ws=workspace(q, kp, k))
    h3b.sync_status()
    assert torch.equal(out, want)
    assert (obuf[..., hd:] == 3.0).all()


def test_equal_calls_give_equal_bits():
    for size in ((5, 1, 24, 8, 128, 1000, 300), (2, 515, 4, 2, 64, 100, 515)):
        t = [x.to(DEV) for x in make(*size, BF)]
        ws = workspace(t[0], t[1], t[3])
        outs = [torch.empty_like(t[0]) for _ in range(3)]
        for o in outs:
            h3b.attention_prefix(*t, o, ws=ws)
        h3b.sync_status()
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_offsets_past_32_bits():
    # two caches in one buffer more than 2^31 elements apart
    batch, heads, hd, nkv = 2, 2, 64, 200
    t = make(batch, 1, heads, heads, hd, 70, nkv, BF)
    far = 2 ** 31 + 4096
    big = torch.empty(far + 2 * nkv * heads * hd, dtype=BF, device=DEV)
    kd = big.as_strided((batch, nkv, heads, hd), (far, heads * hd, hd, 1))
    vd = big.as_strided((batch, nkv, heads, hd), (far, heads * hd, hd, 1), nkv * heads * hd)
    kd.copy_(t[3])
    vd.copy_(t[4])
    out = torch.empty_like(t[0], device=DEV)
    h3b.attention_prefix(t[0].to(DEV), t[1].to(DEV), t[2].to(DEV), kd, vd, out,
                         ws=workspace(t[0], t[1], t[3]))
    h3b.sync_status()
    check(out, *t)


@pytest.mark.parametrize("size", [(6, 1, 8, 4, 128, 300, 200), (2, 300, 3, 3, 64, 200, 300)], ids=str)
def test_graphs_follow_lengths_and_share_a_workspace(size):
    t = [x.to(DEV) for x in make(*size, BF)]
    batch, nkv = size[0], size[6]
    ws = workspace(t[0], t[1], t[3])
    lens = ints([nkv] * batch)
    outs = [torch.zeros_like(t[0]) for _ in range(2)]
    h3b.attention_prefix(*t, outs[0], kv_len=lens, ws=ws)          # loads the kernels
    graphs = []
    for o, causal in zip(outs, (False, True)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            h3b.attention_prefix(*t, o, kv_len=lens, causal=causal and size[1] <= nkv, ws=ws)
        graphs.append(g)
    for step in range(3):
        new = [max(0, nkv - 37 * step - 11 * b) for b in range(batch)]
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        for g in graphs + graphs[::-1]:
            g.replay()
        h3b.sync_status()
        for o, causal in zip(outs, (False, True)):
            ref = torch.zeros_like(o)
            h3b.attention_prefix(*t, ref, kv_len=ints(new), causal=causal, ws=ws)
            h3b.sync_status()
            assert torch.equal(o, ref)


def test_two_streams_with_their_own_workspaces():
    a = [x.to(DEV) for x in make(8, 1, 8, 8, 128, 2000, 500, BF)]
    b = [x.to(DEV) for x in make(2, 400, 4, 4, 128, 300, 400, BF)]
    want = []
    for t in (a, b):
        want.append(torch.empty_like(t[0]))
        h3b.attention_prefix(*t, want[-1], ws=workspace(t[0], t[1], t[3]))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    wss = [workspace(t[0], t[1], t[3]) for t in (a, b)]
    torch.cuda.synchronize()
    got = [[torch.empty_like(a[0]) for _ in range(10)], [torch.empty_like(b[0]) for _ in range(10)]]
    for i in range(10):
        for s, t, g, ws in zip(streams, (a, b), got, wss):
            h3b.attention_prefix(*t, g[i], ws=ws, stream=s)
    torch.cuda.synchronize()
    h3b.sync_status()
    for w, g in zip(want, got):
        assert all(torch.equal(w, x) for x in g)


def test_agrees_with_the_joint_attention():
    # no own keys: the joint attention of the block over the same tokens
    n, heads, hd = 700, 4, 64
    qkv = rnd((n, 3, heads, hd), 1.0, seed=1).to(DEV)
    joint = torch.empty(n, heads * hd, dtype=BF, device=DEV)
    h3b.attention(qkv.view(n, -1), heads, hd, joint, ws=h3b.workspace(h3b.gemm_workspace_size()))
    out = torch.empty(1, n, heads, hd, dtype=BF, device=DEV)
    h3b.attention_prefix(qkv[None, :, 0], qkv[:, 1], qkv[:, 2], None, None, out,
                         ws=h3b.workspace(h3b.attention_prefix_workspace_size(1, n, heads, heads, hd, n, 0)))
    h3b.sync_status()
    # both within u A + u |out| of the same value; A is at most max |v|
    v = qkv[:, 2].float().abs().max().item()
    assert (out.view(n, -1).float() - joint.float()).abs().max().item() <= 4 * 2 ** -8 * v


def test_clips_that_continue_a_clip():
    """The operators as they are used: the keys and values of a conditioning clip are normed and
    rotated once; a batch of clips is projected, normed and rotated in its packed buffer at
    positions that follow the conditioning's, attends to both, and is projected back."""
    heads, hd, split = 4, 64, (16, 24, 24)
    d = heads * hd
    grid_p, grid_c, batch = (2, 4, 6), (3, 4, 6), 3
    n_p, n_c = 48, 72

    def raster(g, t0):
        t, y, x = np.meshgrid(np.arange(g[0]) + t0, np.arange(g[1]), np.arange(g[2]), indexing="ij")
        return np.stack((t, y, x), -1).reshape(-1, 3).astype(np.float32)

    xp, xc = rnd((n_p, d), 1.0, seed=1), rnd((batch * n_c, d), 1.0, seed=2)
    w, bias = rnd((3 * d, d), d ** -0.5, seed=3), rnd((3 * d,), 0.1, seed=4)
    wo, bo = rnd((d, d), d ** -0.5, seed=5), rnd((d,), 0.1, seed=6)
    gate = rnd((d,), 0.5, seed=7, dtype=torch.float32)
    qg, kg = (1 + rnd((hd,), 0.1, seed=s, dtype=torch.float32) for s in (8, 9))
    pos_p, pos_c = raster(grid_p, 0), raster(grid_c, grid_p[0])
    q_len = [72, 48, 72]
    # --- on the GPU
    plan = h3b.make_rope_axes(split)
    sws = h3b.workspace(h3b.gemm_workspace_size())
    wd, bd, qgd, kgd = (t.to(DEV) for t in (w, bias, qg, kg))
    pk = torch.empty(n_p, 3, heads, hd, dtype=BF, device=DEV)
    h3b.gemm_bf16(xp.to(DEV), wd, h3b.EPI_BIAS, bd, pk.view(n_p, -1), ws=sws)
    h3b.qk_norm_rope(plan, pk[:, 1], None, kgd, None, 1e-6, torch.tensor(pos_p, device=DEV), pk[:, 1],
                     None)
    qkv = torch.empty(batch, n_c, 3, heads, hd, dtype=BF, device=DEV)
    h3b.gemm_bf16(xc.to(DEV), wd, h3b.EPI_BIAS, bd, qkv.view(batch * n_c, -1), ws=sws)
    q, k, v = qkv.unbind(2)
    h3b.qk_norm_rope(plan, q, k, qgd, kgd, 1e-6, torch.tensor(pos_c, device=DEV), q, k)
    o = torch.zeros(batch, n_c, heads, hd, dtype=BF, device=DEV)
    lens = ints(q_len)
    h3b.attention_prefix(q, pk[:, 1], pk[:, 2], k, v, o, kv_len=lens, q_len=lens,
                         ws=h3b.workspace(h3b.attention_prefix_workspace_size(
                             batch, n_c, heads, heads, hd, n_p, n_c)))
    res = xc.to(DEV).clone()
    h3b.gemm_bf16(o.view(batch * n_c, d), wo.to(DEV), h3b.EPI_GATE_RESID, bo.to(DEV), res,
                  gate=gate.to(DEV), ws=sws)
    h3b.sync_status()
    # --- the oracle, in 64 bits throughout
    yp = (np64(xp) @ np64(w).T + np64(bias)).reshape(n_p, 3, heads, hd)
    yc = (np64(xc) @ np64(w).T + np64(bias)).reshape(batch, n_c, 3, heads, hd)
    kp = OH.norm_rope(yp[:, 1], np64(kg), 1e-6, pos_p, split)
    qc = OH.norm_rope(yc[:, :, 0], np64(qg), 1e-6, pos_c, split)
    kc = OH.norm_rope(yc[:, :, 1], np64(kg), 1e-6, pos_c, split)
    att = np.nan_to_num(OH.attention_prefix(qc, kp, yp[:, 2], kc, yc[:, :, 2], kv_len=q_len, q_len=q_len))
    y = att.reshape(batch * n_c, d) @ np64(wo).T + np64(bo)
    want = O.gated_residual(np64(xc), np64(gate), y)
    # the residual x carries most of the norm; compare the update: bf16 stores of qkv, of q and k
    # again, of the weights, the output and the residual: five times 2^-8 at most, independent
    assert rel_l2(np64(res) - np64(xc), want - np64(xc)) < 5 * 2 ** -8
    alone = OH.attention_prefix(qc, kp[:0], yp[:0, 2], kc, yc[:, :, 2])
    assert rel_l2(np64(o)[0], alone[0]) > 0.1            # the prefix matters


def test_binding_refuses():
    q, kp, vp, k, v = (t.to(DEV) for t in make(2, 3, 4, 2, 64, 10, 9, BF))
    out, ws = torch.empty_like(q), workspace(q, kp, k)
    n = h3b.launch_count()
    for bad in ((q.float(), kp.float(), vp.float(), k.float(), v.float(), out.float()),
                (q, None, None, None, None, out), (q[:, :, :3], kp, vp, k, v, out[:, :, :3]),
                (q, kp[:, :1].expand(10, 2, 64), vp, k, v, out)):
        with pytest.raises(h3b.H3BError):
            h3b.attention_prefix(*bad, ws=ws)
    for bad in ((q, kp, vp[:5], k, v, out), (q, kp, vp, k, v[:1], out), (q, kp, vp, k[:1], v[:1], out),
                (q, kp.half(), vp.half(), k, v, out), (q, kp, vp, k, v, out[:, :2]),
                (q, kp[:, :1], vp[:, :1], k, v, out)):
        with pytest.raises(ValueError):
            h3b.attention_prefix(*bad, ws=ws)
    with pytest.raises(TypeError):
        h3b.attention_prefix(q[0], kp, vp, k, v, out[0], ws=ws)
    for bad in ((q, kp, None, k, v, out), (q, kp, vp, k, None, out), (q, kp, vp, k, v, None)):
        with pytest.raises(TypeError):
            h3b.attention_prefix(*bad, ws=ws)
    with pytest.raises(ValueError):
        h3b.attention_prefix(q, kp, vp, k, v, out, ws=ws.cpu())
    for kw in (dict(kv_len=torch.zeros(2, dtype=torch.int64, device=DEV)),
               dict(kv_len=torch.zeros(3, dtype=torch.int32, device=DEV)),
               dict(q_len=torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(ValueError):
            h3b.attention_prefix(q, kp, vp, k, v, out, ws=ws, **kw)
    for kw in (dict(scale=-1.0, ws=ws), dict(scale=math.inf, ws=ws)):
        with pytest.raises(h3b.H3BError):
            h3b.attention_prefix(q, kp, vp, k, v, out, **kw)
    for small in (None, ws[: ws.numel() - 16]):
        with pytest.raises(h3b.H3BError) as e:
            h3b.attention_prefix(q, kp, vp, k, v, out, ws=small)
        assert e.value.code == h3b.H3B_EWORKSPACE
    # an empty batch, and no queries: nothing to do
    h3b.attention_prefix(q[:0], kp, vp, k[:0], v[:0], out[:0], ws=ws)
    h3b.attention_prefix(q[:, :0], kp, vp, k, v, out[:, :0], ws=ws)
    assert h3b.launch_count() == n
