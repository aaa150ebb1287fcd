"""Float64 oracle of the operators on heads: rotary positions with several axes, per-head RMS
norm with that rotation (forward and its gradients), and attention over a shared prefix.

Written from the formulas with numpy, independent of the CUDA library.
"""
import numpy as np


def ladder(split, theta=10000.0, shared_freq=False):
    """(axis, frequency) of every pair, pairs numbered axis by axis."""
    axis, freq, rot = [], [], sum(split)
    for a, width in enumerate(split):
        for k in range(width // 2):
            p = len(axis)
            freq.append(float(theta) ** (-2.0 * p / rot if shared_freq else -2.0 * k / width))
            axis.append(a)
    return np.array(axis, int), np.array(freq)


def rope_axes(x, pos, split, theta=10000.0, halves=False, shared_freq=False, inverse=False):
    """x [..., tokens, heads, head_dim]; pos [..., tokens, axes] broadcast over what it lacks."""
    axis, freq = ladder(split, theta, shared_freq)
    n = len(axis)
    ang = np.asarray(pos, np.float64)[..., axis] * freq
    ang = ang[..., None, :] * (-1.0 if inverse else 1.0)
    x = np.asarray(x, np.float64)
    ia = np.arange(n) if halves else 2 * np.arange(n)
    ib = ia + (n if halves else 1)
    y = x.copy()
    y[..., ia] = x[..., ia] * np.cos(ang) - x[..., ib] * np.sin(ang)
    y[..., ib] = x[..., ia] * np.sin(ang) + x[..., ib] * np.cos(ang)
    return y


def norm_rope(x, gain, eps, pos=None, split=None, **kw):
    x = np.asarray(x, np.float64)
    n = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * gain
    return n if split is None else rope_axes(n, pos, split, **kw)


def norm_rope_backward(x, gain, eps, g, pos=None, split=None, **kw):
    """(dx, dgain) of sum(g * norm_rope(x, gain))."""
    x, g = np.asarray(x, np.float64), np.asarray(g, np.float64)
    z = g if split is None else rope_axes(g, pos, split, inverse=True, **kw)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r
    dgain = (z * n).reshape(-1, x.shape[-1]).sum(0)
    w = z * gain
    return r * (w - n * (w * n).mean(-1, keepdims=True)), dgain


def attention_prefix(q, kp, vp, k, v, kv_len=None, q_len=None, causal=False, scale=None):
    """q [batch, n_q, heads, hd]; kp, vp [n_prefix, kv_heads, hd]; k, v [batch, n_kv, kv_heads,
    hd].  Rows past q_len come back as NaN (not written); rows that see no key as zero."""
    q, kp, vp, k, v = (np.asarray(t, np.float64) for t in (q, kp, vp, k, v))
    batch, n_q, heads, hd = q.shape
    group = heads // k.shape[2]
    scale = hd ** -0.5 if scale is None else scale
    out = np.full(q.shape, np.nan)
    for b in range(batch):
        nk = k.shape[1] if kv_len is None else int(kv_len[b])
        nq = n_q if q_len is None else int(q_len[b])
        for h in range(heads):
            keys = np.concatenate((kp[:, h // group], k[b, :nk, h // group]))
            vals = np.concatenate((vp[:, h // group], v[b, :nk, h // group]))
            s = q[b, :nq, h] @ keys.T * scale
            if causal:
                own = np.arange(len(keys))[None] - len(kp)      # negative: the prefix's
                s = np.where(own <= np.maximum(nk - nq + np.arange(nq)[:, None], -1), s, -np.inf)
            top = s.max(-1, keepdims=True, initial=-np.inf)
            p = np.exp(s - np.where(np.isfinite(top), top, 0.0))
            total = p.sum(-1, keepdims=True)
            out[b, :nq, h] = (p @ vals) / np.where(total > 0, total, 1.0)
    return out
