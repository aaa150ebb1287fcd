"""Workloads of the head-norm, position-rotation and shared-prefix attention operators.

Three operators, each in a plain form (elementary torch operations in 32 bits, angles in 64)
and as the calls a user makes of the framework:

  rope_axes        rotary positions with several axes (time, height, width) at explicit
                   positions; inverse=True is the gradient of the rotation
  qk_norm_rope     per-head RMS norm of queries and keys with the rotation in the same pass,
                   and its backward pass (gradients of q, k and of both gains)
  attention_prefix attention for a batch of sequences that share one long prefix: every query
                   reads the shared keys and values and those of its own sequence

They are one path: a batch of clips that continue the same conditioning clip norms and rotates
its queries and keys, keeps the conditioning's keys and values once, and attends to both.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
THETA = 10000.0
EPS = 1e-6


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # one new token of each of four streamed clips, far into the stream: a call whose
        # time is launch latency
        dict(name="rope_axes_stream_token", op="rope_axes", dtype="bf16", batch=4, tokens=1,
             heads=24, head_dim=128, split="32,48,48", pairing="adjacent", shared_freq=False,
             packed=False, per_sample=True, far=90000, inverse=False),
        # the queries of a 512x512 clip (6 x 16 x 16 tokens and 64 audio tokens, 24 heads of
        # 128), read out of the packed projection buffer
        dict(name="rope_axes_clip", op="rope_axes", dtype="bf16", batch=1, tokens=1600, heads=24,
             head_dim=128, split="32,48,48", pairing="adjacent", shared_freq=False, packed=True,
             per_sample=False, far=0, inverse=False),
        # the gradient of the rotation at the 768x1344 clip's 11,344 tokens, pairs half a head
        # apart with one frequency ladder over all axes, two samples on shared positions
        dict(name="rope_axes_gradient_768x1344", op="rope_axes", dtype="fp16", batch=2,
             tokens=11344, heads=24, head_dim=128, split="32,48,48", pairing="halves",
             shared_freq=True, packed=False, per_sample=False, far=0, inverse=True),
        # the tiny model's 40 tokens, 4 heads of 64, in 32 bits
        dict(name="qk_norm_rope_tiny", op="qk_norm_rope", dtype="fp32", batch=1, tokens=40,
             heads=4, kv_heads=4, head_dim=64, split="16,24,24", pairing="adjacent",
             shared_freq=False, packed=True, per_sample=False, far=0),
        # queries and keys of a 512x512 clip out of the packed projection buffer
        dict(name="qk_norm_rope_clip", op="qk_norm_rope", dtype="bf16", batch=1, tokens=1600,
             heads=24, kv_heads=24, head_dim=128, split="32,48,48", pairing="adjacent",
             shared_freq=False, packed=True, per_sample=False, far=0),
        # three 768x1344 clips less a few tokens (an odd count), shared key heads, positions
        # of each sample its own
        dict(name="qk_norm_rope_768x1344_shared_heads", op="qk_norm_rope", dtype="bf16", batch=3,
             tokens=11341, heads=24, kv_heads=8, head_dim=128, split="32,48,48",
             pairing="halves", shared_freq=False, packed=False, per_sample=True, far=500),
        # training step on a 512x512 clip
        dict(name="qk_norm_rope_backward_clip", op="qk_norm_rope_backward", dtype="bf16", batch=1,
             tokens=1600, heads=24, kv_heads=24, head_dim=128, split="32,48,48",
             pairing="adjacent", shared_freq=False, packed=True, per_sample=False, far=0),
        # training step on two 768x1344 clips, shared key heads
        dict(name="qk_norm_rope_backward_768x1344", op="qk_norm_rope_backward", dtype="fp16",
             batch=2, tokens=11343, heads=24, kv_heads=8, head_dim=128, split="32,48,48",
             pairing="halves", shared_freq=True, packed=False, per_sample=False, far=0),
        # one token each of two streams with a short past: launch latency
        dict(name="attention_prefix_token_small", op="attention_prefix", dtype="bf16", batch=2,
             queries=1, heads=4, kv_heads=4, head_dim=64, prefix=257, keys=64, low=33, high=63,
             clip=False, causal=False),
        # one token each of 48 streams that continue one long clip; ragged caches
        dict(name="attention_prefix_token", op="attention_prefix", dtype="bf16", batch=48,
             queries=1, heads=24, kv_heads=8, head_dim=128, prefix=16133, keys=2048, low=1,
             high=2011, clip=False, causal=False),
        # a few tokens at once (drafted ones checked together), causal, shared key heads
        dict(name="attention_prefix_few_tokens", op="attention_prefix", dtype="fp16", batch=16,
             queries=7, heads=16, kv_heads=4, head_dim=64, prefix=4096, keys=4100, low=7,
             high=4100, clip=False, causal=True),
        # four 512x512 clips and shorter ones in one padded batch, each attending to the
        # conditioning clip's 1,024 tokens and to itself
        dict(name="attention_prefix_clips", op="attention_prefix", dtype="bf16", batch=6,
             queries=1600, heads=24, kv_heads=24, head_dim=128, prefix=1024, keys=1600, low=900,
             high=1600, clip=True, causal=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cost(case):
    w = work(case)
    return w["bytes"] / 6e12 + w["flops"] / 1e15


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(("rope_axes", "qk_norm_rope", "qk_norm_rope_backward", "attention_prefix",
                         "attention_prefix"))
        if op == "attention_prefix":
            kv_heads = rng.choice((1, 2, 4, 8, 16, 24))
            heads = kv_heads * rng.choice([g for g in (1, 2, 3, 4, 8) if g * kv_heads <= 32])
            case = dict(op=op, dtype=rng.choice(("bf16", "fp16")), heads=heads, kv_heads=kv_heads,
                        head_dim=rng.choice((64, 128)))
            if rng.random() < 0.5:     # tokens after a cache
                q = rng.choice((1, 1, 1, rng.randint(2, 16)))
                high = _log_int(rng, max(q, 16), 4096)
                case.update(batch=_log_int(rng, 1, 64), queries=q,
                            prefix=_log_int(rng, 1, 16384), keys=high + rng.randint(0, 64),
                            low=rng.randint(q, high), high=high, clip=False,
                            causal=q > 1 and rng.random() < 0.7)
            else:                      # clips
                q = _log_int(rng, 40, 4096)
                case.update(batch=rng.randint(1, 6), queries=q, prefix=_log_int(rng, 64, 4096),
                            keys=q, low=rng.randint((q + 1) // 2, q), high=q, clip=True,
                            causal=rng.random() < 0.3)
            if (case["batch"] * heads * case["queries"] * (case["prefix"] + case["keys"])
                    > 800_000_000):
                continue
        else:
            hd, split = rng.choice(((64, "16,24,24"), (128, "32,48,48"), (128, "16,56,56"),
                                    (128, "128"), (96, "32,32,32"), (128, "32,32"),
                                    (64, "32,32")))
            kv_heads = rng.choice((1, 2, 4, 8, 16, 24))
            heads = kv_heads * rng.choice([g for g in (1, 2, 3, 4, 8) if g * kv_heads <= 32])
            case = dict(op=op, dtype=rng.choice(("bf16", "bf16", "fp16", "fp32")),
                        batch=rng.randint(1, 4), tokens=_log_int(rng, 1, 11344), heads=heads,
                        head_dim=hd, split=split, pairing=rng.choice(("adjacent", "halves")),
                        shared_freq=rng.random() < 0.5, packed=rng.random() < 0.5,
                        per_sample=rng.random() < 0.5, far=rng.choice((0, 0, 1000, 100000)))
            if op == "rope_axes":
                case["inverse"] = rng.random() < 0.5
            else:
                case["kv_heads"] = kv_heads
        if _cost(case) <= most:
            return case


def _lens(case):
    """The sequences' own lengths, from high down to low."""
    b = case["batch"]
    return [case["high"] - (case["high"] - case["low"]) * i // max(1, b - 1) for i in range(b)]


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    hd = case["head_dim"]
    if case["op"] == "attention_prefix":
        h, kv, p = case["heads"], case["kv_heads"], case["prefix"]
        pairs = rows = own_keys = 0
        for n in _lens(case):
            q = n if case["clip"] else case["queries"]
            rows += q
            own_keys += n
            pairs += q * p + (q * n if not case["causal"] else q * n - q * (q - 1) // 2)
        return {"bytes": size * hd * (2 * rows * h + 2 * (p + own_keys) * kv) + 4 * case["batch"],
                "flops": 4 * pairs * h * hd}
    n = case["batch"] * case["tokens"]
    axes = len(case["split"].split(","))
    pos = 4 * axes * case["tokens"] * (case["batch"] if case["per_sample"] else 1)
    if case["op"] == "rope_axes":
        return {"bytes": 2 * size * n * case["heads"] * hd + pos, "flops": 3 * n * case["heads"] * hd}
    e = n * (case["heads"] + case["kv_heads"]) * hd
    if case["op"] == "qk_norm_rope":
        return {"bytes": 2 * size * e + pos + 8 * hd, "flops": 7 * e}
    return {"bytes": 3 * size * e + pos + 16 * hd, "flops": 16 * e}


# ------------------------------------------------------------------------------- inputs
def _positions(case, gen, dev):
    """[tokens, axes] or [batch, tokens, axes]: a raster walk over a grid (coordinates of
    paired tokens sit half way between two columns) that starts far into a stream; the last
    tokens (audio) at the origin."""
    axes = len(case["split"].split(","))
    t = case["tokens"]
    b = case["batch"] if case["per_sample"] else 1
    i = torch.arange(t, device=dev, dtype=torch.float64)
    w = max(1, int(math.sqrt(t / 2)))
    start = case["far"] + torch.randint(0, 50, (b, 1), generator=gen, device=dev).double()
    cols = [start + torch.floor(i / (w * w)), (torch.floor(i / w) % w).expand(b, t),
            (0.5 + 2 * (i % w)).expand(b, t)][:axes]
    pos = torch.stack(cols, -1)
    if t > 8:
        pos[:, t - t // 20:] = 0.0
    pos = pos.float()
    return pos.contiguous() if case["per_sample"] else pos[0].contiguous()


def _split(case):
    return [int(s) for s in case["split"].split(",")]


def _ladder(case, dev):
    """The axis and the frequency (64 bits) of every pair, as a model keeps them."""
    split = _split(case)
    axis = [a for a, s in enumerate(split) for _ in range(s // 2)]
    if case["shared_freq"]:
        freq = [THETA ** (-2.0 * p / sum(split)) for p in range(len(axis))]
    else:
        freq = [THETA ** (-2.0 * k / s) for s in split for k in range(s // 2)]
    return {"axis": torch.tensor(axis, device=dev),
            "freq": torch.tensor(freq, device=dev, dtype=torch.float64)}


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    dt = DTYPES[case["dtype"]]
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dt)

    b, h, hd = case["batch"], case["heads"], case["head_dim"]
    if case["op"] == "attention_prefix":
        kv, nq, nk, p = case["kv_heads"], case["queries"], case["keys"], case["prefix"]
        order = torch.randperm(b, generator=gen, device=dev)
        lens = torch.tensor(_lens(case), dtype=torch.int32, device=dev)[order].contiguous()
        return {"case": case, "q": normal(b, nq, h, hd), "k_prefix": normal(p, kv, hd),
                "v_prefix": normal(p, kv, hd), "k": normal(b, nk, kv, hd),
                "v": normal(b, nk, kv, hd), "kv_len": lens,
                "q_len": lens if case["clip"] else None,
                "out": torch.zeros(b, nq, h, hd, dtype=dt, device=dev)}
    t = case["tokens"]
    state = {"case": case, "pos": _positions(case, gen, dev), **_ladder(case, dev)}
    if case["op"] == "rope_axes":
        if case["packed"]:
            x = normal(b, t, 3 * h, hd)[:, :, :h]
        else:
            x = normal(b, t, h, hd)
        state.update(x=x, out=torch.empty(b, t, h, hd, dtype=dt, device=dev))
        return state
    kv = case["kv_heads"]
    if case["packed"]:
        qkv = normal(b, t, h + 2 * kv, hd)
        q, k = qkv[:, :, :h], qkv[:, :, h:h + kv]
    else:
        q, k = normal(b, t, h, hd), normal(b, t, kv, hd)
    state.update(q=q, k=k)
    for name in ("q_gain", "k_gain"):
        state[name] = 1.0 + 0.1 * torch.randn(hd, generator=gen, device=dev, dtype=torch.float32)
    if case["op"] == "qk_norm_rope_backward":
        state.update(g_q=normal(b, t, h, hd), g_k=normal(b, t, kv, hd),
                     dq_gain=torch.empty(hd, device=dev), dk_gain=torch.empty(hd, device=dev))
    state.update(q_out=torch.empty(b, t, h, hd, dtype=dt, device=dev),
                 k_out=torch.empty(b, t, kv, hd, dtype=dt, device=dev))
    return state


# ------------------------------------------------------------------------------- plain forms
def _cos_sin(state):
    """cos and sin [batch or 1, tokens, 1, pairs]; the angles in 64 bits."""
    angle = state["pos"].double()[..., state["axis"]] * state["freq"]
    if angle.dim() == 2:
        angle = angle[None]
    return torch.cos(angle).float()[:, :, None], torch.sin(angle).float()[:, :, None]


def _rotate(case, x, cos, sin):
    """x [batch, tokens, heads, head_dim] in 32 bits, turned by the angles."""
    rot = sum(_split(case))
    if case["pairing"] == "adjacent":
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _norm_rope(case, x, gain, cos, sin):
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return _rotate(case, x * r * gain, cos, sin)


def _norm_rope_backward(case, x, gain, g, cos, sin):
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    z = _rotate(case, g.float(), cos, -sin)
    n = x * r
    d_gain = (z * n).sum((0, 1, 2))
    z = z * gain
    return r * (z - n * (z * n).mean(-1, keepdim=True)), d_gain


def _attention(s):
    case = s["case"]
    q, kv = s["q"].float(), case["kv_heads"]
    b, nq, h, hd = q.shape
    nk, p = case["keys"], case["prefix"]
    q = q.view(b, nq, kv, h // kv, hd) / math.sqrt(hd)
    far = torch.einsum("bqhgd,phd->bhgqp", q, s["k_prefix"].float())
    near = torch.einsum("bqhgd,bkhd->bhgqk", q, s["k"].float())
    kv_len = s["kv_len"][:, None, None]
    q_len = s["q_len"] if s["q_len"] is not None else torch.full_like(s["kv_len"], nq)
    i = torch.arange(nq, device=q.device)[None, :, None]
    j = torch.arange(nk, device=q.device)[None, None, :]
    seen = (j < kv_len).expand(b, nq, nk)
    if case["causal"]:
        seen = seen & (j <= i + kv_len - q_len[:, None, None])
    near = near.masked_fill_(~seen[:, None, None], -math.inf)
    top = torch.maximum(far.amax(-1, keepdim=True), near.amax(-1, keepdim=True))
    far = far.sub_(top).exp_()
    near = near.sub_(top).exp_()
    total = far.sum(-1) + near.sum(-1)
    o = (torch.einsum("bhgqp,phd->bqhgd", far, s["v_prefix"].float())
         + torch.einsum("bhgqk,bkhd->bqhgd", near, s["v"].float()))
    o = o / total.permute(0, 3, 1, 2)[..., None]
    rows = torch.arange(nq, device=q.device)[None] < q_len[:, None]
    return (o.reshape(b, nq, h, hd) * rows[:, :, None, None]).to(s["q"].dtype)


# ------------------------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    if own:
        return _own(state)
    if case["op"] == "attention_prefix":
        return _attention(state)
    cos, sin = _cos_sin(state)
    if case["op"] == "rope_axes":
        x = state["x"]
        return _rotate(case, x.float(), cos, -sin if case["inverse"] else sin).to(x.dtype)
    q, k, dt = state["q"], state["k"], state["q"].dtype
    if case["op"] == "qk_norm_rope":
        return {"q": _norm_rope(case, q, state["q_gain"], cos, sin).to(dt),
                "k": _norm_rope(case, k, state["k_gain"], cos, sin).to(dt)}
    dq, dq_gain = _norm_rope_backward(case, q, state["q_gain"], state["g_q"], cos, sin)
    dk, dk_gain = _norm_rope_backward(case, k, state["k_gain"], state["g_k"], cos, sin)
    return {"dq": dq.to(dt), "dk": dk.to(dt), "dq_gain": dq_gain, "dk_gain": dk_gain}


def _own(state):
    from video_diffusion_transformer_03_b200 import h3b
    case = state["case"]
    if case["op"] == "attention_prefix":
        if "ws" not in state:      # a program keeps its workspace
            state["ws"] = h3b.workspace(h3b.attention_prefix_workspace_size(
                case["batch"], case["queries"], case["heads"], case["kv_heads"],
                case["head_dim"], case["prefix"], case["keys"]))
        h3b.attention_prefix(state["q"], state["k_prefix"], state["v_prefix"], state["k"],
                             state["v"], state["out"], kv_len=state["kv_len"],
                             q_len=state["q_len"], causal=case["causal"], ws=state["ws"])
        return state["out"]
    if "rope" not in state:        # and its description of the axes
        state["rope"] = h3b.make_rope_axes(
            _split(case), theta=THETA, shared_freq=case["shared_freq"],
            pairing=h3b.ROPE_ADJACENT if case["pairing"] == "adjacent" else h3b.ROPE_HALVES)
    rope, pos = state["rope"], state["pos"]
    if case["op"] == "rope_axes":
        h3b.rope_axes(rope, state["x"], pos, state["out"], inverse=case["inverse"])
        return state["out"]
    if case["op"] == "qk_norm_rope":
        h3b.qk_norm_rope(rope, state["q"], state["k"], state["q_gain"], state["k_gain"], EPS, pos,
                         state["q_out"], state["k_out"])
        return {"q": state["q_out"], "k": state["k_out"]}
    if "ws" not in state:
        state["ws"] = h3b.workspace(h3b.qk_norm_rope_backward_workspace_size(case["head_dim"]))
    h3b.qk_norm_rope_backward(rope, state["q"], state["k"], state["q_gain"], state["k_gain"], EPS,
                              pos, state["g_q"], state["g_k"], state["q_out"], state["k_out"],
                              state["dq_gain"], state["dk_gain"], state["ws"])
    return {"dq": state["q_out"], "dk": state["k_out"], "dq_gain": state["dq_gain"],
            "dk_gain": state["dk_gain"]}


# ------------------------------------------------------------------------------- in 64 bits
def _turn64(case, x, pos, sign):
    """x (64 bits) with its pairs as complex numbers, times exp(i angle)."""
    split = _split(case)
    pos = pos.double()
    if pos.dim() == 2:
        pos = pos[None].expand(x.shape[0], -1, -1)
    angles, done = [], 0
    for a, s in enumerate(split):
        k = torch.arange(s // 2, device=x.device, dtype=torch.float64)
        e = (k + done) * 2 / sum(split) if case["shared_freq"] else k * 2 / s
        angles.append(pos[:, :, a, None] * torch.exp(-math.log(THETA) * e))
        done += s // 2
    angle = sign * torch.cat(angles, -1)[:, :, None]
    rot = sum(split)
    head, tail = x[..., :rot], x[..., rot:]
    if case["pairing"] == "adjacent":
        z = torch.complex(head[..., 0::2], head[..., 1::2])
    else:
        z = torch.complex(head[..., :rot // 2], head[..., rot // 2:])
    z = z * torch.polar(torch.ones_like(angle), angle)
    order = -1 if case["pairing"] == "adjacent" else -2
    y = torch.stack((z.real, z.imag), order).flatten(-2)
    return torch.cat((y, tail), -1)


def _normed64(x, gain):
    return x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS) * gain


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope_axes":
        return _turn64(case, s["x"].double(), s["pos"], -1.0 if case["inverse"] else 1.0)
    if case["op"] == "attention_prefix":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
        g = case["heads"] // case["kv_heads"]
        for b, n in enumerate(s["kv_len"].tolist()):
            rows = n if case["clip"] else case["queries"]
            for h in range(case["kv_heads"]):
                k = torch.cat((s["k_prefix"][:, h], s["k"][b, :n, h])).double()
                v = torch.cat((s["v_prefix"][:, h], s["v"][b, :n, h])).double()
                hidden = None
                if case["causal"]:
                    last = case["prefix"] + n - rows + torch.arange(rows, device=k.device)
                    hidden = torch.arange(k.shape[0], device=k.device)[None] > last[:, None]
                for j in range(h * g, (h + 1) * g):
                    a = s["q"][b, :rows, j].double() @ k.T * case["head_dim"] ** -0.5
                    if hidden is not None:
                        a = a.masked_fill(hidden, -math.inf)
                    out[b, :rows, j] = torch.softmax(a, -1) @ v
        return out
    res, grads = {}, {}
    for x, gain, g in (("q", "q_gain", "g_q"), ("k", "k_gain", "g_k")):
        xv, gv = s[x].double(), s[gain].double()
        if case["op"] == "qk_norm_rope":
            res[x] = _turn64(case, _normed64(xv, gv), s["pos"], 1.0)
            continue
        xv = xv.clone().requires_grad_(True)
        gv = gv.clone().requires_grad_(True)
        y = _turn64(case, _normed64(xv, gv), s["pos"], 1.0)
        grads["d" + x], grads["d" + gain] = torch.autograd.grad(y, (xv, gv), s[g].double())
    return res or {k: grads[k] for k in ("dq", "dk", "dq_gain", "dk_gain")}
