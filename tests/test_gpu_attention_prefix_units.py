"""Attention over a shared prefix where a CTA works through several units (a unit: a head's 256
queries of a sequence): more units than the GPU has SMs, heads of 64 and 128, lengths that leave
the second tile of some units empty, full and causal, against the float64 oracle at the bounds
of tests/test_gpu_attention_prefix.py."""
import numpy as np
import pytest
import torch

from tests.test_gpu_attention_prefix import BF, DEV, HF, call, check, h3b, ints, make, workspace

pytestmark = pytest.mark.gpu

# batch, queries, heads, kv heads, head_dim, prefix, own keys
SIZES = [(6, 300, 24, 24, 128, 130, 300), (5, 515, 16, 4, 128, 64, 260), (9, 130, 24, 8, 128, 0, 140),
         (7, 270, 24, 12, 64, 200, 129)]


def lengths(size, seed):
    rng = np.random.default_rng(seed)
    batch, nq, nkv = size[0], size[1], size[6]
    q_len = [int(x) for x in rng.integers(0, nq + 1, batch)]
    kv_len = [int(x) for x in rng.integers(0, nkv + 1, batch)]
    q_len[0], kv_len[0] = nq, nkv
    q_len[1], kv_len[2] = min(nq, 128), 0          # no second tile; no keys of its own
    q_len[3] = min(nq, 257)                        # two units, the second of one row
    return dict(q_len=q_len, kv_len=kv_len)


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_several_units_a_cta(size, causal, dtype):
    lens = lengths(size, size[0] + causal)
    t = make(*size, dtype, seed=21, **lens)
    kw = dict(causal=causal, **lens)
    out = call(*t, **kw)
    check(out, *t, **kw)
    assert torch.equal(out, call(*t, **kw))


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
def test_several_units_a_cta_full_lengths(dtype):
    t = make(*SIZES[0], dtype, seed=22)
    check(call(*t), *t)


def test_many_short_units_repeat_their_bits():
    # one or two steps a unit, 48 heads of 128 in 8 sequences: units end all the time
    t = [x.to(DEV) for x in make(8, 300, 48, 48, 128, 20, 100, BF, seed=23)]
    lens = ints([300, 129, 256, 200, 1, 128, 257, 299])
    ws = workspace(t[0], t[1], t[3])
    want = None
    for _ in range(20):
        out = torch.zeros_like(t[0])
        h3b.attention_prefix(*t, out, q_len=lens, ws=ws)
        want = out if want is None else want
        assert torch.equal(out, want)
    h3b.sync_status()
    host = [x.cpu() for x in t]
    rows = lens.tolist()
    for b, n in enumerate(rows):
        assert not want[b, n:].any()
    check(call(*host, q_len=rows), *host, q_len=rows)
    again = call(*host, q_len=rows, fill=0.0)
    assert torch.equal(again, want)


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("nq", [1, 200])
def test_large_scores_pick_their_key(nq, dtype):
    """Scores up to 8e6, 2^10 apart and exact: the weight of the highest key is all there is.  It is
    rounded to the type once and the output once, its sum is not: 2 u |v| + u |v|."""
    heads, hd, prefix, nkv = 2, 64, 300, 200
    rng = np.random.default_rng(5)
    q = torch.zeros(1, nq, heads, hd)
    q[..., 0] = 2.0 ** 15
    # 500 different scores, an eighth of 2^13 .. 2^13 a key in steps that both types hold
    steps = torch.tensor(rng.permutation(500).astype(np.float32)) / 2
    k = torch.zeros(500, heads, hd)
    k[..., 0] = steps[:, None]
    v = torch.tensor(rng.standard_normal((500, heads, hd)).astype(np.float32)).to(dtype)
    q, k = q.to(dtype), k.to(dtype)
    # (types of 8 bits of mantissa merge some neighbours: keep the keys that stay alone on top)
    top = int(k[:, 0, 0].float().argmax())
    k[:, :, 0] = torch.where(torch.arange(500)[:, None] == top, k[:, :, 0],
                             torch.clamp(k[:, :, 0].float(), max=240.0).to(dtype))
    out = call(q, k[:prefix], v[:prefix], k[None, prefix:], v[None, prefix:], scale=1.0)
    want = v[top].float()
    u = torch.finfo(dtype).eps / 2
    assert k[:, 0, 0].float().max() * 2.0 ** 15 > 8e6
    assert ((out.float().cpu() - want).abs() <= 3 * u * want.abs() + u * 2 ** -10).all()


@pytest.mark.parametrize("nq", [5, 150])
def test_keys_that_a_causal_query_does_not_see_may_be_anything(nq):
    q, kp, vp, k, v = make(2, nq, 4, 2, 64, 70, nq + 3, BF, seed=31)
    clean = call(q, kp, vp, k, v, causal=True)
    k[:, -1] = float("nan")                        # the last query's own key
    out = call(q, kp, vp, k, v, causal=True)
    assert torch.equal(out[:, :-1], clean[:, :-1]) and out[:, -1].isnan().all()
