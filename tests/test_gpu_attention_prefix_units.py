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
