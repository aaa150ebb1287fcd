"""Tensors that a call of the operators on heads would not look at are refused by the binding,
before anything else (no GPU needed)."""
import pytest
import torch

from video_diffusion_transformer_03_b200 import h3b

X = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16)
P = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
N = torch.zeros(2, dtype=torch.int32)


@pytest.mark.parametrize("args,kw,word", [
    ((None, P, X, X), {}, "v_prefix is given without k_prefix"),
    ((P, P, None, X), {}, "v is given without k"),
    ((P, P, None, None), dict(kv_len=N), "kv_len is given without k"),
    ((None, P, None, X), {}, "v_prefix is given without k_prefix")])
def test_attention_prefix_refuses_half_a_pair(args, kw, word):
    with pytest.raises(ValueError, match=word):
        h3b.attention_prefix(X, *args, X, **kw)


def test_qk_norm_rope_refuses_what_goes_with_k():
    with pytest.raises(ValueError, match="k_out is given without k"):
        h3b.qk_norm_rope(None, X, None, None, None, 1e-6, None, X, X)
    for name, g_k, dk in (("g_k", X, None), ("dk", None, X)):
        with pytest.raises(ValueError, match=name + " is given without k"):
            h3b.qk_norm_rope_backward(None, X, None, None, None, 1e-6, None, X, g_k, X, dk, None, None,
                                      None)
