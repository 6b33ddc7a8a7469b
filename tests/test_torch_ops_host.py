"""The binding that takes torch tensors, on the host: what it refuses before any
CUDA call."""
import pytest
import torch

import lse_weighted_merge_b200 as lm
from lse_weighted_merge_b200 import _native as nat
from lse_weighted_merge_b200 import _torch_ops as ops

FP8 = torch.float8_e4m3fn


def cache(B=2, H=2, L=8, D=64):
    return [torch.zeros(B, H, L, D).to(FP8) for _ in range(2)] + [torch.ones(B, H, L) for _ in range(2)]


def test_arguments_that_are_no_tensors():
    c, x, st = cache(), torch.zeros(2, 2, 3, 64), torch.zeros(2, dtype=torch.int32)
    q = torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16)
    for call in (lambda: lm.kv_quantize_(*c, x, [1], st), lambda: lm.kv_quantize_(None, *c[1:], x, x, st),
                 lambda: lm.kv_quantize_(*c, x, x, 5), lambda: lm.kv_dequantize(*c, "st", 3),
                 lambda: lm.tree_attention(q, c[0], c[1], k_scale=1.0, v_scale=c[3]),
                 lambda: lm.tree_attention(7, c[0], c[1]), lambda: ops.quantize(*c), lambda: ops.attention()):
        with pytest.raises(TypeError):
            call()


@pytest.mark.parametrize("bad", [
    dict(q=torch.zeros(2, 4, 64)), dict(k=torch.zeros(2, 8, 64).to(FP8)), dict(k=torch.zeros(3, 2, 8, 64).to(FP8)),
    dict(k_scale=torch.ones(2, 2, 7)), dict(k_scale=None), dict(q=torch.zeros(2, 1, 64, 4).transpose(2, 3)),
    dict(k_draft=torch.zeros(2, 2, 1, 64)), dict(tree=torch.zeros(1, dtype=torch.int64)),
])
def test_attention_shapes(bad):
    k, v, ks, vs = cache()
    a = dict(q=torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16), k=k, v=v, k_scale=ks, v_scale=vs)
    a.update(bad)
    with pytest.raises(ValueError):
        lm.tree_attention(a.pop("q"), a.pop("k"), a.pop("v"), **a)


def test_default_splits():
    d = nat.lib.lse_merge_tree_default_splits
    for args in ((0, 1, 8, 2, 100, 64, 148), (1, 1, 8, 0, 100, 64, 148), (1, 1, 8, 2, 0, 64, 148)):
        assert d(*args) == 1
    for B, T, Hq, Hkv, L in ((1, 1, 32, 8, 4096), (1, 64, 32, 8, 100000), (64, 1, 32, 8, 4096), (300, 64, 16, 1, 8192),
                             (1, 1, 1, 1, 1), (2, 5, 8, 8, 63)):
        R = d(B, T, Hq, Hkv, L, 128, 148)
        assert 1 <= R <= 64 and (R == 1 or R <= -(-L // 32))


def test_status_needs_a_place_for_its_answer():
    assert nat.lib.lse_merge_tree_status(None) == nat.ENULL
