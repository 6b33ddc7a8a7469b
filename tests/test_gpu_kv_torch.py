"""The 8-bit cache as torch sees it: lazy clones, version counters, calls of no tokens."""
import pytest
import torch

import lse_weighted_merge_b200 as lm
from kv_util import quantised
from test_gpu_kv_cache import cache, ints, rows

pytestmark = pytest.mark.gpu


def test_a_lazy_clone_of_the_cache():
    """A clone that shares its storage until it is written: the write gives it its own,
    and the tensor that it was cloned from stays as it was."""
    (kc, ks), (vc, vs) = (cache(2, 2, 12, 64, i) for i in (1, 2))
    first = [t.view(torch.uint8).clone() if t.dtype != torch.float32 else t.clone() for t in (kc, vc, ks, vs)]
    clones = [torch._lazy_clone(t) for t in (kc, vc, ks, vs)]
    k, v = rows(2, 2, 5, 64, "bf16", 3), rows(2, 2, 5, 64, "bf16", 4)
    lm.kv_quantize_(*clones, k, v, ints([0, 6]))
    for was, now in zip(first, (kc, vc, ks, vs)):
        assert torch.equal(was, now.view(torch.uint8) if now.dtype != torch.float32 else now)
    for c, s, x in ((clones[0], clones[2], k), (clones[1], clones[3], v)):
        codes, scale = quantised(x)
        assert torch.equal(c[0, :, :5].double(), codes[0]) and torch.equal(s[0, :, :5].double(), scale[0])
        assert torch.equal(c[1, :, 6:11].double(), codes[1])


def test_versions_and_saved_tensors():
    """The four written tensors have a new version, others do not; a scale that autograd has
    saved and the write changed is noticed; inference tensors are written as well."""
    (kc, ks), (vc, vs) = (cache(1, 1, 8, 64, i) for i in (1, 2))
    k = rows(1, 1, 2, 64, "bf16", 3)
    st, w = ints([0]), torch.ones(1, 1, 8, device="cuda", requires_grad=True)
    y = (w * ks).sum()
    old = [t._version for t in (kc, vc, ks, vs, k, st)]
    lm.kv_quantize_(kc, vc, ks, vs, k, k, st)
    assert [t._version for t in (kc, vc, ks, vs, k, st)] == [n + 1 for n in old[:4]] + old[4:]
    with pytest.raises(RuntimeError, match="inplace"):
        y.backward()
    old = kc._version
    lm.kv_dequantize(kc, vc, ks, vs, st, 4)
    lm.decode_attention_fp8(torch.zeros(1, 2, 64, dtype=torch.bfloat16, device="cuda"), kc, vc, ks, vs)
    assert kc._version == old
    with torch.inference_mode():
        made = [t.clone() for t in (kc, vc, ks, vs)]
        lm.kv_quantize_(*made, k, k, ints([4]))
    lm.kv_quantize_(*made, k, k, st)
    assert torch.equal(made[2][..., 4:6], ks[..., :2])


def test_attention_of_no_query_tokens():
    """A batch of no sequences, and no drafted tokens: results of that size."""
    (kc, ks), (vc, vs) = (cache(2, 2, 12, 64, i) for i in (1, 2))
    none = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    out, lse = lm.decode_attention_fp8(none, kc[:0], vc[:0], ks[:0], vs[:0], kv_len=ints([]), out_dtype=torch.float32)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4) and out.dtype == torch.float32
    out, lse = lm.tree_attention(none[:, None].expand(0, 3, 4, 64), kc[:0], vc[:0], k_scale=ks[:0], v_scale=vs[:0])
    assert out.shape == (0, 3, 4, 64) and lse.shape == (0, 3, 4)
    q = torch.zeros(2, 0, 4, 64, dtype=torch.bfloat16, device="cuda")
    d = torch.zeros(2, 2, 0, 64, dtype=torch.bfloat16, device="cuda")
    out, lse = lm.tree_attention(q, kc, vc, d, d.clone(), torch.zeros(2, 0, dtype=torch.int64, device="cuda"),
                                 k_scale=ks, v_scale=vs)
    assert out.shape == (2, 0, 4, 64) and lse.shape == (2, 0, 4)
    with pytest.raises(ValueError):
        lm.decode_attention_fp8(none, kc, vc, ks, vs)
