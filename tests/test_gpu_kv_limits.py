"""The largest calls of the 8-bit cache that fit a GPU: row numbers whose threads pass
32 bits."""
import pytest
import torch

import lse_weighted_merge_b200 as lm
from kv_util import FP8, quantised

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
def test_write_of_more_rows_than_2_to_the_29(D):
    """2^29 tokens lie before the cache, the last ones in it: a short cache, and rows
    of one address, so that only the numbers are large."""
    L, before = 40, 2 ** 29
    g = torch.Generator(device="cuda").manual_seed(D)
    row = torch.randn(2, 1, 1, 1, D, generator=g, device="cuda").to(torch.bfloat16)
    k, v = (r.expand(1, 1, before + 33, D) for r in row)
    kc, vc = (torch.zeros(1, 1, L, D, device="cuda").to(FP8) for _ in "kv")
    ks, vs = (torch.full((1, 1, L), 3.0, device="cuda") for _ in "kv")
    lm.kv_quantize_(kc, vc, ks, vs, k, v, torch.tensor([-before], dtype=torch.int32, device="cuda"))
    for c, s, x in ((kc, ks, k), (vc, vs, v)):
        codes, scale = quantised(x[0, 0, :1])
        assert torch.equal(c[0, 0, :33].double(), codes.expand(33, D))
        assert bool((s[0, 0, :33].double() == scale).all())
        assert bool((c[0, 0, 33:].float() == 0).all()) and bool((s[0, 0, 33:] == 3).all())
