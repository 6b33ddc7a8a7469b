"""The largest sizes that the cache's and the attention's calls take, on the host: what
lies beyond is refused before any CUDA call (the addresses are never read)."""
import pytest

from lse_weighted_merge_b200 import _native as nat
from test_kv_host import A, FP8, tree


@pytest.mark.parametrize("cache", [{}, FP8], ids=["16 bits", "8 bits"])
@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("L", [2 ** 31 - 1, 2 ** 31 - 1023])
def test_key_indexes_that_would_pass_32_bits(L, T, cache):
    """A tile reaches past a shard's last key: the index of its last one is an int too.
    (Every token at one address, so that the cache's extent is no reason to refuse.)"""
    far = {n: a + (1 << 44) for n, a in A.items() if n in ("out", "lse", "ws")}
    rc = tree(L=L, T=T, c=(128, 64, 0), s=(2, 1, 0), d=(T * 128, T * 64, 64), qs=(T * 512, 512, 64), tree_b=T,
              **cache, **far)
    assert rc == nat.EDIMS, nat.strerror(rc)


@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("scale", [2.5e38, -2.9e38, float("nan"), float("-inf")])
def test_scales_that_overflow_in_powers_of_two(scale, T):
    """The kernels work in powers of two: scale * log2(e) has to be finite."""
    far = {n: a + (1 << 44) for n, a in A.items() if n in ("out", "lse", "ws")}
    rc = tree(T=T, scale=scale, d=(T * 128, T * 64, 64), qs=(T * 512, 512, 64), tree_b=T, **far)
    assert rc == nat.EDIMS, nat.strerror(rc)
