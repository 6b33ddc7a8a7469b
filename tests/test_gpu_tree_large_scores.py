"""Scores of 10^7 and more, where fp32 has steps of whole units: the key with the largest
one takes all the weight, exact ties share it.

Queries and keys have one element that is not 0, a small whole number, so the scores of
equal keys are equal to the last bit and the next ones lie 10^7 and more below.  The
weights are then 0 or the same number p for every tied key, rounded once to the second
product's type (u_p), and the sums have a handful of fp32 roundings:
    |o - mean| <= u_o |mean| + (u_p + 2^-20) mean of |v|;
the lse is a score in log2 units times ln 2, four fp32 roundings: 2^-22 of it.

Shards (the cache's, the drafts) are merged by their lse.  fp32 has steps of 8 at 7 * 10^7,
so shards with one and with two tied keys, ln 2 apart, may get equal or quite unequal
weights: where ties can fall into shards unevenly, the result is only known to lie between
the tied values."""
import math

import pytest
import torch

from kv_util import U, attention
from test_gpu_tree import KINDS, Case

pytestmark = pytest.mark.gpu


def plain_scores(c, seed):
    """Queries of 1 and keys of -6 .. 6 in the first element, 0 elsewhere."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def small(x):
        n = torch.randint(-6, 7, x.shape[:3], generator=g, device="cuda").float()
        x.view(torch.uint8 if x.element_size() == 1 else torch.int16).zero_()
        x[..., 0] = n.to(x.dtype)

    c.q.zero_()
    c.q[..., 0] = 1
    small(c.k)
    small(c.kd)
    if c.scales:
        c.scales["k_scale"].fill_(1.0)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [2, 12, 40])
@pytest.mark.parametrize("scale", [1e7, -3e8])
def test_the_largest_score_takes_all(scale, T, kind):
    B, L = 2, 420
    for seed, (cached, drafts) in enumerate([([0], []), ([419], []), ([130], []), ([5, 6], []), ([0, 200, 419], []),
                                             ([], [0]), ([77], [0]), ([64, 300], [1])]):
        c = Case(kind, B, T, 8, 2, L, 64, seed=seed)
        plain_scores(c, seed)
        top = 7.0 if scale > 0 else -7.0
        c.tree[:] = -1                     # every draft sees every draft
        c.k[:, :, cached, 0] = torch.tensor(top, device="cuda").to(c.k.dtype)
        c.kd[:, :, drafts, 0] = top
        want, lse = attention(c.q, c.whole("k"), c.whole("v"), c.kd, c.vd, c.tree, scale=scale)[:2]
        v = torch.cat([c.whole("v")[:, :, cached], c.vd[:, :, drafts].double()], 2)     # [B, Hkv, n, D]
        mean, size = (x.mean(2).repeat_interleave(4, 1)[:, None] for x in (v, v.abs()))
        # the 64-bit form says the same, as far as it can: exp(x - lse), where lse and the
        # difference are each rounded to 2^-53 of the lse
        assert bool(((want - mean).abs() <= 2.0 ** -51 * lse.abs()[..., None] * size).all())
        uneven = len(cached) + len(drafts) > 2      # over shards
        least, most = (x.repeat_interleave(4, 1)[:, None] for x in (v.amin(2), v.amax(2)))
        for splits in (1, 3, None):
            out, got = c.run(scale=scale, splits=splits, out_dtype=torch.float32)
            off = (out.double() - mean).abs()
            if uneven:
                off = torch.maximum(least - out.double(), out.double() - most).clamp(min=0)
            err = off / (U[torch.float32] * mean.abs() + (U[c.wt] + 2.0 ** -20) * size)
            assert float(err.max()) <= 1, f"{cached} {drafts}, {splits} shards: {float(err.max()):.3f} of its bound"
            worst = float(((got.double() - lse).abs() / (2.0 ** -22 * lse.abs())).max())
            assert worst <= 1, f"{cached} {drafts}, {splits} shards: lse {worst:.3f} of its bound"


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [2, 12, 40])
def test_a_maximum_that_rises_all_along(T, kind):
    """Each tile's largest score is far above the one before it, or far below."""
    for up in (True, False):
        c = Case(kind, 1, T, 8, 2, 448, 64, seed=3)
        plain_scores(c, 3)
        step = torch.arange(448, device="cuda") // 32           # 0 .. 13
        n = step - 7 if up else 6 - step
        c.k[..., 0] = n.float().to(c.k.dtype)
        want = (c.whole("v")[:, :, 416:] if up else c.whole("v")[:, :, :32])
        mean, size = (x.mean(2).repeat_interleave(4, 1)[:, None] for x in (want, want.abs()))
        for splits in (1, 2, None):
            out, got = c.run(drafts=False, scale=2e7, splits=splits, out_dtype=torch.float32)
            err = (out.double() - mean).abs() / (U[torch.float32] * mean.abs() + (U[c.wt_cache] + 2.0 ** -20) * size)
            assert float(err.max()) <= 1, f"{'up' if up else 'down'}, {splits} shards: {float(err.max()):.3f}"
            lse = 6 * 2e7 + math.log(32)
            assert float((got.double() - lse).abs().max()) <= 2.0 ** -22 * lse
