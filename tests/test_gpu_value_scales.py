"""Attention over e4m3 values whose scales lie far apart: what a key adds to a row's
result is what counts for the row's precision, not its scale.

Bound of a row, from kv_util's with its last term (which lets an error be 2^-31 of the
largest value, whatever its weight) replaced: with W = max_j p_j max_d |v_jd|,
    |o - o64| <= u_o |o64| + (u_p + w) A + n 2^-28 W
A product p_j s_j below f16's normal range is off by 2^-25 at most.  The row's largest
product, of a value that is not all zeros, was 2^4 or more when the row's gain was last
set, and the largest code of its value is at least 224 (as kv_quantize_ writes it): each
key's error is at most 2^-29 of that product times 448, or 2^-28 W.

More than 16 rows per KV head, the last term: n (2^-27 W + 2^-31 p_max V).  A product that
is rounded with its scale was 2^3 or more at the row's largest, so 2^-27 as above.  A tile
whose scales are within 2^15 of each other has them in its values, exactly, and rounds
weights alone, of which the row's largest is 2^7 or more: 2^-32 p_max |v_j| each, with |v_j|
at most V, the largest of all or 2^16 times the smallest that is not zeros."""
import math

import pytest
import torch

import lse_weighted_merge_b200 as lm
from kv_util import U, attention
from test_gpu_tree import Case

pytestmark = pytest.mark.gpu
KINDS8 = ["bf16+e4m3", "f16+e4m3"]


def weighted(q, k, v, scale=None):
    """max over the keys of p_j max_d |v_jd|, and of p_j, [B, T, Hq], in 64 bits."""
    B, T, Hq, D = q.shape
    Hkv = k.shape[1]
    x = torch.einsum("bthgd,bhjd->bthgj", q.double().reshape(B, T, Hkv, Hq // Hkv, D), k)
    p = torch.softmax(x * (1 / math.sqrt(D) if scale is None else scale), -1)
    return [(p * f).amax(-1).reshape(B, T, Hq) for f in (v.abs().amax(-1)[:, None, :, None], 1.0)]


def check_weighted(c, what="", scale=None, **kw):
    """A call of the case without drafts, in fp32, within the bound of this file."""
    got, gl = c.run(drafts=False, out_dtype=torch.float32, scale=scale, **kw)
    k, v = c.whole("k"), c.whole("v")
    out, lse, A, S, n, _ = attention(c.q, k, v, scale=scale)
    D = out.shape[-1]
    w = 2 * ((D + 8) * 2.0 ** -23 * S + 2.0 ** -21 + n * 2.0 ** -23)
    W, p = weighted(c.q, k, v, scale)
    last = 2.0 ** -28 * W
    if c.q.shape[1] * c.q.shape[2] // k.shape[1] > 16:
        size = v.abs().amax(-1)
        V = min(float(size.max()), 2.0 ** 16 * float(size[size > 0].min())) if bool((size > 0).any()) else 0.0
        last = 2.0 ** -27 * W + 2.0 ** -31 * p * V
    bound = U[torch.float32] * out.abs() + (U[torch.float16] + w)[..., None] * A + (n * last)[..., None]
    worst = float(((got.double() - out).abs() / bound.clamp(min=1e-300)).max())
    assert worst <= 1, f"{what}: error {worst:.3f} of its bound"
    lworst = float(((gl.double() - lse).abs() / (w + 2.0 ** -21 * (1 + lse.abs()))).max())
    assert lworst <= 1, f"{what}: lse error {lworst:.3f} of its bound"


def case(kind, T, L, D, exponent, seed=0):
    """Values near 2^exponent (their scales that many powers of two from 1)."""
    c = Case(kind, 2, T, 8, 2, L, D, seed=seed)
    c.scales["v_scale"] *= 2.0 ** exponent
    return c


def zero_values(c, where):
    """What kv_quantize_ writes for a value of zeros: codes 0, scale 1."""
    c.v.view(torch.uint8)[:, :, where] = 0
    c.scales["v_scale"][:, :, where] = 1.0


ROWS = [1, 2, 4, 8, 24, 64]       # T of 4 heads per group: 4, 8, 16 rows; 32, 96, 256
ZEROS = {"first": [0], "last": [-1], "many": list(range(5, 700, 9)), "a tile": list(range(128)),
         "later tiles": list(range(256, 512)), "the start": list(range(300))}


@pytest.mark.parametrize("kind", KINDS8)
@pytest.mark.parametrize("where", ZEROS)
@pytest.mark.parametrize("exponent", [-17, -24, -40, 20])
@pytest.mark.parametrize("T", ROWS)
def test_rows_of_zeros(T, exponent, where, kind):
    """Padding and other tokens whose value is zeros, scale 1, beside small values."""
    for D in (64, 128):
        c = case(kind, T, 700, D, exponent)
        zero_values(c, ZEROS[where])
        for splits in (1, 3, None):
            check_weighted(c, f"D {D}, {splits} shards", splits=splits)


@pytest.mark.parametrize("kind", KINDS8)
@pytest.mark.parametrize("up", [6, 12, 22, 36, 60])
@pytest.mark.parametrize("T", ROWS)
def test_large_values_of_little_weight(T, up, kind):
    """Keys whose values are 2^up larger and whose scores lie far below the others':
    together they add less than the rest, and leave it its precision."""
    for seed, at in enumerate(([0], [699], [350], [1, 130, 257, 600])):
        c = case(kind, T, 700, 128, -10, seed)
        # the query's and all keys' first element make the score
        c.q[..., 0] = 16.0
        c.k.view(torch.uint8)[..., 0] = 0
        c.k[:, :, at, 0] = torch.tensor(-1.0, device="cuda").to(c.k.dtype)
        # 16 * scale * 128^-0.5 / ln 2 powers of two below the others
        c.scales["k_scale"][:, :, at] = (up + 14) * math.log(2) * math.sqrt(128) / 16
        c.k.view(torch.uint8)[:, :, at, 1:] = 0
        c.scales["v_scale"][:, :, at] *= 2.0 ** up
        for splits in (1, 2, None):
            check_weighted(c, f"at {at}, {splits} shards", splits=splits)


@pytest.mark.parametrize("kind", KINDS8)
@pytest.mark.parametrize("spread", [4, 10, 20, 40])
@pytest.mark.parametrize("T", ROWS)
def test_scales_of_all_sizes(T, spread, kind):
    """Every value's scale a power of two of its own, or no power of two."""
    for seed in (1, 2):
        c = case(kind, T, 900, 64, 0, seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        s = c.scales["v_scale"]
        s *= torch.exp2(torch.randint(-spread, spread + 1, s.shape, generator=g, device="cuda").float())
        if seed == 2:
            s *= 1 + torch.rand(s.shape, generator=g, device="cuda")
        for splits in (1, 4):
            check_weighted(c, f"{splits} shards", splits=splits)


@pytest.mark.parametrize("kind", KINDS8)
@pytest.mark.parametrize("T", ROWS)
def test_a_peak_behind_large_values(T, kind):
    """A first stretch of large values, then keys of far higher scores and small values:
    what the first stretch left is nothing beside them."""
    c = case(kind, T, 640, 128, 0)
    c.q[..., 0] = 16.0
    c.k.view(torch.uint8)[..., 0] = 0
    c.scales["v_scale"][:, :, :200] *= 2.0 ** 30
    c.k[:, :, 200:, 0] = torch.tensor(1.0, device="cuda").to(c.k.dtype)
    c.scales["k_scale"][:, :, 200:] = 70 * math.log(2) * math.sqrt(128) / 16
    c.k.view(torch.uint8)[:, :, 200:, 1:] = 0
    for splits in (1, 2, None):
        check_weighted(c, f"{splits} shards", splits=splits)


@pytest.mark.parametrize("kind", KINDS8)
@pytest.mark.parametrize("ahead", [10, 25, 45])
@pytest.mark.parametrize("T", ROWS)
def test_a_sink_of_zeros(T, ahead, kind):
    """A key with nearly all the weight, 2^ahead times the others', whose value is zeros
    of the others' scale: the result is the others', however little they weigh."""
    for at in (0, 31, 200, 639):
        c = case(kind, T, 640, 128, 9)
        c.q[..., 0] = 16.0
        c.k.view(torch.uint8)[..., 0] = 0
        c.k.view(torch.uint8)[:, :, at] = 0
        c.k[:, :, at, 0] = torch.tensor(1.0, device="cuda").to(c.k.dtype)
        c.scales["k_scale"][:, :, at] = ahead * math.log(2) * math.sqrt(128) / 16
        c.v.view(torch.uint8)[:, :, at] = 0
        c.scales["v_scale"][:, :, at] = c.scales["v_scale"][:, :, (at + 1) % 640]
        for splits in (1, 3):
            check_weighted(c, f"at {at}, {splits} shards", splits=splits)


@pytest.mark.parametrize("kind", KINDS8)
@pytest.mark.parametrize("ahead", [60, 100, 118, 140, 300])
@pytest.mark.parametrize("exponent", [-20, 0, 20])
@pytest.mark.parametrize("T", ROWS)
def test_a_sink_of_zeros_over_values_of_all_sizes(T, exponent, ahead, kind):
    """The same with weights of the others near fp32's smallest or below, and values whose
    scales lie far apart: next to nothing, but finite."""
    for at in (0, 130, 639):
        c = case(kind, T, 640, 128, exponent)
        g = torch.Generator(device="cuda").manual_seed(ahead)
        s = c.scales["v_scale"]
        s *= torch.exp2(torch.randint(-15, 16, s.shape, generator=g, device="cuda").float())
        c.q[..., 0] = 16.0
        c.k.view(torch.uint8)[..., 0] = 0
        c.k.view(torch.uint8)[:, :, at] = 0
        c.k[:, :, at, 0] = torch.tensor(1.0, device="cuda").to(c.k.dtype)
        c.scales["k_scale"][:, :, at] = ahead * math.log(2) * math.sqrt(128) / 16
        zero_values(c, at)
        ref = attention(c.q, c.whole("k"), c.whole("v"))
        for splits in (1, 3):
            out, lse = c.run(drafts=False, splits=splits, out_dtype=torch.float32)
            assert bool(torch.isfinite(out).all()), f"at {at}, {splits} shards"
            # weights below 2^-100 may be lost, those of the wider kernel below 2^-32
            floor = 640 * (2.0 ** -100 if T * 4 <= 16 else 2.0 ** -31) * float(c.whole("v").abs().max())
            assert bool(((out.double() - ref[0]).abs() <= 2.0 ** -9 * ref[2] + floor).all())
            assert float((lse.double() - ref[1]).abs().max()) <= 1e-3


@pytest.mark.parametrize("kind", KINDS8)
def test_values_that_are_all_zeros(kind):
    for T in ROWS:
        c = case(kind, T, 300, 64, -20)
        zero_values(c, list(range(300)))
        out, lse = c.run(drafts=False)
        ref = attention(c.q, c.whole("k"), c.whole("v"))
        assert bool((out == 0).all())
        assert float((lse.double() - ref[1]).abs().max()) < 1e-3


@pytest.mark.parametrize("kind", KINDS8)
def test_a_written_prompt_with_padding(kind):
    """kv_quantize_ writes small values and rows of zeros; decode over them."""
    B, Hkv, L, D = 2, 2, 500, 128
    g = torch.Generator(device="cuda").manual_seed(4)
    c = Case(kind, B, 1, 8, Hkv, L, D)
    k, v = (torch.randn(B, Hkv, L, D, generator=g, device="cuda") for _ in "kv")
    v *= 1e-6
    v[:, :, ::7] = 0
    lm.kv_quantize_(c.k, c.v, c.scales["k_scale"], c.scales["v_scale"], k, v,
                    torch.zeros(B, dtype=torch.int32, device="cuda"))
    check_weighted(c)


@pytest.mark.parametrize("kind", KINDS8)
@pytest.mark.parametrize("T", ROWS)
def test_rows_that_were_never_written(T, kind):
    """Zeros with scale 0, as a cache of zeros starts out: keys of score 0, values of 0."""
    for where in ([0], list(range(100, 300)), list(range(640)), [5, 639]):
        c = case(kind, T, 640, 64, -12)
        for x in (c.k, c.v):
            x.view(torch.uint8)[:, :, where] = 0
        for s in c.scales.values():
            s[:, :, where] = 0
        for splits in (1, 3, None):
            check_weighted(c, f"{len(where)} rows, {splits} shards", splits=splits)
