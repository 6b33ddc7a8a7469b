"""The tree attention of more than 16 query rows per KV head, over many key tiles
(128 keys each): rings that wrap, maxima and scales that grow from tile to tile,
row counts around the tiles' 128 and 256, against the 64-bit forms of kv_util."""
import ctypes
import math

import pytest
import torch

import lse_weighted_merge_b200 as lm
from kv_util import attention, check
from lse_weighted_merge_b200 import _native as nat
from test_gpu_tree import KINDS, Case, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_wait_ran_out():
    yield
    n = ctypes.c_uint32(7)
    assert nat.lib.lse_merge_tree_status(ctypes.byref(n)) == 0 and n.value == 0


SHAPES = [  # B, T, Hq, Hkv, L, D: T * Hq / Hkv rows
    (1, 17, 1, 1, 128, 128),
    (2, 5, 8, 2, 127, 64),
    (1, 32, 4, 1, 129, 128),      # 128 rows
    (1, 43, 3, 1, 257, 64),       # 129
    (2, 64, 2, 1, 1025, 128),     # 128, 9 tiles
    (1, 64, 4, 1, 1500, 128),     # 256
    (1, 60, 5, 1, 900, 64),       # 300
    (1, 64, 16, 1, 640, 128),     # 1024
    (1, 11, 7, 1, 2048, 128),     # 77, 16 tiles
    (3, 9, 4, 2, 1300, 64),       # 18
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("splits", [1, 2, None])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_many_tiles(shape, splits, kind):
    Case(kind, *shape, layout="blh").check(splits=splits)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [8, 48])
@pytest.mark.parametrize("up", [True, False])
def test_scores_and_values_that_grow(up, T, kind):
    """Keys that grow (or shrink) along the cache: the running maximum rises in
    every tile; e4m3 values whose scales do the same."""
    c = Case(kind, 2, T, 8, 2, 1200, 128)
    ramp = torch.arange(1200, device="cuda") / 1200
    ramp = 0.2 + 3 * (ramp if up else 1 - ramp)
    if c.scales:
        c.scales["k_scale"] *= ramp
        c.scales["v_scale"] *= torch.exp2((12 * ramp).floor())
    else:
        c.k = (c.k * ramp[:, None]).to(c.k.dtype)
    c.check(splits=1, scale=0.3, out_dtype=torch.float32)
    c.check(splits=2, scale=-0.3, out_dtype=torch.float32)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [7, 40])
def test_uneven(kind, T):
    c = Case(kind, 7, T, 8, 2, 700, 64)
    kv_len, draft_len = ints([0, 1, 700, 128, 129, 256, 511]), ints([T, 5, 0, 1, T, T - 1, 3])
    for splits in (None, 1, 2, 5):
        c.check(kv_len=kv_len, draft_len=draft_len, splits=splits)
        c.check(drafts=False, kv_len=kv_len, draft_len=draft_len, splits=splits)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("T", [6, 64])
def test_values_of_drafts_that_are_no_numbers(kind, T):
    """NaN and infinities in the drafts' values, all tiles of both streams."""
    c = Case(kind, 1, T, 4, 1, 600, 128)
    clean = c.ref()
    c.vd[0, 0, T // 2, 7], c.vd[0, 0, T // 3, 100] = math.inf, math.nan
    out, _ = c.run(splits=1)
    for j, d, ok in ((T // 2, 7, lambda x: x == math.inf), (T // 3, 100, torch.isnan)):
        sees = (c.tree[0] >> j & 1).bool()
        assert bool(ok(out[0, sees][..., d]).all())
        assert bool(torch.isfinite(out[0, ~sees][..., d]).all())
    out[..., 7], out[..., 100] = clean[0][..., 7].to(out.dtype), clean[0][..., 100].to(out.dtype)
    check(out, clean[1].float(), clean, c.wt)


def test_strides_and_offsets():
    """Sequences more than 4 GiB apart, rows of a fused projection, a cache whose
    heads interleave."""
    B, T, Hq, Hkv, L, D = 2, 10, 8, 2, 300, 128
    c = Case("bf16", B, T, Hq, Hkv, L, D)
    want, wl = c.run(splits=1)
    step = (1 << 31) + 4096          # elements
    buf = torch.zeros(step + 2 * Hkv * L * D, dtype=torch.bfloat16, device="cuda")
    for name, off in (("k", 0), ("v", Hkv * L * D)):
        far = buf.as_strided((B, Hkv, L, D), (step, D, Hkv * D, 1), off)
        far.copy_(getattr(c, name))
        setattr(c, name, far)
    qkv = torch.zeros(B, T, Hq + 3, D, dtype=torch.bfloat16, device="cuda")
    qkv[:, :, 1:Hq + 1] = c.q
    c.q = qkv[:, :, 1:Hq + 1]
    got, gl = c.run(splits=1)
    assert torch.equal(got, want) and torch.equal(gl, wl)


def test_repeats_are_the_same_bits():
    for kind in KINDS:
        c = Case(kind, 4, 40, 8, 2, 1100, 128)
        first = c.run()
        for _ in range(20):
            out, lse = c.run()
            assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


@pytest.mark.parametrize("T", [2, 40])
@pytest.mark.parametrize("kind", KINDS)
def test_scores_past_fp32s_integers(kind, T):
    """Scores so large that fp32 has steps of hundreds between them: one key takes all
    the weight, or several share it; rows stay finite and inside their values."""
    c = Case(kind, 2, T, 8, 2, 300, 64)
    for scale in (1e7, -3e8):
        out, lse = c.run(scale=scale, out_dtype=torch.float32)
        assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
        top = max(float(c.whole("v").abs().max()), float(c.vd.double().abs().max()))
        assert float(out.abs().max()) <= top * (1 + 2.0 ** -7)


@pytest.mark.parametrize("kind", ["bf16+e4m3", "f16+e4m3"])
@pytest.mark.parametrize("T", [3, 24, 64])
def test_scales_that_are_no_powers_of_two(kind, T):
    """Any positive scales, some tiles with, some without powers of two, some whose
    scales lie further apart than f16 reaches."""
    c = Case(kind, 2, T, 8, 2, 900, 128)
    g = torch.Generator(device="cuda").manual_seed(3)
    for name in ("k_scale", "v_scale"):
        s = c.scales[name]
        s[:, :, 128:256] *= 1 + torch.rand(2, 2, 128, generator=g, device="cuda")
        s[:, :, 300:310] *= 2.0 ** -20
        s[:, 1, 500:640] *= 1.25
    c.scales["v_scale"][0, :, 700:] *= 2.0 ** 9
    for splits in (1, 3, None):
        c.check(splits=splits, out_dtype=torch.float32)


@pytest.mark.parametrize("kind", ["bf16+e4m3", "bf16"])
def test_one_shard_with_drafts_in_graphs(kind):
    """The lone cached shard that joins the drafts' partial, captured behind the
    writes of its inputs, replayed on two streams at once."""
    cases = [Case(kind, 2, 48, 8, 2, 500, 128, seed=i) for i in (1, 2)]
    eager = [c.run(splits=1) for c in cases]
    torch.cuda.synchronize()
    graphs, outs, held = [], [], [c.q.clone() for c in cases]
    for c, q in zip(cases, held):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.q.copy_(q)
            outs.append(c.run(splits=1))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for c in cases:
        c.q.zero_()
    torch.cuda.synchronize()
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (o, l), (eo, el) in zip(outs, eager):
        assert torch.equal(o, eo) and torch.equal(l, el)


def test_written_then_attended_without_a_pause():
    """A prompt written and attended over in one stream, again and again with other
    contents: every call sees the writes before it."""
    B, T, Hq, Hkv, L, D = 4, 32, 16, 2, 400, 128
    g = torch.Generator(device="cuda").manual_seed(9)
    c = Case("bf16+e4m3", B, T, Hq, Hkv, L, D)
    ks, vs = c.scales["k_scale"], c.scales["v_scale"]
    start = ints([0] * B)
    prompts = [[torch.randn(B, Hkv, L, D, generator=g, device="cuda").to(torch.bfloat16) for _ in "kv"] for _ in range(6)]
    got, wholes = [], []
    for k, v in prompts:
        lm.kv_quantize_(c.k, c.v, ks, vs, k, v, start)
        got.append(c.run(splits=1))
        got.append(c.run(splits=3))
        wholes.append([c.whole("k"), c.whole("v")])
    torch.cuda.synchronize()
    for i, (k, v) in enumerate(wholes):
        ref = attention(c.q, k, v, c.kd, c.vd, c.tree)
        for o, l in got[2 * i:2 * i + 2]:
            check(o, l, ref, c.wt)
