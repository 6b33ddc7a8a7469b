"""Attention over an e4m3 cache and over a cache plus drafted tokens, against
the 64-bit forms of kv_util, whose docstring derives the bounds."""
import math

import pytest
import torch

import lse_weighted_merge_b200 as lm
from kv_util import FP8, attention, check, fp8_cache, store

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Case:
    """Inputs of one call: kind "bf16", "f16" (a cache of q's type), "bf16+e4m3", "f16+e4m3"."""

    def __init__(self, kind, B, T, Hq, Hkv, L, D, layout="bhl", seed=0, tree="tree"):
        g = torch.Generator(device="cuda").manual_seed(seed + 7 * L + T)
        dt = DT[kind.split("+")[0]]
        # the weights' types: over a cache its products' (f16 for e4m3), over
        # the drafts, which are of q's type, q's; where both occur the coarser
        self.wt_cache = torch.float16 if "e4m3" in kind or kind == "f16" else torch.bfloat16
        self.wt = dt

        def values(n):
            x = torch.randn(B, Hkv, n, D, generator=g, device="cuda")
            return x * torch.exp2(torch.randint(-3, 3, (B, Hkv, n, 1), generator=g, device="cuda").float())

        k, v = values(L), values(L)
        self.scales = {}
        if "e4m3" in kind:
            self.k, ks = fp8_cache(k, layout)
            self.v, vs = fp8_cache(v, layout)
            self.scales = dict(k_scale=ks, v_scale=vs)
        else:
            self.k, self.v = store(k.to(dt), layout), store(v.to(dt), layout)
        self.q = torch.randn(B, T, Hq, D, generator=g, device="cuda").to(dt)
        self.kd, self.vd = store(values(T).to(dt), layout), store(values(T).to(dt), layout)
        r = torch.rand(B, T, generator=g, device="cuda").cpu()
        if tree == "tree":
            parents = [[-1 if t == 0 or r[b, t] < 0.1 else int(r[b, t] * t) for t in range(T)] for b in range(B)]
            self.tree = lm.tree_mask(parents)
        else:   # any bits, not a tree; row 0 sees no draft
            self.tree = torch.randint(-2 ** 62, 2 ** 62, (B, T), generator=g, device="cuda") * 2
            self.tree[:, 0] = 0

    def whole(self, name):
        x = getattr(self, name).double()
        return x * self.scales[name + "_scale"].double()[..., None] if self.scales else x

    def ref(self, drafts=True, scale=None, **kw):
        d = (self.kd, self.vd, self.tree) if drafts else (None, None, None)
        return attention(self.q, self.whole("k"), self.whole("v"), *d, scale=scale, **kw)

    def run(self, drafts=True, **kw):
        d = (self.kd, self.vd, self.tree) if drafts else (None, None, None)
        return lm.tree_attention(self.q, self.k, self.v, *d, **self.scales, **kw)

    def check(self, drafts=True, what="", kv_len=None, draft_len=None, scale=None, **kw):
        out, lse = self.run(drafts, kv_len=kv_len, draft_len=draft_len, scale=scale, **kw)
        torch.cuda.synchronize()
        return check(out, lse, self.ref(drafts, scale, kv_len=kv_len, draft_len=draft_len),
                     self.wt if drafts else self.wt_cache, what)


KINDS = ["bf16", "f16", "bf16+e4m3", "f16+e4m3"]
SHAPES = [  # B, T, Hq, Hkv, L, D
    (1, 1, 1, 1, 1, 64),        # one key, one draft
    (2, 5, 8, 2, 300, 128),
    (3, 64, 4, 4, 77, 64),      # the widest tree, one head per group
    (1, 64, 16, 1, 130, 128),   # 1024 query rows
    (2, 7, 6, 3, 33, 64),
    (2, 13, 12, 4, 5, 128),     # fewer cached keys than drafts
    (1, 16, 32, 8, 513, 128),
    (1, 17, 15, 1, 1000, 64),   # 255 rows
    (2, 3, 16, 2, 64, 128),
    (1, 33, 4, 1, 129, 128),    # 132 rows
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_tree_matches(shape, kind):
    Case(kind, *shape).check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("R", [1, 2, 3, 8, 64])
@pytest.mark.parametrize("shape", [(2, 4, 8, 2, 700, 128), (1, 40, 8, 2, 50, 64)], ids=str)
def test_split_counts(shape, R, kind):
    """One shard, odd counts, more shards than keys."""
    Case(kind, *shape, layout="blh").check(splits=R)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [3, 24])
def test_uneven_lengths_and_padding(kind, T):
    B = 8
    c = Case(kind, B, T, 8, 2, 200, 128, layout="blh")
    kv_len = ints([0, 1, 200, 63, 64, 65, 500, -3])
    draft_len = ints([T, 0, 1, T, 2, T - 1, T + 9, -1])
    for splits in (None, 1, 3):
        c.check(kv_len=kv_len, draft_len=draft_len, splits=splits)
        c.check(drafts=False, kv_len=kv_len, draft_len=draft_len, splits=splits)
    out, lse = c.run(kv_len=kv_len, draft_len=draft_len)
    assert bool((out[1] == 0).all()) and bool((lse[1] == -math.inf).all())
    assert bool((out[2, 1:] == 0).all()) and bool((lse[2, 1:] == -math.inf).all())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [2, 31])
def test_rows_that_see_nothing(kind, T):
    """Masks that are no trees: a row without drafts, and without cached keys."""
    c = Case(kind, 2, T, 8, 2, 90, 64, tree="any")
    kv_len = ints([0, 90])
    c.check(kv_len=kv_len)
    out, lse = c.run(kv_len=kv_len)
    assert bool((out[0, 0] == 0).all()) and bool((lse[0, 0] == -math.inf).all())
    assert bool(torch.isfinite(lse[1]).all())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [4, 40])
def test_nan_and_inf_in_places_not_seen(kind, T):
    """Cache rows behind the length, padded drafts, and drafts that some rows
    do not see hold NaN and infinities; rows that do not see them are exact."""
    c = Case(kind, 3, T, 8, 2, 150, 128)
    kv_len, draft_len = ints([100, 0, 149]), ints([T, T - 1, T])
    nan = torch.tensor(math.nan, device="cuda")
    for b, n in ((0, 100), (1, 0), (2, 149)):
        for x in (c.k, c.v):
            x[b, :, n:] = nan.to(x.dtype)
        for s in c.scales.values():
            s[b, :, n:] = nan
    c.kd[1, :, T - 1], c.vd[1, :, T - 1] = math.nan, math.inf
    bad = T // 2      # a draft only it and its descendants see
    clean = c.ref(kv_len=kv_len, draft_len=draft_len)
    c.kd[0, :, bad] = math.nan
    c.vd[0, :, bad, ::3] = math.inf
    c.vd[2, :, bad, 5], c.vd[2, :, bad, 7] = -math.inf, math.nan
    out, lse = c.run(kv_len=kv_len, draft_len=draft_len)
    torch.cuda.synchronize()
    sees = (c.tree >> bad & 1).bool()
    sees[1] = False
    want = [torch.where(sees[..., None, None] if x.dim() == 4 else sees[..., None], torch.zeros_like(x), x) for x in clean]
    got = torch.where(sees[..., None, None], torch.zeros_like(out), out)
    gl = torch.where(sees[..., None], torch.zeros_like(lse), lse)
    check(got, gl, want, c.wt)
    s0, s2 = sees[0], sees[2]
    assert bool(torch.isnan(out[0][s0]).all()) and bool(torch.isnan(lse[0][s0]).all())
    assert bool((out[2][s2][..., 5] == -math.inf).all()) and bool(torch.isnan(out[2][s2][..., 7]).all())
    assert bool(torch.isfinite(out[2][s2][..., 6]).all()) and bool(torch.isfinite(lse[2][s2]).all())


@pytest.mark.parametrize("kind", KINDS)
def test_large_scores_and_unequal_scales(kind):
    """Scores far apart (one key takes nearly all the weight, first or last),
    and values whose sizes differ by many powers of two (past f16's range, so
    the output is fp32)."""
    for T in (2, 20):
        c = Case(kind, 2, T, 8, 2, 400, 64)
        for b, at in ((0, 3), (1, 398)):
            if not c.scales:
                c.k[b, :, at] *= 3
            else:
                c.scales["v_scale"][b, :, at] *= 2.0 ** 20
                c.scales["v_scale"][b, :, 50:90] *= 2.0 ** -30
                c.scales["k_scale"][b, :, at] *= 8
        c.check(scale=0.7, out_dtype=torch.float32)
        c.check(scale=-0.3, out_dtype=torch.float32)
        c.check(scale=0.0, out_dtype=torch.float32)


def test_tiny_and_huge_queries():
    """bf16 queries outside f16's range over an e4m3 cache."""
    for T in (1, 20):
        c = Case("bf16+e4m3", 2, T, 8, 2, 100, 128)
        c.q[0] *= 2.0 ** 60
        c.q[1] *= 2.0 ** -90
        c.scales["k_scale"][0] *= 2.0 ** -60
        c.scales["k_scale"][1] *= 2.0 ** 90
        c.check()


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("kind", KINDS)
def test_output_types_and_one_tree_for_all(kind, out_dtype):
    for T in (3, 33):
        c = Case(kind, 3, T, 8, 4, 90, 128)
        c.tree = c.tree[0].contiguous()
        out, lse = c.run(out_dtype=out_dtype)
        assert out.dtype == out_dtype
        check(out, lse, c.ref(), c.wt)
        out, lse = c.run(drafts=False, out_dtype=out_dtype, splits=1)
        check(out, lse, c.ref(drafts=False), c.wt_cache)


DECODE = [  # B, Hq, Hkv, L, D, splits
    (1, 1, 1, 1, 64, None), (2, 16, 1, 4097, 128, None), (5, 6, 2, 333, 64, 3), (1, 8, 8, 31, 128, 64),
    (96, 8, 2, 150, 128, 1), (3, 14, 2, 1000, 64, None), (2, 32, 8, 32, 128, 2),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("B,Hq,Hkv,L,D,splits", DECODE)
def test_decode_fp8(B, Hq, Hkv, L, D, splits, dtype):
    c = Case(dtype + "+e4m3", B, 1, Hq, Hkv, L, D, layout="blh")
    kv_len = ints([(37 * b + L) % (L + 1) for b in range(B)])
    for n in (None, kv_len):
        out, lse = lm.decode_attention_fp8(c.q[:, 0], c.k, c.v, **c.scales, kv_len=n, splits=splits)
        assert out.shape == (B, Hq, D) and lse.shape == (B, Hq)
        check(out[:, None], lse[:, None], c.ref(drafts=False, kv_len=n), c.wt_cache)


def test_shards_of_a_cache_merge_to_the_whole():
    """Two halves of a cache, the drafts with the second: their partials merge()
    to the attention over all of it."""
    c = Case("bf16", 2, 9, 8, 2, 300, 128)
    a, al = lm.tree_attention(c.q, c.k[:, :, :170], c.v[:, :, :170], out_dtype=torch.float32)
    b, bl = lm.tree_attention(c.q, c.k[:, :, 170:], c.v[:, :, 170:], c.kd, c.vd, c.tree, out_dtype=torch.float32)
    o, lse = lm.merge(torch.stack([a, b]).flatten(1, 2), torch.stack([al, bl]).flatten(1, 2), layout="rbhd",
                      out_dtype=torch.bfloat16)
    check(o.view(2, 9, 8, 128), lse.view(2, 9, 8), c.ref(), c.wt)


@pytest.mark.parametrize("cache", ["16 bits", "8 bits"])
def test_a_drafting_loop(cache):
    """Prompt written, then rounds of: tree attention over the cache and the
    drafts, an accepted path appended, a decode step.  A 16-bit copy of the cache
    is kept in step; after every round the attention agrees with 64 bits."""
    B, Hkv, G, L, D, T = 3, 2, 4, 96, 64, 12
    g = torch.Generator(device="cuda").manual_seed(5)

    def rnd(*s):
        return torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)

    kc, vc = (torch.zeros(B, Hkv, L, D, device="cuda").to(FP8) for _ in range(2))
    ks, vs = torch.zeros(B, Hkv, L, device="cuda"), torch.zeros(B, Hkv, L, device="cuda")
    kv_len = ints([0, 17, 40])
    prompt = rnd(B, Hkv, 40, D), rnd(B, Hkv, 40, D)
    lm.kv_quantize_(kc, vc, ks, vs, *prompt, ints([0, 0, 0]), count=kv_len)
    for rnd_no in range(3):
        parents = [[-1] + [max(0, t - 1 - (t + b + rnd_no) % 3) for t in range(1, T)] for b in range(B)]
        tree = lm.tree_mask(parents)
        q, kd, vd = rnd(B, T, Hkv * G, D), rnd(B, Hkv, T, D), rnd(B, Hkv, T, D)
        whole = [c.double() * s.double()[..., None] for c, s in ((kc, ks), (vc, vs))]
        if cache == "8 bits":
            out, lse = lm.tree_attention(q, kc, vc, kd, vd, tree, k_scale=ks, v_scale=vs, kv_len=kv_len)
        else:   # the same numbers in 16 bits (exact: 4 bits each)
            k16, v16 = lm.kv_dequantize(kc, vc, ks, vs, ints([0] * B), L, count=kv_len)
            out, lse = lm.tree_attention(q, k16, v16, kd, vd, tree, kv_len=kv_len)
        check(out, lse, attention(q, *whole, kd, vd, tree, kv_len=kv_len), torch.bfloat16)
        paths = []
        for b in range(B):   # the path to the last draft, from its root
            path, t = [], T - 1
            while t >= 0:
                path.append(t)
                t = parents[b][t]
            paths.append(path[::-1])
        n = ints([len(p) for p in paths])
        select = ints([p + [-1] * (T - len(p)) for p in paths])
        lm.kv_quantize_(kc, vc, ks, vs, kd, vd, kv_len, count=n, select=select)
        kv_len = kv_len + n
        q1 = rnd(B, Hkv * G, D)
        out, lse = lm.decode_attention_fp8(q1, kc, vc, ks, vs, kv_len=kv_len)
        whole = [c.double() * s.double()[..., None] for c, s in ((kc, ks), (vc, vs))]
        check(out[:, None], lse[:, None], attention(q1[:, None], *whole, kv_len=kv_len), torch.float16)


@pytest.mark.parametrize("kind", ["bf16", "f16+e4m3"])
@pytest.mark.parametrize("T", [4, 48])
def test_graphs_and_streams(kind, T):
    """Captured calls replay to the eager bits on new inputs; two graphs
    captured on one stream replay at the same time on two others."""
    a, b = Case(kind, 2, T, 8, 2, 600, 128, seed=1), Case(kind, 2, T, 8, 2, 600, 128, seed=2)
    eager = [c.run() for c in (a, b)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graphs, outs = [], []
    for c in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(c.run())
        graphs.append(g)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        with torch.cuda.stream(s1):
            graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
    torch.cuda.synchronize()
    for (o, l), (eo, el) in zip(outs, eager):
        assert torch.equal(o, eo) and torch.equal(l, el)
    a.q.copy_(b.q)      # a graph reads its inputs anew
    graphs[0].replay()
    want = a.run()
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], want[0]) and torch.equal(outs[0][1], want[1])
    with torch.cuda.stream(s1):
        o1 = a.run()
    with torch.cuda.stream(s2):
        o2 = b.run()
    torch.cuda.synchronize()
    assert torch.equal(o1[0], want[0]) and torch.equal(o2[0], eager[1][0])


def test_a_step_in_one_graph():
    """Append one token and attend, captured together: each replay reads the
    position anew."""
    B, Hq, Hkv, L, D = 2, 8, 2, 64, 128
    c = Case("bf16+e4m3", B, 1, Hq, Hkv, L, D)
    k, v = torch.empty_like(c.kd), torch.empty_like(c.vd)
    q, pos, n = torch.empty_like(c.q[:, 0]), ints([0, 0]), ints([0, 0])
    ks, vs = c.scales["k_scale"], c.scales["v_scale"]

    def step():
        lm.kv_quantize_(c.k, c.v, ks, vs, k, v, pos)
        return lm.decode_attention_fp8(q, c.k, c.v, ks, vs, kv_len=n)

    g = torch.cuda.CUDAGraph()
    k.normal_(), v.normal_(), q.normal_()
    step()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        out, lse = step()
    for i in range(5):
        k.normal_(), v.normal_(), q.normal_()
        pos.fill_(10 * i)
        n.copy_(pos + 1)
        g.replay()
        torch.cuda.synchronize()
        check(out[:, None], lse[:, None], attention(q[:, None], c.whole("k"), c.whole("v"), kv_len=n), c.wt_cache)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [5, 64])
def test_outputs_in_bounds_and_inputs_untouched(kind, T):
    """Outputs and workspace carved out of guarded buffers; a graph-free raw call."""
    from lse_weighted_merge_b200 import _native as nat
    B, Hq, Hkv, L, D, R = 2, 8, 2, 130, 64, 3
    c = Case(kind, B, T, Hq, Hkv, L, D)
    fp8 = bool(c.scales)
    keep = [x.clone() for x in (c.q, c.k.view(torch.uint8) if fp8 else c.k, c.kd, c.tree)]
    need = nat.tree_workspace_bytes(B, T, Hq, D, R, True)
    sizes = [B * T * Hq * D * 2, B * T * Hq * 4, need]
    bufs = [torch.full((4096 + n + 4096,), 0x3C, dtype=torch.uint8, device="cuda") for n in sizes]
    code = nat.BF16 if c.q.dtype == torch.bfloat16 else nat.F16
    st = c.scales.get("k_scale"), c.scales.get("v_scale")
    nat.tree_raw((c.q.data_ptr(), c.k.data_ptr(), c.v.data_ptr(), st[0].data_ptr() if fp8 else 0,
                  st[1].data_ptr() if fp8 else 0, c.kd.data_ptr(), c.vd.data_ptr(), c.tree.data_ptr(), 0, 0,
                  *(x.data_ptr() + 4096 for x in bufs), need, *c.q.stride()[:3], *c.k.stride()[:3], *c.v.stride()[:3],
                  *(st[0].stride() if fp8 else (0, 0, 0)), *(st[1].stride() if fp8 else (0, 0, 0)),
                  *c.kd.stride()[:3], *c.vd.stride()[:3], T, B, T, Hq, Hkv, L, D, R, code,
                  nat.E4M3 if fp8 else code, code, 1 / math.sqrt(D), 0), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    for x, n in zip(bufs, sizes):
        assert bool((x[:4096] == 0x3C).all()) and bool((x[4096 + n:] == 0x3C).all())
    out = bufs[0][4096:4096 + sizes[0]].view(c.q.dtype).view(B, T, Hq, D)
    lse = bufs[1][4096:4096 + sizes[1]].view(torch.float32).view(B, T, Hq)
    check(out, lse, c.ref(), c.wt)
    for x, y in zip(keep, (c.q, c.k.view(torch.uint8) if fp8 else c.k, c.kd, c.tree)):
        assert torch.equal(x, y)


def test_refusals():
    c = Case("bf16+e4m3", 2, 4, 8, 2, 50, 64)
    d = Case("bf16", 2, 4, 8, 2, 50, 64)
    sc = c.scales
    for call in (
            lambda: lm.tree_attention(c.q, c.k, c.v, c.kd, c.vd, c.tree),                       # no scales
            lambda: lm.tree_attention(d.q, d.k, d.v, d.kd, d.vd, d.tree, **sc),                  # scales without e4m3
            lambda: lm.tree_attention(d.q, d.k, d.v, d.kd, d.vd),                                # no tree
            lambda: lm.tree_attention(d.q, d.k, d.v, None, None, d.tree),
            lambda: lm.tree_attention(d.q, d.k, d.v, d.kd, d.vd, d.tree.int()),
            lambda: lm.tree_attention(d.q, d.k, d.v, d.kd, d.vd, d.tree[:1]),
            lambda: lm.tree_attention(d.q, d.k, d.v, d.kd[:, :, :3], d.vd, d.tree),
            lambda: lm.tree_attention(d.q, d.k.half(), d.v.half(), d.kd, d.vd, d.tree),
            lambda: lm.tree_attention(d.q, d.k, d.v, d.kd, d.vd, d.tree, kv_len=ints([1, 2]).long()),
            lambda: lm.tree_attention(d.q, d.k, d.v, d.kd, d.vd, d.tree, draft_len=ints([1])),
            lambda: lm.tree_attention(d.q, d.k, d.v, d.kd, d.vd, d.tree.cpu()),
            lambda: lm.tree_attention(d.q[:, 0], d.k, d.v),
            lambda: lm.tree_attention(d.q.transpose(2, 3), d.k, d.v),
            lambda: lm.decode_attention_fp8(d.q[:, 0], d.k, d.v, sc["k_scale"], sc["v_scale"]),
            lambda: lm.decode_attention_fp8(c.q[:, 0], c.k, c.v, sc["k_scale"], sc["v_scale"].half()),
            lambda: lm.decode_attention_fp8(c.q, c.k, c.v, **sc),
    ):
        with pytest.raises((ValueError, TypeError)):
            call()
    with pytest.raises(lm.LseMergeError):      # 65 drafts
        q = torch.zeros(1, 65, 2, 64, dtype=torch.bfloat16, device="cuda")
        lm.tree_attention(q, d.k[:1, :, :], d.v[:1])
    with pytest.raises(lm.LseMergeError):      # heads that do not divide
        lm.tree_attention(d.q[:, :, :3], d.k, d.v)
    torch.cuda.synchronize()
