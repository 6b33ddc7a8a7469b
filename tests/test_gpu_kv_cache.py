"""The 8-bit cache on the GPU: rows quantised as they are written and read
back, against the definition in 64 bits.  The scale is a power of two, so the
codes, the scales and the values read back in fp32 are exact and compared for
equality; 16-bit reads round once."""
import math

import pytest
import torch

import lse_weighted_merge_b200 as lm
from kv_util import FP8, U, fp8_cache, quantised, store

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def rows(B, H, T, D, dtype, seed, layout="bhl"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(B, H, T, D, generator=g, device="cuda")
    x *= torch.exp2(torch.randint(-9, 9, (B, H, T, 1), generator=g, device="cuda").float())
    return store(x.to(DT[dtype]), layout)


def cache(B, H, L, D, seed, layout="bhl"):
    """A cache that holds something already: (codes, scale)."""
    return fp8_cache(rows(B, H, L, D, "f32", seed), layout)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def expect(old, old_scale, x, start, count, select):
    """The cache after the write, in 64 bits: (codes, scale)."""
    codes, scale = old.double(), old_scale.double()
    B, _, L, _ = codes.shape
    T = x.shape[2] if select is None else select.shape[1]
    c, s = quantised(x)
    for b in range(B):
        for j in range(T):
            pos = int(start[b]) + j
            src = j if select is None else int(select[b, j])
            if 0 <= pos < L and (count is None or j < int(count[b])) and 0 <= src < x.shape[2]:
                codes[b, :, pos] = c[b, :, src]
                scale[b, :, pos] = s[b, :, src]
    return codes, scale


def write_and_check(k, v, L, start, count=None, select=None, layout="bhl"):
    B, H, _, D = k.shape
    kc, ks = cache(B, H, L, D, 1, layout)
    vc, vs = cache(B, H, L, D, 2, layout)
    want = [expect(c, s, x, start, count, select) for c, s, x in ((kc, ks, k), (vc, vs, v))]
    got = lm.kv_quantize_(kc, vc, ks, vs, k, v, start, count=count, select=select)
    assert got[0] is kc and got[3] is vs
    torch.cuda.synchronize()
    for (codes, scale), c, s in zip(want, (kc, vc), (ks, vs)):
        assert torch.equal(s.double(), scale)
        assert bool(((c.double() == codes) | (torch.isnan(c.double()) & torch.isnan(codes))).all())
    return kc, vc, ks, vs


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("B,H,T,L,layout", [
    (1, 1, 1, 1, "bhl"), (3, 2, 1, 40, "blh"), (2, 5, 77, 80, "bhl"), (4, 3, 33, 50, "blh"), (70, 8, 1, 9, "bhl")])
def test_write_matches_the_definition(B, H, T, L, layout, dtype, D):
    k, v = rows(B, H, T, D, dtype, 3, layout), rows(B, H, T, D, dtype, 4, layout)
    start = ints([(5 * b) % (L - T + 1) for b in range(B)])
    write_and_check(k, v, L, start, layout=layout)


def test_write_counts_positions_and_selection():
    B, H, S, D, L = 6, 2, 9, 128, 30
    k, v = rows(B, H, S, D, "bf16", 5), rows(B, H, S, D, "bf16", 6)
    # before, across both ends, behind the cache; counts of none, some, all, more
    start = ints([-4, 25, 0, 30, 2 ** 31 - 1, -2 ** 31])
    write_and_check(k, v, L, start)
    write_and_check(k, v, L, ints([0, 3, 21, 5, 7, 9]), count=ints([0, 1, 9, 100, -3, 4]))
    # the accepted path of a tree: any rows, some twice, some out of range
    sel = ints([[0, 3, 8, 3], [8, 8, 8, 8], [-1, 2, 9, 1], [0, 1, 2, 3], [5, 4, 3, 2], [7, 0, 2 ** 31 - 1, -2 ** 31]])
    write_and_check(k, v, L, ints([0, 3, 21, 28, 7, 9]), count=ints([4, 2, 4, 3, 0, 4]), select=sel)
    write_and_check(k, v, L, ints([0, 3, 21, 28, 7, 9]), select=ints([[i % 9 for i in range(17)]] * 6))


def test_write_special_values():
    D = 64
    x = torch.zeros(1, 1, 12, D, device="cuda")
    inf, nan = math.inf, math.nan
    x[0, 0, 1] = 448.0                      # exactly the largest code
    x[0, 0, 2, :3] = torch.tensor([inf, -inf, nan])
    x[0, 0, 3] = nan                        # no finite element
    x[0, 0, 4] = torch.linspace(-3.3e38, 3.3e38, D)
    x[0, 0, 5] = 1e-41                      # subnormal
    x[0, 0, 6] = torch.finfo(torch.float32).tiny
    x[0, 0, 7] = -0.0
    x[0, 0, 8, 0], x[0, 0, 8, 1] = 1.0, 2.0 ** -17   # below half a step of the smallest code
    x[0, 0, 9] = torch.arange(D) / 16 + 27   # ties
    x[0, 0, 10, 5] = 449.0                  # one step above: the next power of two
    x[0, 0, 11, 9] = 2.0 ** -140
    start = ints([0])
    kc, vc, ks, vs = write_and_check(x, -x, 12, start)
    assert ks[0, 0, 0] == 1 and ks[0, 0, 1] == 1 and ks[0, 0, 10] == 2 and ks[0, 0, 3] == 1
    assert bool(torch.isnan(kc[0, 0, 3].float()).all()) and int(torch.isnan(kc[0, 0, 2].float()).sum()) == 3


def test_values_read_back_and_written_again_stay():
    """What is read back (in fp32 or bf16: codes have 4 bits) and written again
    stands for the same values.  The bytes may differ: a row whose largest
    element was rounded down to 224 * scale now fits half that scale, which
    holds the same values as codes twice as large."""
    B, H, T, D = 2, 3, 50, 128
    k, v = rows(B, H, T, D, "bf16", 7), rows(B, H, T, D, "bf16", 8)
    start = ints([0, 0])
    first = write_and_check(k, v, T, start)
    for dtype in (torch.float32, torch.bfloat16):
        rk, rv = lm.kv_dequantize(*first, start, T, dtype=dtype)
        again = [torch.zeros_like(t) for t in first]
        lm.kv_quantize_(*again, rk, rv, start)
        for x, y in zip((rk, rv), lm.kv_dequantize(*again, start, T, dtype=dtype)):
            assert torch.equal(x, y)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("layout", ["bhl", "blh"])
def test_read_back(layout, dtype, D):
    B, H, L, T = 5, 3, 61, 23
    kc, ks = cache(B, H, L, D, 11, layout)
    vc, vs = cache(B, H, L, D, 12, layout)
    start, count = ints([0, 38, 55, -7, 61]), ints([23, 5, 23, 23, 9])
    for cnt in (None, count):
        k, v = lm.kv_dequantize(kc, vc, ks, vs, start, T, count=cnt, dtype=DT[dtype])
        for got, c, s in ((k, kc, ks), (v, vc, vs)):
            want = torch.zeros(B, H, T, D, dtype=torch.float64, device="cuda")
            for b in range(B):
                for j in range(T):
                    pos = int(start[b]) + j
                    if 0 <= pos < L and (cnt is None or j < int(cnt[b])):
                        want[b, :, j] = c[b, :, pos].double() * s[b, :, pos].double()[..., None]
            assert got.shape == want.shape and got.dtype == DT[dtype] and got.is_contiguous()
            tiny = 2.0 ** -25 if dtype == "f16" else 0.0     # half of f16's smallest step
            assert bool(((got.double() - want).abs() <= U[DT[dtype]] * want.abs() + tiny).all())
            if dtype != "f16":   # codes times a power of two have 4 significant bits
                assert torch.equal(got.double(), want)


def test_keys_and_values_interleaved_in_one_buffer():
    """k and v of a token side by side (views of one buffer), and rows of a fused projection."""
    B, H, L, D, T = 2, 4, 20, 64, 6
    buf = torch.zeros(B, L, 2, H, D, device="cuda").to(FP8)
    kc, vc = (buf[:, :, i].permute(0, 2, 1, 3) for i in (0, 1))
    ks, vs = torch.zeros(B, H, L, device="cuda"), torch.zeros(B, H, L, device="cuda")
    qkv = rows(B, T, 3 * H, D, "bf16", 21)   # [B, T, 3H, D]
    k, v = qkv[:, :, H:2 * H].permute(0, 2, 1, 3), qkv[:, :, 2 * H:].permute(0, 2, 1, 3)
    lm.kv_quantize_(kc, vc, ks, vs, k, v, ints([3, 14]))
    for c, s, x in ((kc, ks, k), (vc, vs, v)):
        codes, scale = expect(torch.zeros_like(c), torch.zeros_like(s), x, [3, 14], None, None)
        assert torch.equal(c.double(), codes) and torch.equal(s.double(), scale)


def test_empty_calls():
    kc, ks = cache(2, 1, 8, 64, 1)
    vc, vs = cache(2, 1, 8, 64, 2)
    before = kc.view(torch.uint8).clone()
    none = torch.zeros(2, 1, 0, 64, dtype=torch.bfloat16, device="cuda")
    lm.kv_quantize_(kc, vc, ks, vs, none, none, ints([0, 0]))
    assert torch.equal(kc.view(torch.uint8), before)
    k, v = lm.kv_dequantize(kc, vc, ks, vs, ints([0, 0]), 0)
    assert k.shape == v.shape == (2, 1, 0, 64)


def test_refusals():
    kc, ks = cache(2, 2, 8, 64, 1)
    vc, vs = cache(2, 2, 8, 64, 2)
    k = rows(2, 2, 3, 64, "bf16", 1)
    st = ints([0, 0])
    for bad in (dict(k=k[:1]), dict(k=k.transpose(2, 3)), dict(v=k.float()), dict(start=st.long()), dict(start=st[:1]),
                dict(count=st.float()), dict(select=st), dict(start=None), dict(start=st.cpu()), dict(ks=ks[:, :1]),
                dict(vc=vc.float()), dict(ks=ks.double())):
        a = dict(kc=kc, vc=vc, ks=ks, vs=vs, k=k, v=k, start=st, count=None, select=None)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            lm.kv_quantize_(a["kc"], a["vc"], a["ks"], a["vs"], a["k"], a["v"], a["start"], count=a["count"],
                            select=a["select"])
    with pytest.raises(lm.LseMergeError):      # one address for every token
        lm.kv_quantize_(kc[:, :, :1].expand(2, 2, 8, 64), vc, ks, vs, k, k, st)
    with pytest.raises(lm.LseMergeError):      # the same tensor for keys and values
        lm.kv_quantize_(kc, kc, ks, vs, k, k, st)
    with pytest.raises(ValueError):
        lm.kv_dequantize(kc, vc, ks, vs, st, -1)
    with pytest.raises(TypeError):
        lm.kv_dequantize(kc, vc, ks, vs, st, 2, dtype=torch.int32)
    torch.cuda.synchronize()


def test_offsets_past_32_bits():
    """Rows more than 4 GiB apart, in both directions."""
    L, D = 3, 128
    step = (1 << 32) + 4096
    buf = torch.zeros(2 * step + 2 * L * D, dtype=torch.uint8, device="cuda").view(FP8)
    kc = buf.as_strided((2, 1, L, D), (step, L * D, D, 1), 0)
    vc = buf.as_strided((2, 1, L, D), (step, L * D, D, 1), step // 2)
    ks, vs = torch.zeros(2, 1, L, device="cuda"), torch.zeros(2, 1, L, device="cuda")
    k, v = rows(2, 1, L, D, "bf16", 31), rows(2, 1, L, D, "bf16", 32)
    st = ints([0, 0])
    lm.kv_quantize_(kc, vc, ks, vs, k, v, st)
    rk, rv = lm.kv_dequantize(kc, vc, ks, vs, st, L, dtype=torch.float32)
    for got, x in ((rk, k), (rv, v)):
        c, s = quantised(x)
        assert torch.equal(got.double(), c * s[..., None])
    q = torch.randn(2, 4, D, device="cuda").to(torch.bfloat16)
    out, lse = lm.decode_attention_fp8(q, kc, vc, ks, vs)
    near, nl = lm.decode_attention_fp8(q, kc.contiguous(), vc.contiguous(), ks, vs)
    assert torch.equal(out, near) and torch.equal(lse, nl)
