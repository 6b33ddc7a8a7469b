"""The 8-bit cache's and the tree attention's argument checks, on the host:
rejected calls return before any CUDA call (the addresses are never read)."""
import pytest
import torch

import lse_weighted_merge_b200 as lm
from lse_weighted_merge_b200 import _native as nat

A = {n: 0x7f0000000000 + (i << 36) for i, n in enumerate(
    ("kc", "vc", "ks", "vs", "k", "v", "start", "count", "select", "q", "kd", "vd", "tree", "kv_len",
     "draft_len", "out", "lse", "ws"))}


def kv(write=True, **kw):
    B, H, L, D, T, S = (kw.pop(n, d) for n, d in (("B", 2), ("H", 3), ("L", 100), ("D", 64), ("T", 4), ("S", None)))
    S = T if S is None else S
    f = dict(kc=A["kc"], vc=A["vc"], ks=A["ks"], vs=A["vs"], k=A["k"], v=A["v"], start=A["start"], count=0, select=0,
             c=(H * L * D, L * D, D), s=(H * L, L, 1), x=(H * S * D, S * D, D), dtype=nat.BF16)
    f["cv"], f["sv"], f["xv"] = None, None, None
    f.update(kw)
    c2, s2, x2 = f["cv"] or f["c"], f["sv"] or f["s"], f["xv"] or f["x"]
    call = nat.kv_quantize_raw if write else nat.kv_dequantize_raw
    return call((f["kc"], f["vc"], f["ks"], f["vs"], f["k"], f["v"], f["start"], f["count"], f["select"], *f["c"], *c2,
                 *f["s"], *s2, *f["x"], *x2, B, H, L, D, T, S, f["dtype"], 0), 0, check=False)


@pytest.mark.parametrize("write", [True, False], ids=["quantize", "dequantize"])
@pytest.mark.parametrize("kw,code", [
    (dict(dtype=nat.E4M3), nat.EDTYPE), (dict(dtype=-1), nat.EDTYPE),
    (dict(B=0), nat.EDIMS), (dict(H=0), nat.EDIMS), (dict(L=0), nat.EDIMS), (dict(T=0), nat.EDIMS),
    (dict(S=5), nat.EDIMS), (dict(B=1 << 20, T=1 << 20), nat.EDIMS),
    (dict(D=96), nat.EUNSUP), (dict(D=32), nat.EUNSUP),
    (dict(kc=0), nat.ENULL), (dict(vs=0), nat.ENULL), (dict(k=0), nat.ENULL), (dict(start=0), nat.ENULL),
    (dict(c=(19200, -6400, 64)), nat.ESTRIDE), (dict(s=(300, 100, -1)), nat.ESTRIDE),
    (dict(kc=A["kc"] + 8), nat.EALIGN), (dict(v=A["v"] + 2), nat.EALIGN), (dict(ks=A["ks"] + 2), nat.EALIGN),
    (dict(start=A["start"] + 1), nat.EALIGN), (dict(c=(19208, 6400, 64)), nat.EALIGN),
    (dict(x=(768, 256, 60)), nat.EALIGN),
    (dict(k=A["kc"] + 64), nat.EALIAS), (dict(v=A["vs"]), nat.EALIAS),
    (dict(c=(1 << 62, 6400, 64)), nat.EDIMS),
])
def test_cache_refusals(write, kw, code):
    rc = kv(write, **kw)
    assert rc == code, (rc, nat.strerror(rc))


@pytest.mark.parametrize("kw,code", [
    (dict(vc=A["kc"]), nat.EALIAS), (dict(vs=A["ks"]), nat.EALIAS), (dict(ks=A["kc"] + 1024), nat.EALIAS),
    (dict(start=A["ks"]), nat.EALIAS), (dict(count=A["kc"]), nat.EALIAS), (dict(select=A["vc"]), nat.EALIAS),
    (dict(c=(19200, 6400, 0)), nat.ESTRIDE),      # every token at one address
    (dict(c=(6400, 6400, 64)), nat.ESTRIDE),      # sequences share their rows
    (dict(s=(300, 0, 1)), nat.ESTRIDE),
])
def test_quantize_refuses_overlapping_writes(kw, code):
    assert kv(True, **kw) == code


def test_dequantize_refusals_of_its_outputs():
    assert kv(False, v=A["k"]) == nat.EALIAS
    assert kv(False, start=A["k"]) == nat.EALIAS
    assert kv(False, x=(0, 256, 64)) == nat.ESTRIDE
    assert kv(False, select=A["select"]) == nat.EUNSUP


def tree(**kw):
    B, T, Hq, Hkv, L, D, R = (kw.pop(n, d) for n, d in (
        ("B", 2), ("T", 5), ("Hq", 8), ("Hkv", 2), ("L", 100), ("D", 64), ("R", 2)))
    f = dict(q=A["q"], k=A["kc"], v=A["vc"], ks=0, vs=0, kd=A["kd"], vd=A["vd"], tree=A["tree"], kv_len=0,
             draft_len=0, out=A["out"], lse=A["lse"], ws=A["ws"], ws_bytes=1 << 30,
             qs=(T * Hq * D, Hq * D, D), c=(Hkv * L * D, L * D, D), s=(Hkv * L, L, 1), d=(Hkv * T * D, T * D, D),
             tree_b=T, dtype=nat.BF16, cache=nat.BF16, out_dtype=nat.BF16, scale=0.125)
    f.update(kw)
    return nat.tree_raw((f["q"], f["k"], f["v"], f["ks"], f["vs"], f["kd"], f["vd"], f["tree"], f["kv_len"],
                         f["draft_len"], f["out"], f["lse"], f["ws"], f["ws_bytes"], *f["qs"], *f["c"], *f["c"],
                         *f["s"], *f["s"], *f["d"], *f["d"], f["tree_b"], B, T, Hq, Hkv, L, D, R, f["dtype"],
                         f["cache"], f["out_dtype"], f["scale"], 0), 0, check=False)


FP8 = dict(cache=nat.E4M3, ks=A["ks"], vs=A["vs"])


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), nat.EDTYPE), (dict(cache=4), nat.EDTYPE), (dict(out_dtype=3), nat.EDTYPE),
    (dict(T=0), nat.EDIMS), (dict(L=0), nat.EDIMS), (dict(R=0), nat.EDIMS), (dict(B=0), nat.EDIMS),
    (dict(R=70000), nat.EDIMS), (dict(B=70000), nat.EDIMS), (dict(scale=float("nan")), nat.EDIMS),
    (dict(scale=float("inf")), nat.EDIMS), (dict(ws_bytes=1000), nat.EDIMS),
    (dict(T=65), nat.EUNSUP), (dict(Hq=9), nat.EUNSUP), (dict(Hq=34), nat.EUNSUP), (dict(D=80), nat.EUNSUP),
    (dict(dtype=nat.F32, cache=nat.F32), nat.EUNSUP), (dict(cache=nat.F16), nat.EUNSUP),
    (dict(q=0), nat.ENULL), (dict(out=0), nat.ENULL), (dict(ws=0), nat.ENULL), (dict(tree=0), nat.ENULL),
    (dict(vd=0), nat.ENULL), (dict(cache=nat.E4M3), nat.ENULL), ({**FP8, "vs": 0}, nat.ENULL),
    (dict(qs=(2560, -512, 64)), nat.ESTRIDE), (dict(d=(640, 320, -64)), nat.ESTRIDE), (dict(tree_b=-1), nat.ESTRIDE),
    ({**FP8, "s": (200, 100, -1)}, nat.ESTRIDE),
    (dict(q=A["q"] + 8), nat.EALIGN), (dict(tree=A["tree"] + 4), nat.EALIGN), (dict(ws=A["ws"] + 8), nat.EALIGN),
    (dict(c=(12800, 6400, 68)), nat.EALIGN), ({**FP8, "c": (12800, 6400, 72)}, nat.EALIGN),
    (dict(kv_len=A["kv_len"] + 2), nat.EALIGN), (dict(d=(640, 324, 64)), nat.EALIGN),
    (dict(out=A["q"]), nat.EALIAS), (dict(ws=A["kc"]), nat.EALIAS), (dict(lse=A["ws"]), nat.EALIAS),
    (dict(lse=A["tree"]), nat.EALIAS), (dict(out=A["kd"]), nat.EALIAS), ({**FP8, "out": A["vs"]}, nat.EALIAS),
])
def test_tree_refusals(kw, code):
    rc = tree(**kw)
    assert rc == code, (rc, nat.strerror(rc))


def test_workspace_bytes():
    assert nat.tree_workspace_bytes(2, 5, 8, 64, 1, False) == 0
    rows = 2 * 5 * 8
    want = -(-rows * 4 * 64 * 4 // 256) * 256 + rows * 4 * 4
    assert nat.tree_workspace_bytes(2, 5, 8, 64, 3, True) == want == nat.tree_workspace_bytes(2, 5, 8, 64, 4, False)
    with pytest.raises(nat.LseMergeError):
        nat.tree_workspace_bytes(2, 0, 8, 64, 3, True)


def test_binding_rejects_a_struct_of_another_size():
    with pytest.raises(TypeError):
        nat._fast.tree_attention(b"123", 0)
    with pytest.raises(TypeError):
        nat._fast.kv_quantize(bytearray(248), 0)


def test_tree_mask():
    m = lm.tree_mask([-1, 0, 0, 1, -1], device="cpu")
    assert m.tolist() == [0b1, 0b11, 0b101, 0b1011, 0b10000]
    chain = lm.tree_mask([list(range(-1, 63))], device="cpu")
    assert chain.shape == (1, 64) and chain[0, 63] == -1 and chain[0, 62] == (1 << 63) - 1
    assert lm.tree_mask(torch.tensor([[-1], [-1]]), device="cpu").tolist() == [[1], [1]]
    for bad in ([0], [-1, 1], [-2], [list(range(-1, 64))]):
        with pytest.raises(ValueError):
            lm.tree_mask(bad, device="cpu")


def test_no_cpu_path():
    c = torch.zeros(1, 1, 16, 64).to(torch.float8_e4m3fn)
    s = torch.ones(1, 1, 16)
    x = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16)
    st = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        lm.kv_quantize_(c, c.clone(), s, s.clone(), x, x, st)
    with pytest.raises(ValueError, match="CUDA"):
        lm.kv_dequantize(c, c.clone(), s, s.clone(), st, 4)
    with pytest.raises(ValueError, match="CUDA"):
        lm.decode_attention_fp8(x[:, :, 0], c, c, s, s)
    with pytest.raises(TypeError):
        lm.kv_quantize_(x, x, s, s, x, x, st)
    with pytest.raises(ValueError):
        lm.kv_quantize_(c, c, s, s[:, :, :3], x, x, st)
