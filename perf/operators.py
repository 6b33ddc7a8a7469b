"""Measured cases of the 8-bit KV cache and the attention over it.

Four operators, as a serving loop with drafted tokens uses them around one KV
cache [B, Hkv, L, D]:

  write   quantise new keys and values into an e4m3 cache (one power-of-two
          scale per token and head), at each sequence's position
  read    read a stretch of such a cache back in 16 bits
  decode  one query token per sequence over the e4m3 cache
  tree    a tree of drafted query tokens per sequence over a cache (16-bit or
          e4m3) and over the drafts' own keys, each draft seeing the whole
          cache and the drafts its mask names

What write leaves in the cache is given back as it is held: e4m3 numbers and
their scales.  `run` computes them with elementary torch operations in 32 bits, or, where
`own` is true, through the framework's calls.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_ELEM = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}


def listed():
    return [
        # a decode step of 64 sequences appends one token each
        dict(name="write one token each", op="write", B=64, T=1, Hkv=8, L=512, D=128, dtype="bf16",
             layout="bhld", ragged=False, select=False),
        # a prefill of 16 prompts fills the cache
        dict(name="write prompts", op="write", B=16, T=4096, Hkv=8, L=4160, D=128, dtype="bf16",
             layout="bhld", ragged=False, select=False),
        # the accepted path of each drafted tree is appended, uneven counts,
        # cache stored token by token
        dict(name="write accepted drafts", op="write", B=33, T=27, Hkv=5, L=777, D=64, dtype="f16",
             layout="blhd", ragged=True, select=True),
        # whole prefixes go back to 16 bits, as for a copy to a 16-bit cache
        dict(name="read prefixes", op="read", B=16, T=4096, Hkv=8, L=4160, D=128, dtype="bf16",
             layout="bhld", ragged=False),
        # a few hundred tokens of some sequences, uneven counts
        dict(name="read some tokens", op="read", B=5, T=333, Hkv=3, L=1001, D=64, dtype="f16",
             layout="blhd", ragged=True),
        # one sequence at a time: latency counts
        dict(name="decode one sequence", op="decode", B=1, T=1, Hq=32, Hkv=8, L=4096, D=128, dtype="bf16",
             cache="e4m3", layout="bhld", ragged=False),
        # a full decode batch
        dict(name="decode a batch", op="decode", B=64, T=1, Hq=32, Hkv=8, L=4096, D=128, dtype="bf16",
             cache="e4m3", layout="bhld", ragged=False),
        # uneven lengths from empty to full, small heads
        dict(name="decode uneven", op="decode", B=13, T=1, Hq=18, Hkv=3, L=2777, D=64, dtype="f16",
             cache="e4m3", layout="blhd", ragged=True),
        # a short draft for one sequence: latency counts
        dict(name="tree of one sequence", op="tree", B=1, T=5, Hq=32, Hkv=8, L=4096, D=128, dtype="bf16",
             cache="bf16", layout="bhld", ragged=False),
        # an ordinary draft for a batch over a 16-bit cache
        dict(name="trees of a batch", op="tree", B=16, T=16, Hq=32, Hkv=8, L=4096, D=128, dtype="bf16",
             cache="bf16", layout="bhld", ragged=False),
        # the widest drafts over a long 8-bit cache
        dict(name="wide trees, 8-bit cache", op="tree", B=16, T=64, Hq=32, Hkv=8, L=8192, D=128, dtype="bf16",
             cache="e4m3", layout="bhld", ragged=False),
        # uneven lengths and drafts, small heads
        dict(name="trees uneven", op="tree", B=7, T=13, Hq=12, Hkv=4, L=1901, D=64, dtype="f16",
             cache="f16", layout="blhd", ragged=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    most = max((work(c) for c in listed()), key=lambda w: w["bytes"])["bytes"]
    most_flops = max(work(c)["flops"] for c in listed())
    while True:
        c = dict(op=rng.choice(["write", "read", "decode", "tree", "tree"]), B=_log(rng, 1, 96),
                 Hkv=_log(rng, 1, 16), L=_log(rng, 16, 16384), D=rng.choice([64, 128]),
                 dtype=rng.choice(["bf16", "f16"]), layout=rng.choice(["bhld", "blhd"]),
                 ragged=rng.random() < 0.5)
        if c["op"] in ("write", "read"):
            c["T"] = _log(rng, 1, c["L"])
            if c["op"] == "write":
                c["select"] = rng.random() < 0.5
        else:
            c["T"] = _log(rng, 1, 64) if c["op"] == "tree" else 1
            c["Hq"] = c["Hkv"] * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
            c["cache"] = rng.choice([c["dtype"], "e4m3"]) if c["op"] == "tree" else "e4m3"
        w = work(c)
        cache = 2 * c["B"] * c["Hkv"] * c["L"] * c["D"]
        if w["bytes"] <= most and w["flops"] <= most_flops and cache <= 1 << 28:
            return c


def _lens(case, most, least):
    """The lengths of the case's sequences, in order: all `most`, or spread from `least` to `most`."""
    n = case["B"]
    if not case["ragged"] or n == 1:
        return [most] * n
    return [least + (most - least) * i // (n - 1) for i in range(n)]


def work(case):
    B, T, Hkv, L, D = (case[k] for k in ("B", "T", "Hkv", "L", "D"))
    e = _ELEM[case["dtype"]]
    if case["op"] == "write":
        n = sum(_lens(case, T, 0)) * Hkv * 2
        return {"bytes": n * (D * e + D + 4) + 8 * B, "flops": 3 * n * D}
    if case["op"] == "read":
        n = sum(_lens(case, T, 0)) * Hkv * 2
        return {"bytes": n * (D + 4) + B * T * Hkv * 2 * D * e + 8 * B, "flops": n * D}
    Hq, c = case["Hq"], _ELEM[case["cache"]]
    lens, drafts = _lens(case, L, 0), _lens(case, T, 1)
    keys = sum(lens) * Hkv * 2 * (D * c + (4 if case["cache"] == "e4m3" else 0))
    rows = B * T * Hq
    own_keys = 2 * sum(drafts) * Hkv * D * e if case["op"] == "tree" else 0
    pairs = sum(t * n for t, n in zip(drafts, lens)) + (sum(drafts) if case["op"] == "tree" else 0)
    return {"bytes": keys + own_keys + rows * (2 * D * e + 4), "flops": 4 * pairs * Hq * D}


def _store(x, layout):
    """x [B, Hkv, L, D] as a user's cache of that layout: stored so, or token by token."""
    return x.contiguous() if layout == "bhld" else x.transpose(1, 2).contiguous().transpose(1, 2)


def _quantised(x):
    """(codes in e4m3, scale) of x [..., D]: the scale is the smallest power of two by which the row's
    largest magnitude fits e4m3's 448."""
    x = x.float()
    m, e = torch.frexp(x.abs().amax(-1))
    k = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
    k = torch.where(m == 0, torch.zeros_like(k), k)
    scale = torch.ldexp(torch.ones_like(m), k)
    return (x / scale[..., None]).to(torch.float8_e4m3fn), scale


def _values(g, *shape):
    """Keys or values: normal, some channels larger than others, some tokens larger than others."""
    x = torch.randn(shape, generator=g, device="cuda")
    x *= torch.exp(0.4 * torch.randn(shape[1], 1, shape[3], generator=g, device="cuda"))
    return x.mul_(torch.exp(0.3 * torch.randn(shape[0], shape[1], shape[2], 1, generator=g, device="cuda")))


def _trees(rng, B, T):
    """Ancestor masks [B, T] of random trees: bit j of word t is set where draft t sees draft j."""
    words = []
    for _ in range(B):
        row = []
        for t in range(T):
            parent = rng.randint(max(-1, t - 4), t - 1) if t else -1
            row.append((row[parent] if parent >= 0 else 0) | 1 << t)
        words.append([w - (1 << 64) if w >> 63 else w for w in row])
    return torch.tensor(words, dtype=torch.int64, device="cuda")


def prepare(case, seed):
    B, T, Hkv, L, D = (case[k] for k in ("B", "T", "Hkv", "L", "D"))
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    dt, layout = _TYPES[case["dtype"]], case["layout"]

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    def uneven(most, least):
        v = _lens(case, most, least)
        rng.shuffle(v)
        return v if case["ragged"] else None

    s = {"op": case["op"]}
    if case["op"] in ("write", "read"):
        count = uneven(T, 0)
        s["start"] = ints([rng.randint(0, L - T) for _ in range(B)])
        s["count"] = None if count is None else ints(count)
    for name in ("k", "v"):
        if case["op"] == "write":   # an empty cache, and the new tokens
            s[name] = _store(_values(g, B, Hkv, T, D).to(dt), layout)
            s[name + "_cache"] = _store(torch.zeros(B, Hkv, L, D, dtype=torch.float8_e4m3fn, device="cuda"), layout)
            s[name + "_scale"] = _store(torch.zeros(B, Hkv, L, 1, device="cuda"), layout)[..., 0]
        else:
            x = _values(g, B, Hkv, L, D)
            if case["op"] == "read" or case["cache"] == "e4m3":
                codes, scale = _quantised(x)
                s[name + "_cache"] = _store(codes, layout)
                s[name + "_scale"] = _store(scale[..., None], layout)[..., 0]
            else:
                s[name + "_cache"] = _store(x.to(dt), layout)
                s[name + "_scale"] = None
            del x
    if case["op"] == "write":
        s["select"] = ints([sorted(rng.sample(range(T), T)) if i % 2 else [rng.randrange(T) for _ in range(T)]
                            for i in range(B)]) if case["select"] else None
    if case["op"] == "read":
        s["length"], s["dtype"] = T, dt
    if case["op"] in ("decode", "tree"):
        lens = uneven(L, 0)
        s["kv_len"] = None if lens is None else ints(lens)
        q = 1.2 * torch.randn(B, T, case["Hq"], D, generator=g, device="cuda")
        s["q"] = q.to(dt) if case["op"] == "tree" else q[:, 0].to(dt)
    if case["op"] == "tree":
        drafts = uneven(T, 1)
        s["draft_len"] = None if drafts is None else ints(drafts)
        s["tree"] = _trees(rng, B, T)
        s["k_draft"] = _store(_values(g, B, Hkv, T, D).to(dt), layout)
        s["v_draft"] = _store(_values(g, B, Hkv, T, D).to(dt), layout)
    return s


def _places(s, T, L):
    """Of token j of each sequence: its position in the cache, and whether there is such a token."""
    j = torch.arange(T, device="cuda")
    pos = s["start"].long()[:, None] + j
    there = (pos >= 0) & (pos < L)
    if s["count"] is not None:
        there = there & (j < s["count"][:, None])
    return pos.clamp(0, L - 1), there


def _write(s):
    L = s["k_cache"].shape[2]
    T = s["k"].shape[2]
    pos, there = _places(s, T, L)
    b, j = there.nonzero(as_tuple=True)
    p = pos[b, j]
    src = j if s["select"] is None else s["select"].long()[b, j]
    for name in ("k", "v"):
        codes, scale = _quantised(s[name][b, :, src])
        s[name + "_cache"].view(torch.uint8)[b, :, p] = codes.view(torch.uint8)
        s[name + "_scale"][b, :, p] = scale
    return {n: s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")}


def _read(s):
    B, _, L, _ = s["k_cache"].shape
    pos, there = _places(s, s["length"], L)
    b = torch.arange(B, device="cuda")[:, None]
    out = {}
    for name in ("k", "v"):
        codes = s[name + "_cache"].view(torch.uint8)[b, :, pos].view(torch.float8_e4m3fn).float()   # [B, T, Hkv, D]
        x = codes * s[name + "_scale"][b, :, pos][..., None]
        x = torch.where(there[:, :, None, None], x, torch.zeros_like(x))
        out[name] = x.transpose(1, 2).to(s["dtype"])
    return out


def _whole(s, name, kind):
    """The cache's keys or values as numbers of type `kind`, [B, Hkv, L, D]."""
    x = s[name + "_cache"].to(kind)
    return x if s[name + "_scale"] is None else x * s[name + "_scale"].to(kind)[..., None]


def _attend(s):
    q = s["q"] if s["op"] == "tree" else s["q"][:, None]
    B, T, Hq, D = q.shape
    k, v = _whole(s, "k", torch.float32), _whole(s, "v", torch.float32)
    Hkv, L = k.shape[1:3]
    j = torch.arange(L, device="cuda")
    seen = torch.ones(B, T, L, dtype=torch.bool, device="cuda")
    if s["kv_len"] is not None:
        seen = seen & (j < s["kv_len"][:, None, None])
    if s["op"] == "tree":
        t = torch.arange(T, device="cuda")
        among = (s["tree"][:, :, None] >> t & 1).bool()
        if s["draft_len"] is not None:
            live = t < s["draft_len"][:, None]
            among = among & live[:, None, :] & live[:, :, None]
            seen = seen & live[:, :, None]
        seen = torch.cat([seen, among], 2)
        k = torch.cat([k, s["k_draft"].float()], 2)
        v = torch.cat([v, s["v_draft"].float()], 2)
    q = q.float().reshape(B, T, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    x = (q @ k.transpose(2, 3)).mul_(1 / math.sqrt(D)).view(B, Hkv, -1, T, k.shape[2])
    x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-1e30)
    x = x.sub_(m).exp_()
    total = x.sum(-1)
    out = (x.view(B, Hkv, -1, k.shape[2]) @ v).view(B, Hkv, -1, T, D) / total.clamp(min=1e-30)[..., None]
    lse = torch.log(total) + m[..., 0]
    out = out.permute(0, 3, 1, 2, 4).reshape(B, T, Hq, D).to(s["q"].dtype)
    lse = lse.permute(0, 3, 1, 2).reshape(B, T, Hq)
    return {"out": out, "lse": lse} if s["op"] == "tree" else {"out": out[:, 0], "lse": lse[:, 0]}


def run(state):
    s = state
    if own:
        import lse_weighted_merge_b200 as lm
        if s["op"] == "write":
            lm.kv_quantize_(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["k"], s["v"], s["start"],
                            count=s["count"], select=s["select"])
            return {n: s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")}
        if s["op"] == "read":
            k, v = lm.kv_dequantize(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["start"], s["length"],
                                    count=s["count"], dtype=s["dtype"])
            return {"k": k, "v": v}
        if s["op"] == "decode":
            out, lse = lm.decode_attention_fp8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                               kv_len=s["kv_len"])
            return {"out": out, "lse": lse}
        out, lse = lm.tree_attention(s["q"], s["k_cache"], s["v_cache"], s["k_draft"], s["v_draft"], s["tree"],
                                     k_scale=s["k_scale"], v_scale=s["v_scale"], kv_len=s["kv_len"],
                                     draft_len=s["draft_len"])
        return {"out": out, "lse": lse}
    if s["op"] == "write":
        return _write(s)
    if s["op"] == "read":
        return _read(s)
    return _attend(s)


# ---- the definitions in 64 bits, sequence by sequence

def _nearest_e4m3(y):
    """y (64 bits, at most 448) rounded to e4m3: 3 bits below the leading one, down to steps of 2^-9."""
    _, e = torch.frexp(y)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return torch.round(y / step) * step


def _exact_write(s):
    B, Hkv, L, D = s["k_cache"].shape
    out = {}
    start = s["start"].tolist()
    count = [s["k"].shape[2]] * B if s["count"] is None else s["count"].tolist()
    for name in ("k", "v"):
        cache = s[name + "_cache"].double()
        scales = s[name + "_scale"].double()
        for b in range(B):
            x = s[name][b].double()
            if s["select"] is not None:
                x = x[:, s["select"][b].long()]
            n = max(0, min(count[b], x.shape[1], L - start[b]))
            x = x[:, :n]
            big = x.abs().amax(-1)
            k = torch.ceil(torch.log2(big / 448))
            k = torch.where(big > 448 * torch.exp2(k), k + 1, k)
            k = torch.where(big <= 448 * torch.exp2(k - 1), k - 1, k)
            scale = torch.where(big == 0, torch.ones_like(big), torch.exp2(k))
            cache[b, :, start[b]:start[b] + n] = _nearest_e4m3(x / scale[..., None])
            scales[b, :, start[b]:start[b] + n] = scale
        out[name + "_cache"], out[name + "_scale"] = cache, scales
    return out


def _exact_read(s):
    B, Hkv, L, D = s["k_cache"].shape
    start = s["start"].tolist()
    count = [s["length"]] * B if s["count"] is None else s["count"].tolist()
    out = {}
    for name in ("k", "v"):
        got = torch.zeros(B, Hkv, s["length"], D, dtype=torch.float64, device="cuda")
        for b in range(B):
            n = max(0, min(count[b], s["length"], L - start[b]))
            at = slice(start[b], start[b] + n)
            got[b, :, :n] = s[name + "_cache"][b, :, at].double() * s[name + "_scale"][b, :, at].double()[..., None]
        out[name] = got
    return out


def _exact_attend(s):
    tree = s["op"] == "tree"
    q = (s["q"] if tree else s["q"][:, None]).double()
    B, T, Hq, D = q.shape
    Hkv, L = s["k_cache"].shape[1:3]
    G = Hq // Hkv
    lens = [L] * B if s["kv_len"] is None else s["kv_len"].tolist()
    live = [T] * B if not tree or s["draft_len"] is None else s["draft_len"].tolist()
    out = torch.zeros(B, T, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        one = {n: s[n][b:b + 1] if s[n] is not None else None for n in ("k_cache", "v_cache", "k_scale", "v_scale")}
        k, v = (_whole(one, n, torch.float64)[0, :, :lens[b]] for n in ("k", "v"))
        hidden = torch.zeros(live[b], lens[b], dtype=torch.bool, device="cuda")
        if tree:
            words = s["tree"][b].tolist()
            among = torch.tensor([[not words[i] >> j & 1 for j in range(live[b])] for i in range(live[b])],
                                 dtype=torch.bool, device="cuda")
            hidden = torch.cat([hidden, among], 1)
            k = torch.cat([k, s["k_draft"][b, :, :live[b]].double()], 1)
            v = torch.cat([v, s["v_draft"][b, :, :live[b]].double()], 1)
        if k.shape[1] == 0:
            continue
        for h in range(Hq):
            x = q[b, :live[b], h] @ k[h // G].T / math.sqrt(D)
            x = torch.where(hidden, -math.inf, x)
            total = torch.logsumexp(x, 1)
            lse[b, :live[b], h] = total
            at = torch.where(total == -math.inf, torch.zeros_like(total), total)
            out[b, :live[b], h] = torch.exp(x - at[:, None]) @ v[h // G]
    return {"out": out, "lse": lse} if tree else {"out": out[:, 0], "lse": lse[:, 0]}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "write":
        return _exact_write(s)
    return _exact_read(s) if case["op"] == "read" else _exact_attend(s)
