"""Plain 64-bit forms of the 8-bit cache and of the attention over a cache and
drafts, and the error bounds of the GPU results against them.

Error bound of an attention row (from the arithmetic, half a step per rounding):
with u_p the half step of the weights' type (bf16 2^-8, f16 2^-11) and u_o that
of the output type,
    |o - o64| <= u_o |o64| + (u_p + w) A + n 2^-31 max|v|,   A = sum_j p_j |v_j|
  * u_p A: each weight is rounded once to the type of the second product (its
    normaliser sums the unrounded ones);
  * w A: relative error of a weight from its score, twice (numerator and
    normaliser).  A score sums D products in fp32; the tensor core may truncate
    where IEEE rounds, so a step of 2^-23 per term, of at most S = max_j scale *
    sum_d |q_d k_jd|; a few more roundings of the scaled score (2^-22 of it) and
    of exp2 (2^-22); fp32 sums of n weights: n 2^-23:
    w = 2 ((D + 8) 2^-23 S + 2^-21 + n 2^-23);
  * n 2^-31 max|v|: f16 weights keep an absolute 2^-25 of a reference that
    lies at least 2^6 above the largest weight's 1.
lse: w/2 from the scores and the sum, 2^-22 |lse| from the logarithm and the
final fp32 operations, and the same again for the merge of the shards.
"""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
FP8 = torch.float8_e4m3fn


def quantised(x):
    """(values of the codes, scale) of rows x [..., D], in 64 bits."""
    x = x.double()
    fin = torch.isfinite(x)
    a = torch.where(fin, x.abs(), torch.zeros_like(x)).amax(-1)
    m, e = torch.frexp(a / 448)
    k = torch.where(m == 0.5, e - 1, e).clamp(min=-126)      # a / 448 <= 2^k
    k = torch.where(a == 0, torch.zeros_like(k), k)
    scale = torch.ldexp(torch.ones_like(a), k)
    y = torch.where(fin, x, torch.zeros_like(x)) / scale[..., None]
    _, e = torch.frexp(y)
    step = torch.ldexp(torch.ones_like(y), (e - 1).clamp(min=-6) - 3)
    codes = torch.round(y / step) * step
    return torch.where(fin, codes, torch.full_like(codes, math.nan)), scale


def store(x, layout):
    """x [B, H, L, ...] with the storage of "bhl" (as given) or "blh" (token by token)."""
    return x.contiguous() if layout == "bhl" else x.transpose(1, 2).contiguous().transpose(1, 2)


def fp8_cache(x, layout="bhl"):
    """An e4m3 cache (codes, scale) that holds x [B, H, L, D]."""
    codes, scale = quantised(x)
    return (store(codes.float().to(FP8), layout),
            store(scale.float()[..., None], layout)[..., 0])


def attention(q, k, v, kd=None, vd=None, tree=None, kv_len=None, draft_len=None, scale=None):
    """64-bit (out, lse, A, S, n, vmax) of q [B, T, Hq, D] over k, v [B, Hkv, L, D] and drafts."""
    B, T, Hq, D = q.shape
    Hkv, L = k.shape[1:3]
    G = Hq // Hkv
    scale = 1 / math.sqrt(D) if scale is None else scale
    dev = q.device
    out = torch.zeros(B, T, Hq, D, dtype=torch.float64, device=dev)
    lse = torch.full((B, T, Hq), -math.inf, dtype=torch.float64, device=dev)
    A, S = torch.zeros_like(out), torch.zeros_like(lse)
    n = torch.zeros_like(lse)
    vmax = torch.zeros_like(lse)
    for b in range(B):
        ln = L if kv_len is None else max(0, min(L, int(kv_len[b])))
        live = T if draft_len is None else max(0, min(T, int(draft_len[b])))
        if live == 0:
            continue
        kk, vv = k[b, :, :ln].double(), v[b, :, :ln].double()
        seen = torch.ones(live, ln, dtype=torch.bool, device=dev)
        if kd is not None:
            words = (tree if tree.dim() == 1 else tree[b]).tolist()
            among = torch.tensor([[bool(w >> j & 1) for j in range(live)] for w in words[:live]],
                                 dtype=torch.bool, device=dev).reshape(live, live)
            seen = torch.cat([seen, among], 1)
            kk = torch.cat([kk, kd[b, :, :live].double()], 1)
            vv = torch.cat([vv, vd[b, :, :live].double()], 1)
        if kk.shape[1] == 0:
            continue
        qq = q[b, :live].double().reshape(live, Hkv, G, D)
        x = torch.einsum("thgd,hjd->thgj", qq, kk) * scale
        x = torch.where(seen[:, None, None], x, torch.full_like(x, -math.inf))
        tot = torch.logsumexp(x, -1)
        p = torch.exp(x - torch.where(tot == -math.inf, torch.zeros_like(tot), tot)[..., None])
        hidden = ~seen[:, None, None, :, None]
        # hidden keys never reach the row, whatever they hold
        vs = torch.where(hidden, torch.zeros((), dtype=torch.float64, device=dev), vv[None, :, None])
        o = (p[..., None] * vs).sum(-2) if live * Hq * vv.shape[1] * D < 1 << 26 else torch.einsum("thgj,hjd->thgd", p, vv)
        out[b, :live] = o.reshape(live, Hq, D)
        lse[b, :live] = tot.reshape(live, Hq)
        A[b, :live] = torch.einsum("thgj,hjd->thgd", p, torch.nan_to_num(vv, 0, 0, 0).abs()).reshape(live, Hq, D)
        sk = torch.einsum("thgd,hjd->thgj", qq.abs(), torch.nan_to_num(kk, 0, 0, 0).abs()) * abs(scale)
        S[b, :live] = torch.where(seen[:, None, None], sk, torch.zeros_like(sk)).amax(-1).reshape(live, Hq)
        n[b, :live] = float(kk.shape[1])
        vmax[b, :live] = float(torch.nan_to_num(vv, 0, 0, 0).abs().max())
    return out, lse, A, S, n, vmax


def check(got, got_lse, ref, weight_type, what=""):
    """Assert that (got, got_lse) is within the bounds of the 64-bit `ref`."""
    out, lse, A, S, n, vmax = ref
    D = out.shape[-1]
    empty = lse == -math.inf
    g, gl = got.double(), got_lse.double()
    assert bool((gl[empty] == -math.inf).all()) and bool((g[empty] == 0).all()), f"{what}: an empty row is not 0, -inf"
    w = 2 * ((D + 8) * 2.0 ** -23 * S + 2.0 ** -21 + n * 2.0 ** -23)
    bound = U[got.dtype] * out.abs() + (U[weight_type] + w)[..., None] * A + (n * 2.0 ** -31 * vmax)[..., None] + 1e-30
    err = (g - out).abs()[~empty] / bound[~empty]
    assert not bool(torch.isnan(err).any()), f"{what}: NaN"
    worst = float(err.max()) if err.numel() else 0.0
    assert worst <= 1, f"{what}: error {worst:.3f} of its bound"
    lerr = (gl - lse).abs()[~empty] / (w + 2.0 ** -21 * (1 + lse.abs()))[~empty]
    lworst = float(lerr.max()) if lerr.numel() else 0.0
    assert lworst <= 1, f"{what}: lse error {lworst:.3f} of its bound"
    return worst, lworst
