"""The 8-bit KV cache and the attention over a cache, for torch tensors.

A serving loop with drafted tokens around one cache [B, Hkv, L, D]:

    out, lse = tree_attention(q, k_cache, v_cache, k_draft, v_draft, tree_mask(parents), ...)
    kv_quantize_(k_cache, v_cache, k_scale, v_scale, k_draft, v_draft, kv_len,
                 count=accepted, select=path)            # append the accepted drafts
    out, lse = decode_attention_fp8(q, k_cache, v_cache, k_scale, v_scale, kv_len=kv_len + accepted)

The caches are e4m3 (torch.float8_e4m3fn) with one fp32 power-of-two scale per
token and KV head; tree_attention also takes 16-bit caches without scales.
The lse outputs merge across context-parallel shards with merge().  Every
call is enqueued on the current stream of the tensors' device, allocates only
through torch and can be captured in a CUDA graph.
"""
from __future__ import annotations

import math

import torch

from ._native import (E4M3, TREE_MAX_T, kv_dequantize_raw, kv_quantize_raw, tree_raw,
                      tree_workspace_bytes)
from .api import dtype_code

_FP8 = torch.float8_e4m3fn
_SMS: dict = {}   # SM count by device index


def _sms(dev) -> int:
    n = _SMS.get(dev.index)
    if n is None:
        n = _SMS[dev.index] = torch.cuda.get_device_properties(dev).multi_processor_count
    return n


def _same_device(what: str, dev, *tensors) -> None:
    if dev.type != "cuda":
        raise ValueError(f"{what} runs on CUDA tensors only (there is no CPU path)")
    for t in tensors:
        if t is not None and t.device != dev:
            raise ValueError("all tensors must be on the same CUDA device")


def _on_device(dev, call, *args):
    """call(*args, stream) with the tensors' device current (the library
    launches on the current device)."""
    if torch.cuda.current_device() == dev.index:
        return call(*args, torch.cuda.current_stream().cuda_stream)
    with torch.cuda.device(dev):
        return call(*args, torch.cuda.current_stream().cuda_stream)


def _lengths(x, n: int, what: str) -> int:
    """Address of an int32 tensor [n], 0 for None."""
    if x is None:
        return 0
    if x.dtype != torch.int32 or x.dim() != 1 or x.numel() != n or not x.is_contiguous():
        raise ValueError(f"{what} must be a contiguous int32 tensor of {n} elements")
    return x.data_ptr()


def _check_cache(k_cache, v_cache, k_scale, v_scale):
    if k_cache.dtype != _FP8 or v_cache.dtype != _FP8:
        raise TypeError("k_cache and v_cache must be float8_e4m3fn")
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape:
        raise ValueError("k_cache and v_cache must both be [B, Hkv, L, D]")
    if k_scale is None or v_scale is None:
        raise ValueError("an e4m3 cache needs k_scale and v_scale")
    if k_scale.dtype != torch.float32 or v_scale.dtype != torch.float32:
        raise TypeError("k_scale and v_scale must be float32")
    if k_scale.shape != k_cache.shape[:3] or v_scale.shape != k_cache.shape[:3]:
        raise ValueError("k_scale and v_scale must be [B, Hkv, L]")
    if k_cache.stride(3) != 1 or v_cache.stride(3) != 1:
        raise ValueError("k_cache and v_cache must be contiguous along D")


def kv_quantize_(k_cache, v_cache, k_scale, v_scale, k, v, start, *, count=None, select=None):
    """Write tokens into an e4m3 cache, in place, quantising them on the way.

    k_cache, v_cache: float8_e4m3fn [B, Hkv, L, D]; k_scale, v_scale: float32
    [B, Hkv, L] (any strides; codes contiguous along D, D 64 or 128).  k, v
    [B, Hkv, S, D]: float32, float16 or bfloat16, stride 1 along D.  start:
    int32 [B], the position of each sequence's first token; count: int32 [B],
    how many of its tokens are written (default all); select: int32 [B, T],
    which of the S rows of k and v the tokens are (default 0, 1, ..., S - 1), for
    the accepted path of a drafted tree.  A token whose position lies outside
    [0, L), or whose select index lies outside [0, S), is not written; every
    other row of the cache is left as it was.

    Each row's scale is the smallest power of two by which its largest finite
    magnitude fits e4m3's 448; elements that are not finite are stored as
    NaN.  Returns (k_cache, v_cache, k_scale, v_scale).
    """
    _check_cache(k_cache, v_cache, k_scale, v_scale)
    B, Hkv, L, D = k_cache.shape
    if k.dim() != 4 or k.shape != v.shape or k.shape[0] != B or k.shape[1] != Hkv or k.shape[3] != D:
        raise ValueError("k and v must both be [B, Hkv, S, D]")
    if k.dtype != v.dtype:
        raise TypeError("k and v must share one dtype")
    if k.stride(3) != 1 or v.stride(3) != 1:
        raise ValueError("k and v must be contiguous along D")
    dev = k_cache.device
    _same_device("kv_quantize_", dev, v_cache, k_scale, v_scale, k, v, start, count, select)
    S = T = k.shape[2]
    sel = 0
    if select is not None:
        if select.dtype != torch.int32 or select.dim() != 2 or select.shape[0] != B or not select.is_contiguous():
            raise ValueError("select must be a contiguous int32 tensor [B, T]")
        T, sel = select.shape[1], select.data_ptr()
    start_ptr, count_ptr = _lengths(start, B, "start"), _lengths(count, B, "count")
    if start_ptr == 0 and B:
        raise ValueError("start must be given")
    if B * Hkv * T == 0 or (S == 0 and select is not None):
        return k_cache, v_cache, k_scale, v_scale
    _on_device(dev, kv_quantize_raw, (
        k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), k.data_ptr(), v.data_ptr(),
        start_ptr, count_ptr, sel, *k_cache.stride()[:3], *v_cache.stride()[:3], *k_scale.stride(),
        *v_scale.stride(), *k.stride()[:3], *v.stride()[:3], B, Hkv, L, D, T, S, dtype_code(k.dtype), 0))
    return k_cache, v_cache, k_scale, v_scale


def kv_dequantize(k_cache, v_cache, k_scale, v_scale, start, length: int, *, count=None,
                  dtype=torch.bfloat16):
    """Read ``length`` tokens of every sequence back from an e4m3 cache.

    Returns (k, v), dense [B, Hkv, length, D] of ``dtype`` (bfloat16, float16 or
    float32): row j of sequence b is code * scale at position start[b] + j,
    rounded once; rows j >= count[b] (int32 [B], default length) and rows
    whose position lies outside [0, L) are zeros.
    """
    _check_cache(k_cache, v_cache, k_scale, v_scale)
    B, Hkv, L, D = k_cache.shape
    dev = k_cache.device
    _same_device("kv_dequantize", dev, v_cache, k_scale, v_scale, start, count)
    if length < 0:
        raise ValueError("length must not be negative")
    code = dtype_code(dtype)
    start_ptr, count_ptr = _lengths(start, B, "start"), _lengths(count, B, "count")
    if start_ptr == 0 and B:
        raise ValueError("start must be given")
    k, v = torch.empty((2, B, Hkv, length, D), dtype=dtype, device=dev).unbind(0)
    if B * Hkv * length == 0:
        return k, v
    x = (Hkv * length * D, length * D, D)
    _on_device(dev, kv_dequantize_raw, (
        k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), k.data_ptr(), v.data_ptr(),
        start_ptr, count_ptr, 0, *k_cache.stride()[:3], *v_cache.stride()[:3], *k_scale.stride(),
        *v_scale.stride(), *x, *x, B, Hkv, L, D, length, length, code, 0))
    return k, v


def tree_mask(parents, device=None):
    """The ancestor masks of drafted trees, as tree_attention takes them.

    parents: [T] or [B, T] integers (lists or a tensor): the draft that each
    draft continues, smaller than its own index, or -1 where it continues the
    cached sequence.  Returns int64 of the same shape on ``device`` (default
    the current CUDA device): bit j of word t is set where draft t sees draft
    j, its ancestors and itself.  Computed on the host.
    """
    p = torch.as_tensor(parents, dtype=torch.int64).cpu()
    if p.dim() not in (1, 2) or p.shape[-1] > TREE_MAX_T:
        raise ValueError(f"parents must be [T] or [B, T] with T <= {TREE_MAX_T}")
    if bool((p >= torch.arange(p.shape[-1])).any()) or bool((p < -1).any()):
        raise ValueError("a draft's parent must be an earlier draft, or -1")
    rows = []
    for row in p.reshape(-1, p.shape[-1]).tolist():
        words: list[int] = []
        for t, parent in enumerate(row):
            words.append((words[parent] if parent >= 0 else 0) | 1 << t)
        rows.append([w - (1 << 64) if w >> 63 else w for w in words])
    return torch.tensor(rows, dtype=torch.int64).reshape(p.shape).to(device if device is not None else "cuda")


def _splits(dev, units: int, L: int) -> int:
    """Shards of the cached keys: enough for about two CTAs per SM, a power of
    two of at least 64 keys each, at most 64."""
    want = -(-2 * _sms(dev) // units)
    splits = 1
    while splits < want and splits < 64 and splits * 64 < L:
        splits *= 2
    return splits


def _attend(q, k_cache, v_cache, k_draft, v_draft, tree, k_scale, v_scale, kv_len, draft_len, splits, scale,
            out_dtype):
    B, T, Hq, D = q.shape
    Hkv, L = k_cache.shape[1], k_cache.shape[2]
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape or k_cache.shape[0] != B or k_cache.shape[3] != D:
        raise ValueError("k_cache and v_cache must be [B, Hkv, L, D] with q's B and D")
    fp8 = k_cache.dtype == _FP8
    if fp8:
        _check_cache(k_cache, v_cache, k_scale, v_scale)
    elif k_cache.dtype != q.dtype or v_cache.dtype != q.dtype:
        raise TypeError("the cache must be of q's dtype, or float8_e4m3fn with scales")
    elif k_scale is not None or v_scale is not None:
        raise ValueError("k_scale and v_scale go with a float8_e4m3fn cache")
    if q.stride(3) != 1 or k_cache.stride(3) != 1 or v_cache.stride(3) != 1:
        raise ValueError("q, k_cache and v_cache must be contiguous along D")
    dev = q.device
    _same_device("attention", dev, k_cache, v_cache, k_draft, v_draft, tree, k_scale, v_scale, kv_len, draft_len)
    drafts = k_draft is not None
    kd = vd = tr = tr_b = 0
    d_str = (0, 0, 0, 0, 0, 0)
    if drafts:
        if v_draft is None or tree is None:
            raise ValueError("k_draft, v_draft and tree go together")
        if tuple(k_draft.shape) != (B, Hkv, T, D) or v_draft.shape != k_draft.shape:
            raise ValueError("k_draft and v_draft must be [B, Hkv, T, D]")
        if k_draft.dtype != q.dtype or v_draft.dtype != q.dtype:
            raise TypeError("k_draft and v_draft must be of q's dtype")
        if k_draft.stride(3) != 1 or v_draft.stride(3) != 1:
            raise ValueError("k_draft and v_draft must be contiguous along D")
        if tree.dtype != torch.int64 or tree.shape[-1] != T or tree.dim() > 2 or \
                (tree.dim() == 2 and tree.shape[0] != B) or (T > 1 and tree.stride(-1) != 1):
            raise ValueError("tree must be int64 [T] or [B, T], contiguous along T")
        kd, vd, tr = k_draft.data_ptr(), v_draft.data_ptr(), tree.data_ptr()
        tr_b = tree.stride(0) if tree.dim() == 2 else 0
        d_str = (*k_draft.stride()[:3], *v_draft.stride()[:3])
    elif v_draft is not None or tree is not None:
        raise ValueError("k_draft, v_draft and tree go together")
    out_dtype = out_dtype or q.dtype
    code, out_code = dtype_code(q.dtype), dtype_code(out_dtype)
    G = Hq // Hkv if Hkv else 0
    if splits is None:
        splits = _splits(dev, max(1, B * Hkv * -(-T * G // 16)), L)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    klen, dlen = _lengths(kv_len, B, "kv_len"), _lengths(draft_len, B, "draft_len")
    out = torch.empty((B, T, Hq, D), dtype=out_dtype, device=dev)
    lse = torch.empty((B, T, Hq), dtype=torch.float32, device=dev)
    # the workspace is this call's own: calls on other streams, and graphs
    # captured from them, never share one
    need = tree_workspace_bytes(B, T, Hq, D, splits, drafts)
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    _on_device(dev, tree_raw, (
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr() if fp8 else 0,
        v_scale.data_ptr() if fp8 else 0, kd, vd, tr, klen, dlen, out.data_ptr(), lse.data_ptr(),
        ws.data_ptr() if need else 0, need, *q.stride()[:3], *k_cache.stride()[:3], *v_cache.stride()[:3],
        *(k_scale.stride() if fp8 else (0, 0, 0)), *(v_scale.stride() if fp8 else (0, 0, 0)), *d_str, tr_b,
        B, T, Hq, Hkv, L, D, splits, code, E4M3 if fp8 else code, out_code, scale, 0))
    return out, lse


def decode_attention_fp8(q, k_cache, v_cache, k_scale, v_scale, *, kv_len=None, splits: int | None = None,
                         scale: float | None = None, out_dtype=None):
    """decode_attention over an e4m3 cache: one query token per sequence.

    q [B, Hq, D] (bfloat16 or float16); k_cache, v_cache float8_e4m3fn [B, Hkv,
    L, D] with k_scale, v_scale float32 [B, Hkv, L], as kv_quantize_ leaves
    them (any positive scales do); Hq a multiple of Hkv, at most 16 times; D 64
    or 128; kv_len an optional int32 tensor [B].  The keys are cut into
    ``splits`` shards whose partials are merged by weight (default: enough to
    fill the GPU).  Returns (out [B, Hq, D], lse [B, Hq]).
    """
    if q.dim() != 3 or k_cache.dim() != 4:
        raise ValueError("q must be [B, Hq, D] and the caches [B, Hkv, L, D]")
    if k_cache.dtype != _FP8:
        raise TypeError("k_cache and v_cache must be float8_e4m3fn")
    out, lse = _attend(q.unsqueeze(1), k_cache, v_cache, None, None, None, k_scale, v_scale, kv_len, None, splits,
                       scale, out_dtype)
    return out.squeeze(1), lse.squeeze(1)


def tree_attention(q, k_cache, v_cache, k_draft=None, v_draft=None, tree=None, *, k_scale=None, v_scale=None,
                   kv_len=None, draft_len=None, splits: int | None = None, scale: float | None = None,
                   out_dtype=None):
    """Attention of T drafted tokens per sequence over a cache and each other.

    q [B, T, Hq, D] (bfloat16 or float16, T <= 64); k_cache, v_cache [B, Hkv,
    L, D] of q's dtype, or float8_e4m3fn with k_scale and v_scale; k_draft,
    v_draft [B, Hkv, T, D] of q's dtype, the drafts' own keys and values, not in
    the cache yet; tree int64 [T] or [B, T]: token t sees all kv_len[b] cached
    keys (int32 [B], default L) and the drafts j whose bit is set in its word
    (see tree_mask).  draft_len (int32 [B]): sequence b has draft_len[b] drafts,
    the rest of its T rows is padding: 0 and -inf.  A row that sees no key also
    gives 0 and -inf.  Without k_draft, v_draft and tree the tokens attend to
    the cache alone (a shard of it, say: the lse merges with others').

    Strides are free but for stride 1 along D; Hq is a multiple of Hkv, at most
    16 times; D 64 or 128.  ``splits``: shards of the cached keys, whose
    partials are merged by weight.  Returns (out [B, T, Hq, D], lse [B, T, Hq]).
    """
    if q.dim() != 4 or k_cache.dim() != 4:
        raise ValueError("q must be [B, T, Hq, D] and the caches [B, Hkv, L, D]")
    return _attend(q, k_cache, v_cache, k_draft, v_draft, tree, k_scale, v_scale, kv_len, draft_len, splits, scale,
                   out_dtype)
