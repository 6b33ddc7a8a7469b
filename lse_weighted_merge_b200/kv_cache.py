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

import torch

from ._native import TREE_MAX_T, _raise

try:
    from . import _torch_ops
except ImportError as e:
    raise ImportError("the extension of csrc/torch_ops.cpp is missing, or was built for another torch: build it with "
                      "`python -m lse_weighted_merge_b200.build`. These calls have no fallback.") from e


def kv_quantize_(k_cache, v_cache, k_scale, v_scale, k, v, start, *, count=None, select=None):
    """Write tokens into an e4m3 cache, in place, quantising them on the way.

    k_cache, v_cache: float8_e4m3fn [B, Hkv, L, D], D 64 or 128, stride 1 along D,
    the other strides whole multiples of 16 bytes; k_scale, v_scale: float32
    [B, Hkv, L], any strides.  k, v [B, Hkv, S, D]: float32, float16 or bfloat16,
    strides as the caches'.  start: int32 [B], the position of each sequence's
    first token; count: int32 [B], how many of its tokens are written (default
    all); select: int32 [B, T], which of the S rows of k and v the tokens are
    (default 0, 1, ..., S - 1), for the accepted path of a drafted tree.  A token
    whose position lies outside [0, L), or whose select index lies outside [0, S),
    is not written; every other row of the cache is left as it was.

    Each row's scale is the smallest power of two by which its largest finite
    magnitude fits e4m3's 448; elements that are not finite are stored as
    NaN.  Returns (k_cache, v_cache, k_scale, v_scale).
    """
    rc = _torch_ops.quantize(k_cache, v_cache, k_scale, v_scale, k, v, start, count, select)
    if rc:
        _raise(rc)
    return k_cache, v_cache, k_scale, v_scale


def kv_dequantize(k_cache, v_cache, k_scale, v_scale, start, length: int, *, count=None,
                  dtype=torch.bfloat16):
    """Read ``length`` tokens of every sequence back from an e4m3 cache.

    Returns (k, v), dense [B, Hkv, length, D] of ``dtype`` (bfloat16, float16 or
    float32): row j of sequence b is code * scale at position start[b] + j,
    rounded once; rows j >= count[b] (int32 [B], default length) and rows
    whose position lies outside [0, L) are zeros.
    """
    got = _torch_ops.dequantize(k_cache, v_cache, k_scale, v_scale, start, length, count, dtype)
    if type(got) is int:
        _raise(got)
    return got


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


def decode_attention_fp8(q, k_cache, v_cache, k_scale, v_scale, *, kv_len=None, splits: int | None = None,
                         scale: float | None = None, out_dtype=None):
    """decode_attention over an e4m3 cache: one query token per sequence.

    q [B, Hq, D] (bfloat16 or float16); k_cache, v_cache float8_e4m3fn [B, Hkv,
    L, D] with k_scale, v_scale float32 [B, Hkv, L], as kv_quantize_ leaves
    them (any positive scales do, the values' within 2^70 of each other; 0 stands
    for a key or value of zeros); Hq a multiple of Hkv, at most 16 times; D 64
    or 128; kv_len an optional int32 tensor [B].  The keys are cut into
    ``splits`` shards whose partials are merged by weight (default: enough to
    fill the GPU).  L is 1 or more (an empty cache is kv_len 0).  Returns (out
    [B, Hq, D], lse [B, Hq]).
    """
    got = _torch_ops.attention(True, q, k_cache, v_cache, None, None, None, k_scale, v_scale, kv_len, None, splits,
                               scale, out_dtype)
    if type(got) is int:
        _raise(got)
    return got


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

    Stride 1 along D, the other strides whole multiples of 16 bytes (scales: any);
    Hq is a multiple of Hkv, at most 16 times; D 64 or 128; L is 1 or more (an
    empty cache is kv_len 0); B or T may be 0.  ``splits``: shards of the cached
    keys, whose partials are merged by weight.  Returns (out [B, T, Hq, D], lse [B, T, Hq]).
    """
    got = _torch_ops.attention(False, q, k_cache, v_cache, k_draft, v_draft, tree, k_scale, v_scale, kv_len,
                               draft_len, splits, scale, out_dtype)
    if type(got) is int:
        _raise(got)
    return got
