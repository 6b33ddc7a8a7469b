"""Tree attention whose values arrive long after its keys: the cached values lie in
pinned host memory, the keys on the GPU, so that a block has the scores and weights of
its last keys before the values of any.  The answer is that of values on the GPU, bit
for bit: the end of a block waits for all of its products."""
import ctypes
import math

import pytest
import torch

from kv_util import check
from lse_weighted_merge_b200 import _native as nat
from test_gpu_tree import KINDS, Case

pytestmark = pytest.mark.gpu
CODE = {torch.bfloat16: nat.BF16, torch.float16: nat.F16}


def call(c, v_address, splits, drafts):
    """tree_attention of the case with its cached values at v_address."""
    B, T, Hq, D = c.q.shape
    Hkv, L = c.k.shape[1:3]
    out = torch.full((B, T, Hq, D), math.nan, device="cuda")
    lse = torch.full((B, T, Hq), math.nan, device="cuda")
    ws = torch.zeros(max(16, nat.tree_workspace_bytes(B, T, Hq, D, splits, drafts)), dtype=torch.uint8, device="cuda")
    ks, vs = (c.scales.get(n) for n in ("k_scale", "v_scale"))
    s = (ks.stride(), vs.stride()) if c.scales else ((0, 0, 0), (0, 0, 0))
    d = (c.kd.data_ptr(), c.vd.data_ptr(), c.tree.data_ptr()) if drafts else (0, 0, 0)
    dt = CODE[c.q.dtype]
    nat.tree_raw((c.q.data_ptr(), c.k.data_ptr(), v_address, ks.data_ptr() if c.scales else 0,
                  vs.data_ptr() if c.scales else 0, *d, 0, 0, out.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(),
                  *c.q.stride()[:3], *c.k.stride()[:3], *c.v.stride()[:3], *s[0], *s[1], *c.kd.stride()[:3],
                  *c.vd.stride()[:3], T, B, T, Hq, Hkv, L, D, splits, dt, nat.E4M3 if c.scales else dt, nat.F32,
                  1 / math.sqrt(D), 0), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    return out, lse


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,L", [(8, 128), (8, 384), (24, 128), (24, 300), (48, 512)])
def test_values_in_host_memory(T, L, kind):
    """T * 4 query rows: one tile of them (32, 96 rows) or two (192)."""
    c = Case(kind, 12, T, 32, 8, L, 128)
    far = torch.empty(c.v.shape, dtype=torch.uint8 if c.scales else c.v.dtype, pin_memory=True)
    far.copy_(c.v.view(torch.uint8) if c.scales else c.v)
    for splits in (1, 2):
        for drafts in (True, False):
            want = call(c, c.v.data_ptr(), splits, drafts)
            check(*want, c.ref(drafts), c.wt if drafts else c.wt_cache)
            for _ in range(3):
                got = call(c, far.data_ptr(), splits, drafts)
                assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    n = ctypes.c_uint32(7)
    assert nat.lib.lse_merge_tree_status(ctypes.byref(n)) == 0 and n.value == 0
