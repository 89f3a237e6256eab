"""Edges of the attention of requests that share prefixes, on the GPU against the plain 64-bit decode
(_paged.py), which knows nothing of sharing.

Tolerance: that of test_paged_shared.py."""
import math

import pytest
import torch

from flash_attention_gqa_gb300 import binding
from test_paged_shared import BF16, E4M3, Problem, _ok

pytestmark = pytest.mark.gpu
TYPES = pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])


NONE = {
    "rows8": dict(K=2, G=8, T=1, H=128, page=16),
    "rows3": dict(K=1, G=3, T=1, H=64, page=1),
    "rows16": dict(K=2, G=16, T=1, H=64, page=8),
    "rows32": dict(K=1, G=32, T=1, H=128, page=64),
    "rows40": dict(K=1, G=40, T=1, H=64, page=16),
    "rows8_h256": dict(K=2, G=8, T=1, H=256, page=32),
    "rows16_h256": dict(K=1, G=16, T=1, H=256, page=16),
}


@TYPES
@pytest.mark.parametrize("many", [False, True], ids=["few", "many"])
@pytest.mark.parametrize("name", NONE)
def test_requests_with_nothing_of_their_own(lib, name, many, dtype):
    """All that some members hold is the prefix, which ends anywhere in 8 keys.  What the call before has left
    in shared memory is NaN: it is read by nobody.  (With many requests, single warps take the own keys.)"""
    groups = [(8 * i + 40 + i, [0, 3, 0, 17 + i]) for i in range(8)]
    p = Problem(14, groups * (12 if many else 1), [5, 0], dtype=dtype, **NONE[name])
    p.on_device()
    n = 8000
    junk = [torch.full((n // 8, p.q.shape[1], 8, p.H), math.nan, dtype=BF16, device="cuda").to(dtype) for _ in range(2)]
    table = torch.arange(n // 8, dtype=torch.int32, device="cuda").expand(64, -1).contiguous()
    lens = torch.full((64,), n, dtype=torch.int32, device="cuda")
    binding.paged_attention_decode(p.args[0][:1].expand(64, -1, -1, -1, -1).contiguous(), *junk, table, lens)
    o, lse = p.run()
    p.check(o, lse)
    o2, lse2 = p.run()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    _ok()
