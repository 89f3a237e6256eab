"""The paged cache operators where they can go wrong: waits that run out, values at the ends of
their types, sizes at the limits of a launch, errors of other calls."""
import pytest
import torch

from flash_attention_gqa_gb300 import binding
import _paged as P
from test_paged import BF16, E4M3, _check, _decode, _ok

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("H", [64, 128, 256])
def test_decode_waits_that_run_out_anywhere_leave_nothing_behind(lib, H, dtype):
    """Limits from none to longer than any wait, so that one runs out at the queries, the copies, the
    products or the last product: the call ends, its products with it, and the next is right."""
    p = P.problem(4, B=24, K=2, G=40, T=1, H=H, lens=[3000, 700, 40, 1] * 6, page=16, dtype=dtype)
    want = _check(p)
    for limit in (1, 300, 1000, 2000, 4000, 8000, 16000, 64000):
        assert binding.fa_set_wait_limit_ns(limit) == binding.FA_OK
        try:
            o, lse = _decode(p)
            rc = binding.fa_check_status()
        finally:
            assert binding.fa_set_wait_limit_ns(2_000_000_000) == binding.FA_OK
        assert rc in (binding.FA_OK, binding.FA_ERR_DEVICE_TIMEOUT)
        assert rc or (torch.equal(o, want[0]) and torch.equal(lse, want[1]))
        again = _decode(p)
        _ok()
        assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
