"""Edges of the attention of requests that share prefixes, on the GPU against the plain 64-bit decode
(_paged.py), which knows nothing of sharing.

Tolerance: that of test_paged_shared.py, for the rows that are numbers."""
import math

import pytest
import torch

from flash_attention_gqa_gb300 import binding
import _paged as P
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


# ------------------------------------------------------ values that are no numbers
# Rows of a request: the kernels for requests' own keys go by them (8 and 32: mma.sync, in bf16 up to 16 at
# H = 256; 40 and more: tcgen05), with many requests by single warps.
ROWS = {
    "rows8": dict(K=2, G=8, T=1, H=128, page=16),
    "rows32": dict(K=2, G=8, T=4, H=64, page=16),
    "rows40": dict(K=2, G=8, T=5, H=128, page=32),
    "rows32_h256": dict(K=2, G=8, T=4, H=256, page=64),
}


def _put(cache, p, b, s, head, x, dims=slice(None)):
    """`x` into position s of request b."""
    page = cache.shape[2]
    cache[int(p.table[b, s // page]), head, s % page, dims] = x


def _check(p):
    """A row is no number exactly where the definition says so, infinities stay infinities, and the
    others are within their roundings."""
    p.on_device()
    o, lse = (x.cpu() for x in p.run())
    _ok()
    ro, rl, (size, _) = P.decode(p.q, *p.caches, p.table, p.lens, *p.scales)
    clean = [torch.nan_to_num(c.float(), 0.0, 0.0, 0.0) for c in p.caches]
    # (a score of -inf has no weight and no rounding)
    reach = P.decode(torch.nan_to_num(p.q.float()), *clean, p.table, p.lens, *p.scales)[2][1]
    assert torch.equal(torch.isnan(o), torch.isnan(ro)) and torch.equal(torch.isnan(lse), torch.isnan(rl))
    assert torch.equal(torch.isinf(o), torch.isinf(ro)) and torch.equal(o[torch.isinf(o)].double(), ro[torch.isinf(ro)])
    odd, odd_row = ~torch.isfinite(ro), torch.isnan(rl)
    zero = lambda x, where: torch.where(where, torch.zeros_like(x), x)  # noqa: E731
    P.check_decode(zero(o, odd), zero(lse, odd_row), (zero(ro, odd), zero(rl, odd_row), (zero(size, odd), reach)),
                   p.H, p.e4m3, int(p.lens.max()) + 16)
    return odd, odd_row


def _problem(rows, dtype, groups, alone=(), **kw):
    """In every group, members with T and more tokens of their own."""
    c = {**ROWS[rows], **kw}
    return Problem(13, [(n, [c["T"] + t for t in tails]) for n, tails in groups], alone, dtype=dtype, **c)


LONG = [(2100, [0, 5, 70]), (96, [0, 40])]


@TYPES
@pytest.mark.parametrize("rows", ROWS)
def test_queries_that_are_nan(lib, rows, dtype):
    """One query row of a member, all rows of another, one of a request in no group."""
    p = _problem(rows, dtype, LONG, [30])
    p.q[p.members[0], 1, 3, -1, 9] = math.nan
    p.q[p.members[4], 0] = math.nan
    alone = next(b for b in range(6) if b not in p.members)
    p.q[alone, 0, 2, 0, 0] = math.nan
    odd, odd_row = _check(p)
    assert odd_row.sum() == 2 + p.q.shape[2] * p.q.shape[3] and odd_row[p.members[0], 1, 3, -1]


@TYPES
@pytest.mark.parametrize("rows", ROWS)
def test_own_keys_that_are_nan(lib, rows, dtype):
    """The first own key, the only one that a first query has, and a newest key, which only a last one sees."""
    p = _problem(rows, dtype, LONG)
    a, b = p.members[0], p.members[3]
    _put(p.caches[0], p, a, 2100, 0, math.nan)
    _put(p.caches[0], p, b, int(p.lens[b]) - 1, 1, math.nan, 7)
    odd, odd_row = _check(p)
    assert odd_row[a, 0].all() and odd_row[b, 1, :, -1].all()
    assert odd_row.sum() == p.q.shape[2] * (p.q.shape[3] + 1)


@TYPES
@pytest.mark.parametrize("rows", ROWS)
def test_prefixes_that_are_nan(lib, rows, dtype):
    """All keys of a short prefix for one kv head, and one key of a long prefix for the other."""
    p = _problem(rows, dtype, LONG)
    lead = p.members[3]
    for s in range(96):
        for b in p.members[3:]:     # (a last page that is not full is a copy)
            _put(p.caches[0], p, b, s, 1, math.nan)
    for b in p.members[:3]:
        _put(p.caches[0], p, b, 1500, 0, math.nan, 0)
    odd, odd_row = _check(p)
    assert odd_row[p.members[3:], 1].all() and odd_row[p.members[:3], 0].all()
    assert not odd_row[lead, 0].any() and not odd_row[p.members[0], 1].any()


@pytest.mark.parametrize("rows", ROWS)
def test_infinities_of_prefixes(lib, rows):
    """Values: results of their sign.  Keys: scores of -inf have no weight, a whole prefix of them neither;
    one of +inf leaves no number."""
    p = _problem(rows, BF16, LONG)
    p.q[..., 0] = p.q[..., 0].abs().clamp(min=1e-3)
    p.q[p.members[1], 0, 0, 0, 0] *= -1              # this row's scores of the key below are +inf
    for b in p.members[:3]:
        _put(p.caches[0], p, b, 700, 0, -math.inf, 0)
        _put(p.caches[1], p, b, 20, 1, math.inf, 3)
        _put(p.caches[1], p, b, 2040, 1, -math.inf, 5)
    for b in p.members[3:]:
        for s in range(96):
            _put(p.caches[0], p, b, s, 1, -math.inf, 0)
    odd, odd_row = _check(p)
    assert odd_row.sum() == 1 and odd_row[p.members[1], 0, 0, 0]
    assert odd[p.members[:3], 1][..., 3].all() and odd[p.members[:3], 1][..., 5].all()


@TYPES
def test_nan_with_own_keys_by_warps(lib, dtype):
    """Many requests, whose own keys single warps take."""
    p = _problem("rows8", dtype, [(100, [i % 50 for i in range(32)])] * 10, [1, 40])
    assert len(p.lens) * 2 >= 2 * 2 * 152
    for g in range(10):
        b = p.members[32 * g]                        # with one own key
        if g % 2:
            p.q[b, 0, g % 8, 0, g] = math.nan
        else:
            _put(p.caches[0], p, b, 100, 1, math.nan)
    odd, odd_row = _check(p)
    assert odd_row.sum() == 5 + 5 * 8


# ------------------------------------------------------------ pages and tiles, waits
@TYPES
@pytest.mark.parametrize("layout", ["head", "token"])
@pytest.mark.parametrize("page", [128, 256, 1024])
@pytest.mark.parametrize("H", [64, 128, 256])
def test_pages_larger_than_a_tile(lib, H, page, layout, dtype):
    """Tiles of 128 keys (64 at H = 256) that begin anywhere in a page; prefixes that end with a page, at a
    tile's end within one, and within a tile."""
    groups = [(2048, [1, 40, 300]), (page + 64, [5, 9]), (1500, [2, 77])]
    p = Problem(H + page, groups, [30], K=2, G=8, T=1, H=H, page=page, dtype=dtype, layout=layout, pad=64).on_device()
    p.check(*p.run())
    _ok()


@TYPES
@pytest.mark.parametrize("H", [64, 128, 256])
@pytest.mark.parametrize("T", [1, 5])
def test_short_limits_of_waits(lib, H, T, dtype):
    """Limits from none to longer than any wait: a call ends with an error, or its results are the same, and
    the next call's are."""
    groups = [(5000, [T + 9, T + 40, T + 1])] * 2 + [(640, [T, T + 11])]
    p = Problem(12, groups, [12], K=2, G=8, T=T, H=H, page=64, dtype=dtype).on_device()
    want = p.run()
    p.check(*want)
    for limit in (1, 300, 1000, 2000, 4000, 8000, 16000, 64000):
        assert binding.fa_set_wait_limit_ns(limit) == binding.FA_OK
        try:
            o, lse = p.run()
            rc = binding.fa_check_status()
        finally:
            assert binding.fa_set_wait_limit_ns(2_000_000_000) == binding.FA_OK
        assert rc in (binding.FA_OK, binding.FA_ERR_DEVICE_TIMEOUT)
        assert rc or (torch.equal(o, want[0]) and torch.equal(lse, want[1]))
        again = p.run()
        _ok()
        assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
