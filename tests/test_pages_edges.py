"""Pages between steps at the ends of the ranges that a call may have, on the GPU against _pages.py."""
import numpy as np
import pytest
import torch

from flash_attention_gqa_gb300 import binding
from _pages import random_pool
from test_pages import Device, _bad_value, _i32, _ok

pytestmark = pytest.mark.gpu
INT32_MAX = 2 ** 31 - 1


def _gigabytes(n):
    if torch.cuda.mem_get_info()[0] < n << 30:
        pytest.skip(f"needs {n} GB of device memory")


def _with_list(pool, n):
    """The pool's tensors with a free list of n entries, whose last are the pool's."""
    d = Device(pool)
    d.free = torch.empty(n, dtype=torch.int32, device="cuda")
    spare = len(pool.free) - pool.used
    d.free[n - spare:] = _i32(pool.free[pool.used:])
    d.used.fill_(n - spare)
    return d, spare


@pytest.mark.parametrize("wrong", [False, True], ids=["met", "not_met"])
@pytest.mark.parametrize("in_place", [True, False], ids=["in_place", "apart"])
def test_compact_with_the_longest_free_list(lib, in_place, wrong):
    """Entries up to the last that an int counts: the steps of the kernel's threads pass it."""
    _gigabytes(20)
    pool = random_pool(np.random.default_rng(3), 30, 16, 700, spare=100)
    d, spare = _with_list(pool, INT32_MAX)
    if wrong:
        d.free[-1] = d.free[-2]
    was = d.free[-spare:].clone()
    want, most = pool.copy(), 50
    moves = np.tile(np.int32([-1, -1, 0]), (most, 1)) if wrong else want.compact(most)
    out = (d.table, d.shares, d.free) if in_place else (
        torch.full_like(d.table, 88), torch.full_like(d.shares, 88), torch.empty_like(d.free))
    got = torch.full((most, 3), 44, dtype=torch.int32, device="cuda")
    binding.fa_paged_compact(d.lens, d.table, d.shares, d.free, d.used, *out, got, pool.page)
    torch.cuda.synchronize()
    assert np.array_equal(got.cpu().numpy(), moves)
    assert np.array_equal(out[0].cpu().numpy(), want.table) and np.array_equal(out[1].cpu().numpy(), want.shares)
    assert torch.equal(out[2][-spare:].cpu(), was.cpu() if wrong else torch.tensor(want.free[want.used:]))
    assert d.used.item() == INT32_MAX - spare
    if wrong:
        _bad_value()
    _ok()


def test_compact_with_the_most_moves(lib):
    """Room for as many moves as an int counts; those behind the last that is needed are none."""
    _gigabytes(40)
    pool = random_pool(np.random.default_rng(4), 20, 16, 300, spare=80)
    d, want = Device(pool), pool.copy()
    moves = want.compact(len(pool.shares))
    moves = moves[moves[:, 0] >= 0]
    assert len(moves) > 10
    got = torch.empty((INT32_MAX, 3), dtype=torch.int32, device="cuda")
    binding.fa_paged_compact(d.lens, d.table, d.shares, d.free, d.used, d.table, d.shares, d.free, got, pool.page)
    d.equals(want, free_from=pool.used)
    n = len(moves)
    assert np.array_equal(got[:n].cpu().numpy(), moves)
    for at in (n, INT32_MAX // 2, INT32_MAX - 20000):
        assert (got[at:at + 20000].cpu() == torch.tensor([-1, -1, 0])).all()
    _ok()
