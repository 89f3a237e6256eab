"""Requests forked, freed and cut, pools compacted and pages copied, on the GPU against the loops of
_pages.py.  All of it is whole numbers and bytes: results are equal."""
import numpy as np
import pytest
import torch

from flash_attention_gqa_gb300 import binding
import _paged as P
from _pages import Pool, random_pool, up

pytestmark = pytest.mark.gpu
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _ok():
    torch.cuda.synchronize()
    assert binding.fa_check_status() == binding.FA_OK


def _bad_value():
    torch.cuda.synchronize()
    assert binding.fa_check_status() == binding.FA_ERR_DEVICE_VALUE
    _ok()


class Device:
    """A pool's tensors on the device."""

    def __init__(self, pool):
        self.lens, self.table, self.shares, self.free = (_i32(x) for x in (
            pool.lens, pool.table, pool.shares, pool.free))
        self.used, self.page = _i32([pool.used]), pool.page

    def outputs(self, in_place):
        """(lens_out, free_used_out)"""
        if in_place:
            return self.lens, self.used
        return torch.full_like(self.lens, 77), torch.full_like(self.used, 77)

    def equals(self, pool, lens=None, used=None, table=None, shares=None, free=None, free_from=0):
        torch.cuda.synchronize()
        for name, got, want in (("lens", self.lens if lens is None else lens, pool.lens),
                                ("table", self.table if table is None else table, pool.table),
                                ("shares", self.shares if shares is None else shares, pool.shares),
                                ("free", (self.free if free is None else free)[free_from:], pool.free[free_from:]),
                                ("used", self.used if used is None else used, [pool.used])):
            assert np.array_equal(got.cpu().numpy(), want), name


def _free(pool, rows, keep=None, in_place=True):
    d = Device(pool)
    lens, used = d.outputs(in_place)
    binding.fa_paged_free(_i32(rows), d.lens, d.table, d.shares, d.free, d.used, lens, used, pool.page,
                          None if keep is None else _i32(keep))
    return d, lens, used


def _fork(pool, parents, children, fork_lens=None, in_place=True):
    d = Device(pool)
    lens, used = d.outputs(in_place)
    copies = torch.full((len(parents), 3), 55, dtype=torch.int32, device="cuda")
    binding.fa_paged_fork(_i32(parents), _i32(children), d.lens, d.table, d.shares, d.free, d.used, lens, copies,
                          used, pool.page, None if fork_lens is None else _i32(fork_lens))
    return d, lens, used, copies


SIZES = [(1, 16, 40), (2, 1, 9), (7, 4, 100), (40, 16, 300), (64, 64, 3000), (300, 16, 50), (300, 8, 700),
         (8192, 16, 60), (3, 65536, 200000), (5, 2, 5000), (257, 128, 129)]
each_size = pytest.mark.parametrize("size", SIZES, ids=lambda s: "B%d_page%d_len%d" % s)
both_places = pytest.mark.parametrize("in_place", [False, True], ids=["apart", "in_place"])


# ------------------------------------------------------------------- free

@both_places
@each_size
def test_free(lib, size, in_place):
    B, page, longest = size
    rng = np.random.default_rng(B + page)
    pool = random_pool(rng, B, page, longest)
    pool.check()
    rows = np.array([r for r in rng.permutation(B) if rng.random() < 0.6] + [-1, -5])
    rng.shuffle(rows)
    want = pool.copy()
    want.free_rows(rows)
    want.check()
    d, lens, used = _free(pool, rows, in_place=in_place)
    d.equals(want, lens, used)
    if not in_place:
        assert np.array_equal(d.lens.cpu().numpy(), pool.lens)
    _ok()


def _cuts(pool, rng, rows):
    """Tokens to keep that leave no shared page in part."""
    keep = []
    for r in rows:
        n = int(pool.lens[r]) if r >= 0 else 0
        k = int(rng.integers(0, n + 1)) if rng.random() < 0.8 else n
        while 0 < k < n and k % pool.page and pool.shares[pool.table[r, k // pool.page]] > 0:
            k = k // pool.page * pool.page
        keep.append(k)
    return keep


@both_places
@each_size
def test_free_of_the_last_tokens(lib, size, in_place):
    B, page, longest = size
    rng = np.random.default_rng(B * 3 + page)
    pool = random_pool(rng, B, page, longest)
    rows = [r for r in rng.permutation(B) if rng.random() < 0.9] + [-1]
    keep = _cuts(pool, rng, rows)
    want = pool.copy()
    want.free_rows(rows, keep)
    want.check()
    d, lens, used = _free(pool, rows, keep, in_place)
    d.equals(want, lens, used)
    _ok()


def test_free_of_every_holder_of_a_page_at_once(lib):
    pool = random_pool(np.random.default_rng(1), 6, 16, 200, fork=0)
    pool.free_rows([1, 2, 3, 4, 5])
    if pool.lens[0] == 0:
        pool.lens[0] = 100
        pool.table[0, :7] = pool.free[pool.used:pool.used + 7]
        pool.used += 7
    pool.fork([0] * 5, [1, 2, 3, 4, 5])
    pool.check()
    want = pool.copy()
    want.free_rows([5, 0, 3, 1, 2, 4])
    want.check()
    assert want.used == 0
    d, lens, used = _free(pool, [5, 0, 3, 1, 2, 4])
    d.equals(want)
    _ok()


def test_free_of_a_pool_of_two_million_pages(lib):
    n_pages, page = 1 << 21, 16
    rng = np.random.default_rng(4)
    ids = rng.permutation(n_pages)
    lens = np.array([16 * 30000 - 3, 1, 16 * 5000])
    table = np.zeros((3, 30000))
    at = 0
    for b, n in enumerate(lens):
        table[b, :up(int(n), page)] = ids[at:at + up(int(n), page)]
        at += up(int(n), page)
    pool = Pool(table, lens, np.zeros(n_pages), ids, at, page)
    want = pool.copy()
    want.free_rows([0, 2], [0, 17])
    d, lens, used = _free(pool, [0, 2], [0, 17])
    d.equals(want)
    moves = torch.empty((6000, 3), dtype=torch.int32, device="cuda")
    more = want.compact(6000)
    binding.fa_paged_compact(d.lens, d.table, d.shares, d.free, d.used, d.table, d.shares, d.free, moves, page)
    d.equals(want)
    assert np.array_equal(moves.cpu().numpy(), more)
    _ok()


@both_places
@pytest.mark.parametrize("fault", ["row", "twice", "keep", "long", "negative", "len", "used", "shared", "list"])
def test_free_that_cannot_be_met_changes_nothing(lib, fault, in_place):
    page = 16
    pool = Pool(np.arange(24).reshape(4, 6), [90, 33, 0, 0], np.zeros(30), np.r_[np.arange(24), 24:30], 24, page)
    pool.table[2, :2] = pool.table[0, :2]
    pool.table[2, 2] = 12
    pool.lens[2] = 40
    pool.shares[:2] = 1
    rows, keep = [0, 1, -1], [90, 20, 0]
    if fault == "row":
        rows[1] = 4
    elif fault == "twice":
        rows[2] = 0
    elif fault == "keep":
        keep[1] = -1
    elif fault == "long":
        keep[1] = 34
    elif fault == "negative":
        pool.lens[1] = -1
    elif fault == "len":
        pool.lens[1] = 97
    elif fault == "used":
        pool.used = 31
    elif fault == "shared":
        keep[0] = 24          # within page 1, which request 2 holds too
    else:
        pool.used = 0         # the list has given out nothing
    d, lens, used = _free(pool, rows, keep, in_place)
    d.equals(pool, lens, used)
    _bad_value()


def test_free_of_odd_pages(lib):
    """Ids out of range are skipped; a page that two requests hold without a count comes back once."""
    pool = Pool(np.arange(24).reshape(4, 6), [90, 33, 0, 0], np.zeros(30), np.arange(30), 24, 16)
    pool.table[0, 2], pool.table[0, 3], pool.table[1, 0] = -1, 30, 5
    d, lens, used = _free(pool, [1, 0])
    torch.cuda.synchronize()
    assert used.item() == 24 - 6 and lens.tolist() == [0] * 4
    assert d.free[18:24].tolist() == [0, 1, 4, 5, 7, 8] and not d.shares.any()
    _bad_value()


# ------------------------------------------------------------------- fork

@both_places
@pytest.mark.parametrize("cut", [False, True], ids=["all", "cut"])
@each_size
def test_fork(lib, size, cut, in_place):
    B, page, longest = size
    rng = np.random.default_rng(B * 7 + page)
    pool = random_pool(rng, B, page, longest, spare=B + 20, fork=0.2)
    living, empty = np.nonzero(pool.lens)[0], np.nonzero(pool.lens == 0)[0]
    if not len(living):
        pool.lens[0] = longest
        pool.table[0, :up(longest, page)] = pool.free[:up(longest, page)]
        pool.used = up(longest, page)
        living, empty = np.array([0]), np.arange(1, B)
    parents = rng.choice(living, len(empty))
    parents[rng.random(len(parents)) < 0.2] = -1
    lens = [int(rng.integers(0, pool.lens[p] + 1)) if p >= 0 else -3 for p in parents] if cut else None
    want = pool.copy()
    copies = want.fork(parents, empty, lens)
    want.check()
    d, lens_out, used, got = _fork(pool, parents, empty, lens, in_place)
    d.equals(want, lens_out, used)
    assert np.array_equal(got.cpu().numpy(), copies)
    _ok()


@both_places
@pytest.mark.parametrize("fault", ["parent", "child", "below", "twice", "held", "self", "chain", "long",
                                   "negative", "len", "pages", "used"])
def test_fork_that_cannot_be_met_changes_nothing(lib, fault, in_place):
    pool = Pool(np.arange(48).reshape(8, 6), [90, 33, 0, 0, 0, 0, 0, 0], np.zeros(50), np.arange(50), 46, 16)
    parents, children, lens = [0, 1, 0, -1], [2, 3, 4, 0], [90, 20, 16, 0]
    if fault == "parent":
        parents[1] = 8
    elif fault == "child":
        children[1] = 8
    elif fault == "below":
        children[1] = -1
    elif fault == "twice":
        children[1] = 4
    elif fault == "held":
        children[2] = 1
    elif fault == "self":
        parents[2] = children[2] = 5
        lens[2] = 0
    elif fault == "chain":
        parents[1], lens[1] = 2, 0      # the first entry's child
    elif fault == "long":
        lens[0] = 91
    elif fault == "negative":
        lens[0] = -1
    elif fault == "len":
        pool.lens[1] = 97
    elif fault == "pages":
        pool.used = 49
    else:
        pool.used = -1
    d, lens_out, used, copies = _fork(pool, parents, children, lens, in_place)
    d.equals(pool, lens_out, used)
    assert copies.tolist() == [[-1, -1, 0]] * 4
    _bad_value()


def test_fork_of_odd_pages(lib):
    pool = Pool(np.arange(48).reshape(8, 6), [90, 33, 0, 0, 0, 0, 0, 0], np.zeros(50), np.arange(50), 47, 16)
    pool.table[0, 1], pool.table[1, 2], pool.free[47] = 50, -4, 2 ** 30
    d, lens, used, copies = _fork(pool, [0, 1], [4, 5])
    assert copies.tolist() == [[-1, -1, 0]] * 2 and used.item() == 49
    assert lens.tolist() == [90, 33, 0, 0, 90, 33, 0, 0]
    assert d.table[4].tolist() == [0, 50, 2, 3, 4, 2 ** 30] and d.table[5, :3].tolist() == [6, 7, 48]
    assert d.shares.nonzero()[:, 0].tolist() == [0, 2, 3, 4, 6, 7]
    _bad_value()


def test_fork_and_free_of_nothing(lib):
    pool = random_pool(np.random.default_rng(1), 5, 16, 100)
    for in_place in (False, True):
        d, lens, used, _ = _fork(pool, [], [], in_place=in_place)
        d.equals(pool, lens, used)
        d, lens, used = _free(pool, [], in_place=in_place)
        d.equals(pool, lens, used)
    none = Pool(np.zeros((0, 3)), [], np.zeros(0), [], 0, 16)
    d, lens, used = _free(none, [-1])
    d.equals(none, lens, used)
    d, lens, used, copies = _fork(none, [-1, -2], [0, 0])
    assert copies.tolist() == [[-1, -1, 0]] * 2
    _ok()


# ---------------------------------------------------------------- compact

@both_places
@pytest.mark.parametrize("share", [1.0, 0.3, 0.0], ids=["all", "some", "none"])
@each_size
def test_compact(lib, size, share, in_place):
    B, page, longest = size
    rng = np.random.default_rng(B * 5 + page)
    pool = random_pool(rng, B, page, longest, spare=int(rng.integers(0, 2 * B + 60)))
    full = pool.copy()
    need = int((full.compact(len(pool.shares))[:, 0] >= 0).sum())
    most = int(share * need) + (9 if share == 1.0 else 0)
    want = pool.copy()
    moves = want.compact(most)
    d = Device(pool)
    out = (d.table, d.shares, d.free) if in_place else tuple(torch.full_like(x, 88) for x in (
        d.table, d.shares, d.free))
    got = torch.full((most, 3), 44, dtype=torch.int32, device="cuda")
    binding.fa_paged_compact(d.lens, d.table, d.shares, d.free, d.used, *out, got, page)
    d.equals(want, table=out[0], shares=out[1], free=out[2], free_from=pool.used)
    assert np.array_equal(got.cpu().numpy(), moves)
    if share == 1.0:
        held = np.nonzero(want.holders())[0]
        assert not len(held) or not (want.free[want.used:] < held.max()).any()
    _ok()


@both_places
@pytest.mark.parametrize("fault", ["table", "below", "list", "twice", "both", "len", "long", "used"])
def test_compact_that_cannot_be_met_changes_nothing(lib, fault, in_place):
    pool = Pool(np.r_[np.arange(20, 44)].reshape(4, 6), [90, 33, 0, 5], np.zeros(50),
                np.r_[np.arange(20, 44), np.arange(20)], 24, 16)
    if fault == "table":
        pool.table[1, 2] = 50
    elif fault == "below":
        pool.table[0, 0] = -1
    elif fault == "list":
        pool.free[30] = 1 << 22
    elif fault == "twice":
        pool.free[30] = pool.free[31]
    elif fault == "both":
        pool.free[30] = 20
    elif fault == "len":
        pool.lens[3] = -2
    elif fault == "long":
        pool.lens[3] = 97
    else:
        pool.used = 45
    d = Device(pool)
    out = (d.table, d.shares, d.free) if in_place else tuple(torch.full_like(x, 88) for x in (
        d.table, d.shares, d.free))
    moves = torch.full((9, 3), 44, dtype=torch.int32, device="cuda")
    binding.fa_paged_compact(d.lens, d.table, d.shares, d.free, d.used, *out, moves, pool.page)
    d.equals(pool, table=out[0], shares=out[1], free=out[2], free_from=pool.used)
    assert moves.tolist() == [[-1, -1, 0]] * 9
    _bad_value()


# ------------------------------------------------------------------- copy

def _bits(c):
    return c.contiguous().view(torch.uint8)


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("shape", [
    # layers, pages, K, page, H, layout, pad, moves
    (0, 9, 1, 1, 64, "head", 0, 3), (0, 40, 3, 16, 128, "head", 32, 17), (2, 40, 3, 16, 128, "token", 0, 17),
    (3, 12, 8, 64, 256, "head", 16, 5), (0, 12, 5, 256, 64, "token", 0, 5), (1, 700, 2, 4, 64, "token", 16, 300),
    (0, 6, 7, 1024, 128, "head", 0, 2)], ids=lambda s: "L%d_pages%d_K%d_page%d_H%d_%s_%d_%d" % s)
def test_copy(lib, shape, dtype):
    L, n, K, page, H, layout, pad, count = shape
    gen = torch.Generator().manual_seed(n + H)
    rng = np.random.default_rng(n)
    perm = rng.permutation(n)
    moves = [(int(perm[0 if i < 2 else i]), int(perm[n - 1 - i]), int(rng.integers(0, page + 1)))
             for i in range(min(count, n // 2))]
    moves[0] = (moves[0][0], moves[0][1], page)
    moves.insert(1, (-1, -1, 0))
    caches = [torch.stack([P.cache(n, K, page, H, dtype, layout, gen, pad=pad) for _ in range(L or 1)])
              for _ in range(2)]
    if pad:     # torch.stack drops the gap: give pages their stride back
        wide = [torch.full((L or 1, n, K * page * H + pad), 3.0).to(dtype) for _ in range(2)]
        views = []
        for w, c in zip(wide, caches):
            inner = (K, page) if layout == "head" else (page, K)
            v = w.as_strided((L or 1, n, *inner, H), (w.stride(0), w.stride(1), inner[1] * H, H, 1))
            v = v if layout == "head" else v.transpose(2, 3)
            v.copy_(c)
            views.append(v)
        caches = views
    elif layout == "token":
        caches = [c.transpose(2, 3).contiguous().transpose(2, 3) for c in caches]
    dev = [P.to_device(c, "cuda") for c in caches]
    before = [_bits(c).clone() for c in caches]
    binding.fa_paged_copy(_i32(moves), *(dev if L else [c[0] for c in dev]))
    torch.cuda.synchronize()
    for b, c in zip(before, dev):
        want = b.clone()
        for src, dst, tokens in moves:
            if src >= 0:
                want[:, dst, :, :tokens] = b[:, src, :, :tokens]
        assert torch.equal(_bits(c.cpu()), want)
        if pad:
            gap = c.as_strided((L or 1, n, pad), (c.stride(0), c.stride(1), 1), c.storage_offset() + K * page * H)
            assert (gap.float() == 3.0).all()
    _ok()


def test_copy_of_odd_moves(lib):
    caches = [torch.randn((5, 2, 16, 64), device="cuda").bfloat16() for _ in range(2)]
    want = [c.clone() for c in caches]
    moves = [(0, 5, 3), (-1, 2, 3), (0, -1, 3), (1, 2, 17), (1, 2, -1), (7, 2, 3), (3, 4, 2), (-7, -2, 99)]
    for w in want:
        w[4, :, :2] = w[3, :, :2]
    binding.fa_paged_copy(_i32(moves), *caches)
    torch.cuda.synchronize()
    assert all(torch.equal(c, w) for c, w in zip(caches, want))
    _bad_value()
    binding.fa_paged_copy(_i32(np.zeros((0, 3))), *caches)
    binding.fa_paged_copy(_i32(moves), *(c[None][:0] for c in caches))
    _ok()


def test_copy_past_32_bits(lib):
    """A page that begins 5 GB into the cache."""
    caches = [torch.empty((2600, 8, 1024, 128), dtype=BF16, device="cuda") for _ in range(2)]
    for c in caches:
        c[2599] = torch.randn(c.shape[1:], device="cuda").bfloat16()
        c[3] = 0
    binding.fa_paged_copy(_i32([(2599, 3, 1000)]), *caches)
    for c in caches:
        assert torch.equal(c[3, :, :1000], c[2599, :, :1000]) and not c[3, :, 1000:].any()
    _ok()


# --------------------------------------------------------------- together

def test_a_server_of_forks(lib):
    """Requests grow, fork, are cut, end and are compacted for 40 steps, in place; every request's tokens
    stay its own."""
    rng = np.random.default_rng(8)
    B, page, K, H, n_pages, cols = 12, 8, 2, 64, 150, 30
    d = Device(Pool(np.full((B, cols), -1), np.zeros(B), np.zeros(n_pages), rng.permutation(n_pages), 0, page))
    host = Pool(np.full((B, cols), -1), np.zeros(B), np.zeros(n_pages), d.free.cpu().numpy(), 0, page)
    caches = [torch.zeros((2, n_pages, K, page, H), dtype=BF16, device="cuda") for _ in range(2)]
    texts, fresh = [[] for _ in range(B)], 0
    for step in range(40):
        # growth
        new = np.array([int(rng.integers(0, 12)) if rng.random() < 0.6 and len(t) < 180 else 0 for t in texts])
        while sum(up(len(t) + int(n), page) - up(len(t), page) for t, n in zip(texts, new)) > n_pages - host.used:
            new[int(np.argmax(new))] = 0
        total = int(new.sum())
        lens, starts, slots, positions, used = binding.paged_tables(
            d.lens, _i32(new), d.free, d.used, d.table, n_pages=n_pages, page_size=page, max_tokens=total + 3)
        d.lens, d.used = lens, used
        kv = torch.zeros((total + 3, K, H), dtype=BF16, device="cuda")
        ids = torch.arange(fresh, fresh + total) % 251
        kv[:total] = ids.to(BF16)[:, None, None].cuda()
        for layer in range(2):
            binding.fa_paged_append(kv, kv + 1, slots, caches[0][layer], caches[1][layer])
        for b in range(B):
            for j in range(up(len(texts[b]), page), up(len(texts[b]) + int(new[b]), page)):
                host.table[b, j] = host.free[host.used]
                host.used += 1
            texts[b] = texts[b] + [(fresh + i) % 251 for i in range(int(new[b]))]
            fresh += int(new[b])
        host.lens[:] = [len(t) for t in texts]
        # some end, some are cut
        rows = [r for r in rng.permutation(B) if rng.random() < 0.3]
        keep = [k if rng.random() < 0.6 else 0 for k in _cuts(host, rng, rows)]
        binding.paged_free(_i32(rows), d.lens, d.table, d.shares, d.free, d.used, page_size=page, keep=_i32(keep))
        host.free_rows(rows, keep)
        for r, k in zip(rows, keep):
            texts[r] = texts[r][:k]
        # some fork
        living, empty = np.nonzero(host.lens)[0], np.nonzero(host.lens == 0)[0]
        if len(living) and len(empty) <= n_pages - host.used:
            parents = rng.choice(living, len(empty))
            copies = binding.paged_fork(_i32(parents), _i32(empty), d.lens, d.table, d.shares, d.free, d.used,
                                        page_size=page)
            host.fork(parents, empty)
            binding.fa_paged_copy(copies, *caches)
            for p, c in zip(parents, empty):
                texts[c] = list(texts[p])
        if step % 3 == 2:
            most = int(rng.integers(1, 40))
            moves = binding.paged_compact(d.lens, d.table, d.shares, d.free, d.used, page_size=page, max_moves=most)
            assert np.array_equal(moves.cpu().numpy(), host.compact(most))
            binding.fa_paged_copy(moves, *caches)
        host.check()
        d.equals(host, free_from=host.used)
        for b, text in enumerate(texts):
            for i, x in enumerate(text):
                p = int(host.table[b, i // page])
                if i % 7 == 0 or i == len(text) - 1:
                    for c, add in zip(caches, (0, 1)):
                        want = float(torch.tensor(float(x)).bfloat16() + add)
                        assert c[1, p, 1, i % page, 5].item() == pytest.approx(want, abs=0.51)
    _ok()


def test_free_and_fork_in_a_graph_on_a_side_stream(lib):
    """A beam step captured once and replayed on what the replays before it have left."""
    pool = random_pool(np.random.default_rng(5), 9, 16, 300, spare=60, fork=0, pinned=0)
    pool.free_rows([0, 2, 4, 6])
    living = [b for b in range(9) if pool.lens[b]]
    parents = [living[i % len(living)] for i in range(4)]
    children = [0, 2, 4, 6]
    pool.check()
    d = Device(pool)
    ch, pa = _i32(children), _i32(parents)
    copies = torch.zeros((4, 3), dtype=torch.int32, device="cuda")
    caches = [torch.zeros((len(pool.shares), 2, 16, 64), dtype=BF16, device="cuda") for _ in range(2)]

    def step():
        binding.fa_paged_free(ch, d.lens, d.table, d.shares, d.free, d.used, d.lens, d.used, 16)
        binding.fa_paged_fork(pa, ch, d.lens, d.table, d.shares, d.free, d.used, d.lens, copies, d.used, 16)
        binding.fa_paged_copy(copies, *caches)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
        for _ in range(3):
            graph.replay()
            pool.free_rows(children)
            want = pool.fork(parents, children)
    side.synchronize()
    pool.check()
    d.equals(pool)
    assert np.array_equal(copies.cpu().numpy(), want)
    _ok()
