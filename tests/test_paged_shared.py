"""Attention of requests that share prefixes on the GPU against the plain 64-bit decode (_paged.py), which
knows nothing of sharing.

Tolerance: that of the decode (_paged.check_decode).  The join of a prefix's and a request's own sums adds
two factors 2^(m_p - M), each off by 2^-21 with its argument, and three fp32 operations: below 16 * 2^-24
in all, which is the rounding of 16 more keys' sums."""
import math

import pytest
import torch

from flash_attention_gqa_gb300 import binding
import _paged as P

pytestmark = pytest.mark.gpu
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _ok():
    torch.cuda.synchronize()
    assert binding.fa_check_status() == binding.FA_OK


class Problem:
    """groups: (prefix, tokens of each member behind it); alone: lengths of requests in no group.  Requests
    are shuffled; full pages of a prefix are shared, the tokens of a last one that is not full are copies;
    what no request owns is NaN."""

    def __init__(self, seed, groups, alone=(), *, K, G, T, H, page, dtype=BF16, layout="head", pad=0, wide=True):
        gen = torch.Generator().manual_seed(seed)
        sizes = [(p, t, g) for g, (p, tails) in enumerate(groups) for t in tails] + [(0, n, -1) for n in alone]
        B = len(sizes)
        row = torch.randperm(B, generator=gen).tolist()       # request of each
        need = sum(P.up(p + t, page) for p, t, _ in sizes)
        perm = torch.randperm(need + 3, generator=gen).tolist()
        # wide: a table that reaches far enough for the groups to be looked at (small calls do not)
        width = max([P.up(p + t, page) for p, t, _ in sizes] + [0, (1 << 20) // page if wide else 0]) + 2
        table, lens = torch.full((B, width), -1, dtype=torch.int32), [0] * B
        owned = torch.zeros(need + 3, page, dtype=torch.bool)
        at, first, copies = 0, {}, []
        self.members, self.starts, self.prefix = [], [0], [p for p, _ in groups]
        for i, (p, t, g) in enumerate(sizes):
            b, n = row[i], p + t
            lens[b] = n
            full = p // page if g in first else 0
            for j in range(P.up(n, page)):
                if j < full:
                    table[b, j] = table[first[g], j]
                    continue
                table[b, j] = perm[at]
                at += 1
                owned[int(table[b, j]), :min(page, n - j * page)] = True
                if g in first and j == full and p % page:
                    copies.append((int(table[first[g], j]), int(table[b, j]), p % page))
            first.setdefault(g, b)
        for g, (_, tails) in enumerate(groups):
            k = self.starts[-1]
            self.members += row[k:k + len(tails)]
            self.starts.append(k + len(tails))
        self.q = (torch.randn((B, K, G, T, H), generator=gen) * H ** -0.5).to(BF16)
        self.caches = []
        for _ in range(2):
            c = P.cache(need + 3, K, page, H, torch.float32, layout, gen, pad=pad)
            if dtype == E4M3:
                c.mul_(32)
            for src, dst, n in copies:
                c[dst, :, :n] = c[src, :, :n]
            c.copy_(torch.where(owned[:, None, :, None], c, torch.tensor(float("nan"))))
            raw = c.as_strided((c.untyped_storage().nbytes() // 4,), (1,)).to(dtype)
            self.caches.append(raw.as_strided(c.shape, c.stride()))
        self.scales = [None, None]
        if dtype == E4M3:
            self.scales = [(torch.rand(K, generator=gen) + 0.5) / 32 for _ in range(2)]
        self.table, self.lens, self.H, self.e4m3 = table, torch.tensor(lens, dtype=torch.int32), H, dtype == E4M3

    def on_device(self):
        self.dev = [P.to_device(c, "cuda") for c in self.caches]
        self.args = (self.q.cuda(), *self.dev, self.table.cuda(), self.lens.cuda())
        self.kw = dict(zip(("k_scale", "v_scale"), (None if s is None else s.cuda() for s in self.scales)))
        return self

    def run(self, members=None, starts=None, prefix=None, **kw):
        return binding.paged_attention_decode_shared(
            *self.args, _i32(self.members if members is None else members),
            _i32(self.starts if starts is None else starts), _i32(self.prefix if prefix is None else prefix),
            **self.kw, **kw)

    def check(self, o, lse, want=None):
        torch.cuda.synchronize()
        want = want or P.decode(self.q, *self.caches, self.table, self.lens, *self.scales)
        n = int(self.lens.max()) if len(self.lens) else 0
        P.check_decode(o.cpu(), lse.cpu(), want, self.H, self.e4m3, n + 16)
        return want


CASES = {
    "pair": ([(16, [1, 1])], [], dict(K=1, G=1, T=1, H=64, page=16)),
    "one_key": ([(1, [1, 2, 3])], [1], dict(K=2, G=2, T=1, H=64, page=1)),
    "alone": ([], [5, 0, 300, 77], dict(K=2, G=4, T=1, H=128, page=16)),
    "single_member": ([(64, [9]), (32, [1, 40])], [], dict(K=2, G=8, T=1, H=128, page=16)),
    "samples": ([(512, [1, 30, 100, 7, 64, 65, 2, 500, 128, 127, 129, 3])], [40], dict(K=2, G=8, T=1, H=128, page=16)),
    "chunks": ([(130, list(range(1, 38)))], [], dict(K=1, G=7, T=1, H=64, page=2)),      # 259 rows: 3 chunks
    "straddle": ([(96, [3] * 9)], [], dict(K=3, G=5, T=3, H=128, page=32)),              # 135 rows
    "odd_prefix": ([(100, [5, 60, 1]), (7, [2, 2])], [3], dict(K=2, G=4, T=1, H=128, page=16)),
    "odd_prefix_h256": ([(333, [5, 60, 1, 9])], [], dict(K=1, G=3, T=2, H=256, page=64)),
    "drafts": ([(200, [8, 9, 70]), (0, [20, 30]), (8, [8, 8])], [8, 100], dict(K=2, G=4, T=8, H=128, page=8)),
    "full_rows": ([(256, [16, 17, 300])], [], dict(K=2, G=8, T=16, H=128, page=32)),     # G * T = 128
    "rows40": ([(192, [9, 64, 3, 10])], [50], dict(K=2, G=8, T=5, H=64, page=64)),
    "rows20_h256": ([(192, [9, 64, 200])], [50], dict(K=1, G=4, T=5, H=256, page=16)),
    "long": ([(6000, [40, 3])], [], dict(K=1, G=8, T=1, H=128, page=64)),
    "long_h256": ([(3000, [40, 3, 1])], [], dict(K=1, G=16, T=1, H=256, page=8)),
    "prompts": ([(16 * i, [1 + 5 * j for j in range(i)]) for i in range(1, 9)], [1, 2, 200],
                dict(K=2, G=4, T=1, H=128, page=16)),
    "many": ([(64, [1 + i % 9 for i in range(40)]) for _ in range(8)], [], dict(K=1, G=2, T=1, H=64, page=16)),
    "big_page": ([(100, [5, 6])], [], dict(K=2, G=2, T=1, H=64, page=256)),
    "padded": ([(48, [5, 6, 30])], [9], dict(K=3, G=8, T=1, H=64, page=16, pad=32)),
    "token_layout": ([(80, [5, 6, 30, 90])], [9], dict(K=4, G=8, T=1, H=128, page=16, layout="token")),
}


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("wide", [True, False], ids=["wide", "narrow"])
@pytest.mark.parametrize("name", CASES)
def test_shared(lib, name, wide, dtype):
    groups, alone, kw = CASES[name]
    p = Problem(len(name), groups, alone, dtype=dtype, wide=wide, **kw).on_device()
    o, lse = p.run()
    p.check(o, lse)
    o2, lse2 = p.run()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    # a prefix that ends behind what some first query sees is cut, and reported
    if wide and any(len(tails) > 0 and min(tails) < kw["T"] - 1 for _, tails in groups):
        assert binding.fa_check_status() == binding.FA_ERR_DEVICE_VALUE
    _ok()


@pytest.mark.parametrize("T", [1, 4])
def test_prefix_up_to_the_last_visible_key(lib, T):
    """A prefix may reach to the first query's last key: queries then have few keys of their own, or none."""
    p = Problem(3, [(65, [T - 1, T - 1, 40])], K=2, G=4, T=T, H=128, page=16).on_device()
    p.check(*p.run())
    _ok()


FAULTS = ["prefix", "negative", "member", "below", "twice", "twice_elsewhere", "falls", "past", "first",
          "nobody", "len"]


@pytest.mark.parametrize("fault", FAULTS)
def test_groups_that_do_not_hold_together(lib, fault):
    """Reported, and the result is right all the same."""
    least = 0 if fault == "prefix" else 2       # (a first query that does not see the whole prefix)
    p = Problem(9, [(64, [2, 9, 40]), (32, [7, 100, 3, least])], [12], K=2, G=4, T=2, H=128, page=16)
    members, starts, prefix = list(p.members), list(p.starts), list(p.prefix)
    if fault == "negative":
        prefix[0] = -5
    elif fault == "member":
        members[1] = 8
    elif fault == "below":
        members[0] = -1
    elif fault == "twice":
        members[4] = members[3]
    elif fault == "twice_elsewhere":
        members[5] = members[0]
    elif fault == "falls":
        starts[1] = 8
    elif fault == "past":
        starts[2] = 8
    elif fault == "first":
        starts[0] = -1
    elif fault == "nobody":
        members = [-1, 8, 99] + members[3:]
    elif fault == "len":
        p.lens[p.members[4]] = -3
    p.on_device()
    o, lse = p.run(members, starts, prefix)
    torch.cuda.synchronize()
    assert binding.fa_check_status() == binding.FA_ERR_DEVICE_VALUE
    if fault == "len":
        p.lens[p.members[4]] = 0
        want = P.decode(p.q, *p.caches, p.table, p.lens)
        p.check(o, lse, want)
    else:
        p.check(o, lse)
    _ok()


def test_tables_with_pages_out_of_range(lib):
    """Of a prefix and of a request's own: their keys count as zeros, as in the decode."""
    p = Problem(5, [(64, [1, 9, 40])], [30], K=2, G=4, T=1, H=64, page=16)
    first = int(p.table[p.members[0], 1])
    p.table[p.table == first] = 10 ** 6
    p.table[p.members[2], 5] = -1
    p.on_device()
    o, lse = p.run()
    torch.cuda.synchronize()
    assert binding.fa_check_status() == binding.FA_ERR_DEVICE_VALUE
    zeros = [torch.cat([torch.nan_to_num(c.float()), torch.zeros_like(c[:1].float())]) for c in p.caches]
    table = p.table.clone()
    table[(table < 0) | (table >= len(p.caches[0]))] = len(p.caches[0])
    want = P.decode(p.q, *zeros, table, p.lens)
    P.check_decode(o.cpu(), lse.cpu(), want, 64, False, 120)
    _ok()


def test_empty_and_masked_rows(lib):
    """Requests without tokens, and with fewer than T, beside sharing ones."""
    p = Problem(6, [(16, [2, 5])], [0, 1, 2, 0], K=2, G=2, T=3, H=64, page=4).on_device()
    o, lse = p.run(prefix=[16])
    p.check(o, lse)
    assert (lse == -math.inf).any()
    _ok()


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_values_that_are_not_finite(lib, dtype):
    """A NaN or infinite value reaches the rows that keep its key, and no other."""
    p = Problem(7, [(40, [5, 6, 9])], [20], K=2, G=2, T=4, H=64, page=16, dtype=dtype)
    a, b = p.members[0], p.members[1]
    v = p.caches[1]
    last = int(p.lens[a]) - 1           # the newest token of one request: its last query only
    v[int(p.table[a, last // 16]), 0, last % 16, 3] = math.nan
    alone = [x for x in range(4) if x not in p.members][0]
    v[int(p.table[alone, 0]), 1, 2, 7] = math.inf if dtype == BF16 else math.nan
    p.on_device()
    o, lse = p.run()
    torch.cuda.synchronize()
    bad = ~torch.isfinite(o.cpu())
    want = torch.zeros_like(bad)
    want[a, 0, :, 3, 3] = True
    want[alone, 1, :, :, 7] = True
    assert torch.equal(bad, want) and torch.isfinite(lse).all()
    assert b != a
    _ok()


def test_more_requests_than_a_wave(lib):
    groups = [(32, [1 + (i * 7 + g) % 40 for i in range(9)]) for g in range(30)]
    p = Problem(8, groups, [3] * 30, K=4, G=2, T=1, H=64, page=16).on_device()
    p.check(*p.run())
    _ok()


# With two items or more for each CTA the requests' own keys go to single warps.
def _tails(n, most, least=1):
    return [least + (i * 37 + i * i) % most for i in range(n)]


WARPS = {
    "h128_rows8": ([(100, _tails(16, 90))] * 20, [0, 1, 33], dict(K=2, G=8, T=1, H=128, page=16)),
    "h128_rows16": ([(64, _tails(16, 60, 4))] * 20, [0, 1, 3, 40], dict(K=2, G=4, T=4, H=128, page=32)),
    "h256_rows8": ([(33, _tails(16, 70, 2))] * 10, [0, 1, 50], dict(K=2, G=4, T=2, H=256, page=16)),
    "h64_rows32": ([(40, _tails(20, 50, 4))] * 16, [0, 2, 70], dict(K=2, G=8, T=4, H=64, page=8)),
    "h64_rows16": ([(40, _tails(20, 50, 8))] * 16, [0, 7, 70], dict(K=2, G=2, T=8, H=64, page=4)),
    "one_head": ([(16, _tails(14, 40))] * 48, [5] * 30, dict(K=1, G=3, T=1, H=64, page=256)),
    "long_and_short": ([(32, [900] + [1] * 40)] * 8, [700, 1], dict(K=2, G=4, T=1, H=128, page=64)),
    "one_long": ([(32, [2000] + [1] * 319)], [], dict(K=2, G=1, T=1, H=64, page=64, layout="token")),
}


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("name", WARPS)
def test_own_keys_by_warps(lib, name, dtype):
    groups, alone, kw = WARPS[name]
    p = Problem(len(name), groups, alone, dtype=dtype, **kw).on_device()
    assert len(p.lens) * kw["K"] >= 2 * 152 * (1 if kw["H"] == 256 else 2)
    o, lse = p.run()
    p.check(o, lse)
    o2, lse2 = p.run()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    _ok()


# Small calls are decodes, by warps where there are four short items or more for each CTA.
SMALL = {
    "h128_rows8": ([(16, _tails(17, 70))] * 20, [0, 1, 33], dict(K=4, G=8, T=1, H=128, page=16)),
    "h128_rows16": ([(16, _tails(17, 60, 4))] * 20, [0, 1, 3, 40], dict(K=4, G=4, T=4, H=128, page=16)),
    "h256_rows8": ([(33, _tails(16, 40, 2))] * 10, [0, 1, 50], dict(K=4, G=4, T=2, H=256, page=8)),
    "h64_rows32": ([(8, _tails(20, 50, 4))] * 17, [0, 2, 70], dict(K=4, G=8, T=4, H=64, page=8)),
    "h64_rows8": ([(7, _tails(20, 50))] * 31, [0, 70], dict(K=4, G=1, T=1, H=64, page=1)),
    "longer": ([(64, _tails(31, 150))] * 20, [0, 200], dict(K=4, G=2, T=1, H=64, page=16, layout="token")),
}


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("name", SMALL)
def test_small_calls_by_warps(lib, name, dtype):
    groups, alone, kw = SMALL[name]
    p = Problem(len(name), groups, alone, dtype=dtype, wide=False, **kw).on_device()
    each = len(p.lens) * kw["K"] // (152 if kw["H"] == 256 else 304)
    assert each >= 4 and p.table.shape[1] * kw["page"] <= (256 if each >= 8 else 128)
    o, lse = p.run()
    p.check(o, lse)
    o2, lse2 = p.run()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    _ok()


def test_agrees_with_the_decode_on_a_large_case(lib):
    """64 samples of an 8000-token prompt, 8 kv heads: against the decode without sharing, both rounded
    to bf16 once."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    B, K, G, H, page, prefix = 64, 8, 8, 128, 64, 8000 // 64 * 64
    own = torch.randint(1, 600, (B,), generator=torch.Generator().manual_seed(2))
    held = [P.up(int(n), page) for n in own]
    n_pages = prefix // page + sum(held)
    perm = torch.randperm(n_pages, generator=torch.Generator().manual_seed(3)).int()
    table = torch.full((B, prefix // page + max(held)), -1, dtype=torch.int32)
    at = prefix // page
    table[:, :at] = perm[:at]
    for b in range(B):
        table[b, prefix // page:prefix // page + held[b]] = perm[at:at + held[b]]
        at += held[b]
    caches = [torch.randn((n_pages, K, page, H), generator=gen, device="cuda").to(BF16) for _ in range(2)]
    q = (torch.randn((B, K, G, 1, H), generator=gen, device="cuda") * H ** -0.5 * 3).to(BF16)
    lens = (own + prefix).int().cuda()
    o, lse = binding.paged_attention_decode_shared(q, *caches, table.cuda(), lens, _i32(list(range(B))),
                                                   _i32([0, B]), _i32([prefix]))
    ro, rl = binding.paged_attention_decode(q, *caches, table.cuda(), lens)
    torch.cuda.synchronize()
    assert (lse - rl).abs().max() <= 2e-5
    # (two roundings to bf16 apart, of values that differ by their fp32 sums)
    size = ro.abs().float().amax(-1, keepdim=True)
    assert ((o.float() - ro.float()).abs() <= 2.0 ** -7 * ro.float().abs() + 2.0 ** -13 * size).all()
    _ok()


def test_graphs_and_streams(lib):
    """Captured with growing lengths and replayed; the same workspace in two graphs, one after the other."""
    p = Problem(11, [(64, [4, 9, 40]), (32, [7, 8])], [12], K=2, G=4, T=1, H=128, page=64).on_device()
    q, kc, vc, table, lens = p.args
    m, s, f = _i32(p.members), _i32(p.starts), _i32(p.prefix)
    n = binding.fa_paged_decode_shared_workspace_size(6, 2, 4, 1, 128, 2, 5)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)
    side, graphs, outs = torch.cuda.Stream(), [], []
    for _ in range(2):
        o, lse = torch.empty_like(q), torch.empty((6, 2, 4, 1), device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            with torch.cuda.graph(graph, stream=side):
                binding.fa_paged_decode_shared(q, kc, vc, table, lens, m, s, f, o, lse, ws)
        graphs.append(graph)
        outs.append((o, lse))
    for step in range(3):
        for g in graphs:
            g.replay()
        for o, lse in outs:
            p.check(o, lse)
        assert torch.equal(outs[0][0], outs[1][0])
        lens -= 1
        p.lens -= 1
        q.mul_(-1)
        p.q = -p.q
        if step < 2:
            f.sub_(16)
    o, lse = binding.paged_attention_decode_shared(*p.args, m, s, f, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    p.check(o, lse)
    _ok()


def test_waits_that_run_out_are_reported(lib):
    """The prefix kernel's waits on its copies, with no time at all: an error, and the next call is right."""
    p = Problem(12, [(640, [4, 9, 40, 11])], [12], K=2, G=8, T=1, H=128, page=64).on_device()
    want = p.check(*p.run())
    binding.fa_set_wait_limit_ns(1)
    try:
        p.run()
        torch.cuda.synchronize()
        assert binding.fa_check_status() in (binding.FA_ERR_DEVICE_TIMEOUT, binding.FA_OK)
    finally:
        binding.fa_set_wait_limit_ns(2_000_000_000)
    p.check(*p.run(), want)
    _ok()
