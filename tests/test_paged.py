"""The paged cache operators on the GPU against plain 64-bit forms (_paged.py): tables, append,
decode, and the three together as a serving program runs them."""
import math

import numpy as np
import pytest
import torch

import oracle
from flash_attention_gqa_gb300 import binding
import _paged as P

pytestmark = pytest.mark.gpu
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _ok():
    torch.cuda.synchronize()
    assert binding.fa_check_status() == binding.FA_OK


# ------------------------------------------------------------------ tables

def _tables_case(seed, B, page, c_hi, n_hi, pad=5, max_pages=None):
    rng = np.random.default_rng(seed)
    cached = rng.integers(0, c_hi + 1, B)
    new = rng.integers(0, n_hi + 1, B)
    cached[rng.random(B) < 0.2] = 0
    new[rng.random(B) < 0.2] = 0
    cols = max([P.up(int(a + b), page) for a, b in zip(cached, new)] + [1]) + 2
    cols = max_pages or cols
    held = [P.up(int(c), page) for c in cached]
    need = sum(P.up(int(a + b), page) for a, b in zip(cached, new)) - sum(held)
    n_pages = sum(held) + need + 9
    perm = rng.permutation(n_pages)
    table = np.full((B, cols), -7, dtype=np.int64)
    at = 0
    for b in range(B):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    return cached, new, perm[at:], 4, table, page, int(new.sum()) + pad, n_pages


def _run_tables(case, in_place=False, positions=True):
    cached, new, free, used, table, page, max_tokens, n_pages = case
    c, n, f, u, t = _i32(cached), _i32(new), _i32(free), _i32([used]), _i32(table)
    total = c if in_place else torch.empty_like(c)
    u_out = u if in_place else torch.empty_like(u)
    starts = torch.empty(len(cached) + 1, dtype=torch.int32, device="cuda")
    slots = torch.full((max_tokens,), 99, dtype=torch.int64, device="cuda")
    pos = torch.full((max_tokens,), 99, dtype=torch.int32, device="cuda") if positions else None
    binding.fa_paged_tables(c, n, f, u, t, total, starts, slots, pos, u_out, n_pages, page)
    torch.cuda.synchronize()
    return [x if x is None else x.cpu().numpy() for x in (t, total, starts, slots, pos, u_out)]


TABLES = [  # seed, B, page, largest cached, largest new
    (0, 1, 16, 0, 1), (1, 1, 16, 100, 1), (2, 3, 1, 9, 5), (3, 64, 16, 500, 1),
    (4, 33, 64, 300, 700), (5, 1000, 16, 90, 3), (6, 1025, 8, 40, 9), (7, 8192, 16, 40, 2),
    (8, 5, 65536, 70000, 70000), (9, 40, 32, 10, 4000), (10, 2, 16, 3, 70000), (11, 2049, 2, 5, 40),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("shape", TABLES, ids=lambda s: f"B{s[1]}_page{s[2]}_c{s[3]}_n{s[4]}")
def test_tables(lib, shape, in_place):
    case = _tables_case(*shape)
    want = P.tables(case[0], case[1], case[2], case[3], case[4], case[5], case[6])
    got = _run_tables(case, in_place)
    for name, g, w in zip(("table", "total", "starts", "slots", "positions", "used"), got, want):
        assert np.array_equal(g.ravel(), np.asarray(w).ravel()), name
    _ok()


def test_tables_without_positions_and_without_requests(lib):
    case = _tables_case(1, 7, 16, 50, 9)
    want = P.tables(*case[:7])
    got = _run_tables(case, positions=False)
    assert np.array_equal(got[3], want[3]) and got[4] is None
    empty = (np.zeros(0, int), np.zeros(0, int), np.arange(3), 2, np.zeros((0, 4), int), 16, 6, 3)
    t, total, starts, slots, pos, used = _run_tables(empty)
    assert starts.tolist() == [0] and used.tolist() == [2]
    assert slots.tolist() == [-1] * 6 and pos.tolist() == [-1] * 6
    _ok()


@pytest.mark.parametrize("fault", ["tokens", "pages", "columns", "cached", "new", "used", "huge"])
def test_tables_that_cannot_be_met_change_nothing(lib, fault):
    case = list(_tables_case(3, 40, 16, 200, 30))
    cached, new, free, used, table, page, max_tokens, n_pages = case
    if fault == "tokens":
        case[6] = int(new.sum()) - 1
    elif fault == "pages":
        need = P.tables(*case[:7])[5]
        case[2] = free[:need - 1]
    elif fault == "columns":
        case[4] = table[:, :P.up(int((cached + new).max()), page) - 1]
    elif fault == "cached":
        cached[3] = -1
    elif fault == "new":
        new[39] = -1
    elif fault == "used":
        case[3] = -1
    else:
        new[0] = cached[0] = 2 ** 31 - 1
    t, total, starts, slots, pos, u = _run_tables(tuple(case))
    assert np.array_equal(t, case[4]) and np.array_equal(total, cached)
    assert not starts.any() and (slots == -1).all() and (pos == -1).all() and u[0] == case[3]
    assert binding.fa_check_status() == binding.FA_ERR_DEVICE_VALUE
    _ok()


def test_tables_page_ids_out_of_range_give_no_slot(lib):
    case = list(_tables_case(3, 4, 16, 40, 60))
    case[2] = np.array(case[2])
    case[2][case[3]] = case[7]          # the first page taken
    want = P.tables(*case[:7])
    got = _run_tables(tuple(case))
    slots = np.where(want[3] >= case[7] * 16, -1, want[3])
    assert (slots != want[3]).any() and np.array_equal(got[3], slots)
    assert np.array_equal(got[0], want[0])
    assert binding.fa_check_status() == binding.FA_ERR_DEVICE_VALUE


# ------------------------------------------------------------------ append

def _stored(x, scale):
    """What an e4m3 cache holds of x [N, K, H]: x / scale in fp32, saturated, rounded once."""
    return (x.float() / scale[None, :, None]).clamp(-448, 448).to(E4M3)


def _append_case(seed, N, K, H, page, dtype, layout, pad=0, skip=True, fused=True, n_pages=None):
    gen = torch.Generator().manual_seed(seed)
    n_pages = n_pages or P.up(N, page) + 3
    heads = 3 * K if fused else 2 * K
    kv = (torch.randn((N, heads, H), generator=gen) * 3).bfloat16()
    slots = torch.randperm(n_pages * page, generator=gen)[:N]
    if skip:
        slots[torch.rand(N, generator=gen) < 0.2] = -1
    caches = [P.cache(n_pages, K, page, H, dtype, layout, gen, fill=1.5, pad=pad) for _ in range(2)]
    scales = [None, None]
    if dtype == E4M3:
        scales = [torch.rand(K, generator=gen) / 10 + 0.003 for _ in range(2)]
    return kv[:, heads - 2 * K:heads - K], kv[:, heads - K:], slots, caches, scales


def _check_append(k, v, slots, caches, scales, page):
    dev = [P.to_device(c, "cuda") for c in caches]
    kv = [x.cuda() if x.is_contiguous() else P.to_device(x, "cuda") for x in (k, v)]
    s = [None if x is None else x.cuda() for x in scales]
    binding.fa_paged_append(*kv, slots.cuda(), *dev, *s)
    torch.cuda.synchronize()
    n_slots = caches[0].shape[0] * page
    for x, before, got, scale in zip((k, v), caches, dev, scales):
        put = x if scale is None else _stored(x, scale)
        bits = torch.int16 if scale is None else torch.uint8
        want = before.clone()
        for i, slot in enumerate(slots.tolist()):
            if 0 <= slot < n_slots:
                want.view(bits)[slot // page, :, slot % page] = put[i].contiguous().view(bits)
        assert torch.equal(got.cpu().contiguous().view(bits), want.contiguous().view(bits))


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("shape", [
    (1, 1, 64, 1, "head"), (7, 3, 64, 4, "token"), (64, 8, 128, 16, "token"),
    (130, 5, 128, 8, "head"), (300, 2, 256, 64, "head"), (33, 1, 256, 256, "token"),
    (1500, 8, 64, 32, "head")], ids=lambda s: "N%d_K%d_H%d_page%d_%s" % s)
def test_append(lib, shape, dtype):
    N, K, H, page, layout = shape
    case = _append_case(N, N, K, H, page, dtype, layout, pad=32 if N % 2 else 0, skip=N > 1,
                        fused=N % 3 != 0)
    _check_append(*case, page)
    _ok()


def test_append_slots_past_the_cache_are_skipped_and_reported(lib):
    k, v, slots, caches, scales = _append_case(5, 20, 2, 64, 8, BF16, "head", skip=False)
    n_slots = caches[0].shape[0] * 8
    slots[3], slots[11], slots[12] = n_slots, 2 ** 40, -2 ** 40
    _check_append(k, v, slots, caches, scales, 8)
    assert binding.fa_check_status() == binding.FA_ERR_DEVICE_VALUE
    _ok()


def test_append_e4m3_edges(lib):
    """Saturation, infinities, NaN, ties, subnormals and signed zeros, and no scales."""
    edge = torch.tensor([0.0, -0.0, math.inf, -math.inf, math.nan, 448.0, 464.0, 1e30, -449.0,
                         2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -11, 1.0625, 1.1875, -17.0, 2.0 ** -133])
    x = edge.repeat(4 * 64 // 16).reshape(2, 2, 64).bfloat16()
    for scales in ([torch.ones(2)] * 2, [torch.tensor([0.1, 7.0])] * 2):
        caches = [P.cache(3, 2, 4, 64, E4M3, "head", None, fill=1.0) for _ in range(2)]
        _check_append(x, x.clone(), torch.tensor([5, 0]), caches, scales, 4)
    dev = [P.to_device(P.cache(3, 2, 4, 64, E4M3, "head", None, fill=1.0), "cuda") for _ in range(2)]
    binding.fa_paged_append(x.cuda(), x.cuda(), torch.tensor([5, 0], device="cuda"), *dev)
    assert torch.equal(dev[0][1, :, 1].cpu().view(torch.uint8),
                       _stored(x, torch.ones(2))[0].contiguous().view(torch.uint8))
    _ok()


def test_append_of_nothing(lib):
    c = torch.zeros((2, 1, 8, 64), dtype=BF16, device="cuda")
    x = torch.zeros((0, 1, 64), dtype=BF16, device="cuda")
    binding.fa_paged_append(x, x, torch.zeros(0, dtype=torch.int64, device="cuda"), c, c.clone())
    _ok()


# ------------------------------------------------------------------ decode

def _decode(p, window=0, workspace=None):
    q, kc, vc, table, lens, ks, vs = p
    dev = [None if x is None else x.cuda() for x in (q, table, lens, ks, vs)]
    caches = [P.to_device(c, "cuda") for c in (kc, vc)]
    return binding.paged_attention_decode(dev[0], *caches, dev[1], dev[2], k_scale=dev[3],
                                          v_scale=dev[4], window=window, workspace=workspace)


def _check(p, window=0):
    o, lse = _decode(p, window)
    _ok()
    q, kc, vc, table, lens, ks, vs = p
    want = P.decode(q, kc, vc, table, lens, ks, vs, window)
    P.check_decode(o.cpu(), lse.cpu(), want, q.shape[-1], kc.dtype == E4M3,
                   int(lens.max()) if len(lens) else 0)
    return o, lse


LENS = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 200, 511, 700]


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("H", [64, 128, 256])
@pytest.mark.parametrize("heads", [(1, 1), (2, 8), (3, 5), (1, 16), (2, 9)],
                         ids=lambda h: "K%d_G%d" % h)
def test_decode(lib, heads, H, dtype):
    K, G = heads
    _check(P.problem(G, B=len(LENS), K=K, G=G, T=1, H=H, lens=LENS, page=16, dtype=dtype))


@pytest.mark.parametrize("page", [1, 2, 4, 8, 32, 64, 256, 1024, 65536])
@pytest.mark.parametrize("layout", ["head", "token"])
def test_decode_page_sizes_and_layouts(lib, page, layout):
    dtype, H = (BF16, 128) if page in (1, 8, 64, 1024) else (E4M3, 64)
    _check(P.problem(page, B=5, K=3, G=4, T=1, H=H, lens=[5, 0, 331, 64, 190], page=page,
                     dtype=dtype, layout=layout, pad=32 if page > 1 else 0,
                     spare=3 if page < 65536 else 0))


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("rows", [(4, 2), (8, 4), (1, 7), (17, 1), (3, 11), (5, 13), (16, 8), (1, 128),
                                  (128, 1)], ids=lambda r: "G%d_T%d" % r)
def test_decode_many_rows(lib, rows, dtype):
    """Several new tokens a request (causal among them; some lengths below T) and many heads."""
    G, T = rows
    for H in (64, 128, 256):
        _check(P.problem(T, B=6, K=2, G=G, T=T, H=H, lens=[0, 1, 6, 130, 77, 32], page=16,
                         dtype=dtype))


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("rows", [(16, 2), (8, 6), (12, 8), (128, 1)], ids=lambda r: "G%d_T%d" % r)
def test_decode_many_rows_of_long_requests(lib, rows, dtype):
    """The same, split over many CTAs, whose teams of warps and partials are joined."""
    G, T = rows
    for H in (64, 128, 256):
        _check(P.problem(H, B=3, K=2, G=G, T=T, H=H, lens=[2500, 17, 800], page=16, dtype=dtype))
        _check(P.problem(H, B=2, K=1, G=G, T=T, H=H, lens=[1100, 900], page=64, dtype=dtype), 333)


@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("window", [1, 2, 16, 50, 128, 10 ** 6, 2 ** 31 - 1])
def test_decode_window(lib, window, T):
    for dtype, H in ((BF16, 64), (E4M3, 128)):
        _check(P.problem(window % 97, B=6, K=2, G=3, T=T, H=H, lens=[0, 1, 49, 51, 300, 450],
                         page=8, dtype=dtype), window)


@pytest.mark.parametrize("case", [(1, 1, 8, 128, BF16, 20000), (1, 2, 4, 256, BF16, 9001),
                                  (2, 1, 8, 64, E4M3, 30011), (1, 8, 20, 128, BF16, 3333)],
                         ids=lambda c: "B%d_K%d_G%d_H%d_S%d" % (c[0], c[1], c[2], c[3], c[5]))
def test_decode_split_over_a_long_cache(lib, case):
    B, K, G, H, dtype, S = case
    _check(P.problem(3, B=B, K=K, G=G, T=1, H=H, lens=[S - 17 * b for b in range(B)], page=64,
                     dtype=dtype))


def test_decode_ragged_batch(lib):
    rng = np.random.default_rng(0)
    lens = [int(x) for x in np.exp(rng.uniform(0, math.log(1500), 300))]
    _check(P.problem(4, B=300, K=2, G=4, T=1, H=64, lens=lens, page=16))


@pytest.mark.parametrize("page", [1, 4, 8, 16, 128])
@pytest.mark.parametrize("rows", [(40, 1), (12, 5)], ids=lambda r: "G%d_T%d" % r)
def test_decode_many_rows_page_sizes_and_layouts(lib, rows, page):
    G, T = rows
    for H, layout, dtype in ((64, "head", BF16), (128, "token", BF16), (256, "token", BF16),
                             (128, "token", E4M3)):
        _check(P.problem(page, B=4, K=2, G=G, T=T, H=H, lens=[300, 3, 129, 64], page=page,
                         layout=layout, dtype=dtype, pad=32))


def test_decode_many_rows_ragged_batch(lib):
    """Several requests a CTA: the next one's queries arrive during the last one's end."""
    rng = np.random.default_rng(1)
    lens = [int(x) for x in np.exp(rng.uniform(0, math.log(900), 220))]
    for H, G, T in ((64, 33, 1), (128, 9, 4), (256, 40, 1)):
        p = P.problem(H, B=220, K=2, G=G, T=T, H=H, lens=lens, page=16)
        o, lse = _check(p)
        again = _decode(p)
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


def test_decode_many_rows_large_scores(lib):
    """The base of the exponents moves, and o with it, along the keys."""
    for H in (64, 128, 256):
        p = P.problem(9, B=3, K=1, G=64, T=1, H=H, lens=[900, 64, 1], page=16)
        q, kc, *_ = p
        kc.mul_(torch.linspace(0.05, 3, kc.shape[0])[:, None, None, None].bfloat16())
        _check(((q.float() * 40).bfloat16(), *p[1:]))


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("B", [3, 200])
@pytest.mark.parametrize("longest", [64, 256, 272, 512, 528])
def test_decode_short_tables(lib, B, longest, dtype):
    """Around the lengths up to which a request is not split, whose rule goes by the columns of
    the table; few and many requests."""
    rng = np.random.default_rng(longest)
    lens = [longest, 0, 1] + [int(x) for x in rng.integers(0, longest + 1, B - 3)]
    for H, G in ((64, 3), (128, 12)):
        _check(P.problem(5, B=B, K=2, G=G, T=1, H=H, lens=lens, page=16, dtype=dtype, extra_cols=0))
    _check(P.problem(6, B=B, K=2, G=8, T=2, H=64, lens=lens, page=16, dtype=dtype, extra_cols=90), 100)


def test_decode_large_scores(lib):
    """Scores in the hundreds: the running maximum carries them."""
    p = P.problem(9, B=3, K=2, G=4, T=1, H=128, lens=[700, 64, 1], page=16)
    p = ((p[0].float() * 60).bfloat16(), *p[1:])
    _check(p)


def test_decode_8bit_query_range(lib):
    """Query rows far from 1: rows of a magnitude that fp16 does not hold, and a row of zeros."""
    p = list(P.problem(10, B=2, K=1, G=8, T=1, H=64, lens=[100, 33], page=16, dtype=E4M3))
    size = torch.tensor([1e-30, 1e-8, 1.0, 3.0, 0.0, 1e-38, 1e-4, 20.0])[:, None, None]
    p[0] = (p[0].float() * size).bfloat16()
    _check(tuple(p))
    # far apart within a row, the large part on dims where every key is zero
    p[0][..., 0] = 1e5
    for c in (p[1],):
        c.view(torch.uint8)[..., 0] = 0
    _check(tuple(p))


@pytest.mark.parametrize("G", [2, 5, 10, 20, 40], ids=lambda g: "G%d" % g)
def test_decode_infinities_and_nan_of_masked_keys_stay_there(lib, G):
    """Tokens past a query and before its window never reach it, whatever they hold; the query
    that sees one has it in its result."""
    for dtype in (BF16, E4M3):
        p = P.problem(11, B=2, K=2, G=G, T=3, H=64, lens=[40, 35], page=16, dtype=dtype)
        q, kc, vc, table, lens, ks, vs = p
        bad = math.nan if dtype == E4M3 else math.inf
        last = 39                                   # request 0's last key: only t = 2 sees it
        vc[int(table[0, last // 16]), 0, last % 16, 3] = bad
        kc[int(table[0, last // 16]), 1, last % 16] = math.nan
        first = 35 - 3 - 20 + 1                     # request 1, window 20: only t = 0 sees it
        vc[int(table[1, first // 16]), 1, first % 16, 5] = bad
        o, lse = _decode(p, 20)
        _ok()
        o, lse = o.cpu().float(), lse.cpu()
        bo = ~torch.isfinite(o)
        assert bo[0, 0, :, 2, 3].all() and bo[0, 1, :, 2].all() and bo[1, 1, :, 0, 5].all()
        assert torch.isnan(lse[0, 1, :, 2]).all()
        assert bo.sum() == G + G * 64 + G
        clean = [x.clone() for x in (kc, vc)]
        for c in clean:
            c.copy_(torch.nan_to_num(c.float(), 0.0, 0.0, 0.0).to(dtype))
        want = P.decode(q, *clean, table, lens, ks, vs, 20)
        want[2][1].nan_to_num_(0.0)
        fine = ~bo
        P.check_decode(torch.where(fine, o, want[0].float()), torch.where(torch.isnan(lse), want[1].float(), lse),
                       want, 64, dtype == E4M3, 40)


@pytest.mark.parametrize("G", [4, 36])
def test_decode_infinities_of_kept_keys(lib, G):
    """An infinite value that a query keeps is in its result as such; scores of -inf have no weight,
    and one of +inf leaves no number."""
    p = P.problem(21, B=3, K=1, G=G, T=1, H=64, lens=[300, 1, 40], page=16)
    q, kc, vc, table, lens, *_ = p
    q.abs_().clamp_(min=1e-3)
    at = lambda b, s: (int(table[b, s // 16]), 0, s % 16)
    vc[at(0, 17)][2], vc[at(0, 290)][3], vc[at(1, 0)][4] = math.inf, -math.inf, math.inf
    vc[at(0, 5)][6], vc[at(0, 200)][6] = math.inf, -math.inf          # both: no number
    kc[at(2, 7)] = -math.inf
    o, lse = (x.cpu() for x in _decode(p))
    _ok()
    inf, none = torch.isinf(o[..., 0, :]), torch.isnan(o[..., 0, :])
    assert (o[0, 0, :, 0, 2] == math.inf).all() and (o[0, 0, :, 0, 3] == -math.inf).all()
    assert (o[1, 0, :, 0, 4] == math.inf).all() and none[0, 0, :, 6].all()
    assert inf.sum() == 3 * G and none.sum() == G
    # the key of -inf scores counts as absent
    n = 40
    keep = [s for s in range(n) if s != 7]
    k, v = (torch.stack([c[at(2, s)] for s in keep]).double() for c in (kc, vc))
    x = q[2, 0, :, 0].double() @ k.T
    w = torch.softmax(x, -1)
    assert ((o[2, 0, :, 0].double() - w @ v).abs()
            <= 2.0 ** -8 * (w @ v).abs() + 2.0 ** -13 * (w @ v.abs())).all()
    assert (lse[2, 0, :, 0].double() - torch.logsumexp(x, -1)).abs().max() <= 2.0 ** -14
    kc[at(2, 7)] = math.inf
    o, lse = (x.cpu() for x in _decode(p))
    _ok()
    assert torch.isnan(o[2]).all() and not torch.isnan(lse[0]).any()


def test_decode_bad_pages_and_lengths_are_reported(lib):
    p = P.problem(12, B=4, K=2, G=4, T=1, H=128, lens=[50, 60, 20, 33], page=16)
    q, kc, vc, table, lens, *_ = p
    clean = _decode(p)
    _ok()
    table[1, 2] = kc.shape[0]
    o, lse = _decode(p)
    assert binding.fa_check_status() == binding.FA_ERR_DEVICE_VALUE
    for b in (0, 2, 3):
        assert torch.equal(o[b], clean[0][b]) and torch.equal(lse[b], clean[1][b])
    zk, zv = kc.clone(), vc.clone()                 # keys of the bad page count as zeros
    zk = torch.cat([zk, torch.zeros_like(zk[:1])])
    zv = torch.cat([zv, torch.zeros_like(zv[:1])])
    want = P.decode(q, zk, zv, table, lens)
    P.check_decode(o.cpu(), lse.cpu(), want, 128, False, 60)
    for value, same in ((-5, 0), (10 ** 6, None)):
        p = P.problem(12, B=4, K=2, G=4, T=1, H=128, lens=[50, 60, 20, 33], page=16, extra_cols=0)
        p[4][2] = value
        if same is None:
            p[3][2, :] = p[3][0, :]                 # the whole row is pages: clamped to all of it
            for c in p[1:3]:
                c.nan_to_num_(0.5)
            p[3].clamp_(min=0)
        o, lse = _decode(p)
        assert binding.fa_check_status() == binding.FA_ERR_DEVICE_VALUE
        for b in (0, 1, 3):
            if same == 0:
                assert torch.equal(o[b], clean[0][b]) and torch.equal(lse[b], clean[1][b])
        if same == 0:
            assert (o[2] == 0).all() and torch.isneginf(lse[2]).all()
        else:
            p[4][2] = p[3].shape[1] * 16
            want = P.decode(p[0], p[1], p[2], p[3], p[4])
            P.check_decode(o.cpu(), lse.cpu(), want, 128, False, 64)


def test_decode_without_columns(lib):
    """Empty requests need no pages at all."""
    q = torch.ones((2, 1, 2, 1, 64), dtype=BF16, device="cuda")
    c = torch.zeros((0, 1, 16, 64), dtype=BF16, device="cuda")
    o, lse = binding.paged_attention_decode(q, c, c, torch.zeros((2, 0), dtype=torch.int32, device="cuda"),
                                            _i32([0, 0]))
    _ok()
    assert (o == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("G", [2, 40])
def test_decode_offsets_past_32_bits(lib, G):
    """A cache of over 4 GiB a tensor, and its last page."""
    K, H, page, n_pages = 4, 128, 64, 70000
    caches = [torch.zeros((n_pages, K, page, H), dtype=BF16, device="cuda") for _ in range(2)]
    assert caches[0].numel() * 2 > 1 << 32
    p = P.problem(13, B=2, K=K, G=G, T=1, H=H, lens=[150, 70], page=page)
    q, kc, vc, table, lens, *_ = p
    far = torch.arange(n_pages - kc.shape[0], n_pages)
    far[0] = 3
    for big, small in zip(caches, (kc, vc)):
        big[far.cuda()] = small.cuda()
    moved = torch.where(table >= 0, far[table.clamp(min=0).long()].int(), table)
    o, lse = binding.paged_attention_decode(q.cuda(), *caches, moved.cuda(), lens.cuda())
    _ok()
    P.check_decode(o.cpu(), lse.cpu(), P.decode(q, kc, vc, table, lens), H, False, 150)
    # and a token written there
    x = torch.randn((1, K, H), device="cuda").bfloat16()
    slot = torch.tensor([n_pages * page - 1], device="cuda")
    binding.fa_paged_append(x, x, slot, *caches)
    _ok()
    assert torch.equal(caches[1][-1, :, -1], x[0])


def test_decode_repeats_bitwise_whatever_the_workspace_holds(lib):
    p = P.problem(14, B=3, K=2, G=8, T=1, H=128, lens=[5000, 17, 900], page=16)
    n = binding.fa_paged_decode_workspace_size(3, 2, 8, 1, 128)
    first = None
    for fill in (0, 255, 1, 127):
        ws = torch.full((max(n, 256),), fill, dtype=torch.uint8, device="cuda")
        for _ in range(3):
            got = _decode(p, workspace=ws)
            first = first or got
            assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])
    _ok()


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("H", [64, 128, 256])
def test_decode_many_rows_repeats_bitwise(lib, H, dtype):
    """Whatever the workspace holds, on two streams at once, and captured and replayed."""
    p = P.problem(14, B=3, K=2, G=20, T=3, H=H, lens=[5000, 17, 900], page=16, dtype=dtype)
    n = binding.fa_paged_decode_workspace_size(3, 2, 20, 3, H)
    first = _check(p, 4000)
    for fill in (0, 255, 127):
        got = _decode(p, 4000, torch.full((n,), fill, dtype=torch.uint8, device="cuda"))
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])
    q, table, lens, ks, vs = (x if x is None else x.cuda() for x in (p[0], *p[3:]))
    caches = [P.to_device(x, "cuda") for x in p[1:3]]
    call = lambda: binding.paged_attention_decode(q, *caches, table, lens, k_scale=ks, v_scale=vs, window=4000)
    torch.cuda.synchronize()
    streams, results = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(10):
        for st in streams:
            with torch.cuda.stream(st):
                results.append(call())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        results.append(call())
    for _ in range(3):
        graph.replay()
    _ok()
    for o, lse in results:
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_decode_many_rows_bad_pages_count_as_zeros(lib, dtype):
    for H in (64, 128, 256):
        p = P.problem(12, B=4, K=2, G=36, T=1, H=H, lens=[50, 260, 20, 33], page=16, dtype=dtype)
        q, kc, vc, table, lens, ks, vs = p
        table[1, 2], table[1, 9] = kc.shape[0], kc.shape[0]
        o, lse = _decode(p)
        assert binding.fa_check_status() == binding.FA_ERR_DEVICE_VALUE
        zero = torch.zeros_like(kc[:1].contiguous())
        zk, zv = (torch.cat([c.contiguous().view(torch.uint8), zero.view(torch.uint8)]).view(dtype)
                  for c in (kc, vc))
        want = P.decode(q, zk, zv, table, lens, ks, vs)
        P.check_decode(o.cpu(), lse.cpu(), want, H, dtype == E4M3, 260)


def test_decode_many_rows_8bit_query_range(lib):
    """Query rows far from 1, as above, with the rows' scaling shared by two threads each."""
    for H in (64, 256):
        p = list(P.problem(10, B=2, K=1, G=40, T=1, H=H, lens=[300, 33], page=16, dtype=E4M3))
        size = torch.tensor([1e-30, 1e-8, 1.0, 3.0, 0.0, 1e-38, 1e-4, 20.0]).repeat(5)[:, None, None]
        p[0] = (p[0].float() * size).bfloat16()
        _check(tuple(p))
        for d in (0, H - 1):                        # the large part in either half of the dims
            large = [x if x is None else x.clone() for x in p]
            large[0][..., d] = 1e5
            large[1].view(torch.uint8)[..., d] = 0
            _check(tuple(large))


@pytest.mark.parametrize("H", [64, 128, 256])
def test_decode_wait_that_runs_out_ends_with_an_error(lib, H):
    """Many query rows: the kernel's warps wait for one another, each time with a limit (of no time
    here).  Whatever the workspace holds where one runs out, the call ends, and the next is right."""
    p = P.problem(4, B=24, K=2, G=40, T=1, H=H, lens=[3000, 700, 40, 1] * 6, page=16)
    want = _decode(p)
    n = binding.fa_paged_decode_workspace_size(24, 2, 40, 1, H)
    for fill in (0, 1, 127, 255):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        assert binding.fa_set_wait_limit_ns(1) == binding.FA_OK
        try:
            o, lse = _decode(p, workspace=ws)
            rc = binding.fa_check_status()
            assert rc in (binding.FA_OK, binding.FA_ERR_DEVICE_TIMEOUT)   # OK: none has run out
            assert rc or (torch.equal(o, want[0]) and torch.equal(lse, want[1]))
        finally:
            assert binding.fa_set_wait_limit_ns(2_000_000_000) == binding.FA_OK
    _check(p)
    _ok()


def test_decode_on_two_streams(lib):
    ps = [P.problem(15 + i, B=4, K=2, G=8, T=1, H=128, lens=[900, 3000, 17, 64], page=16)
          for i in range(2)]
    want = [_decode(p) for p in ps]
    dev = [[P.to_device(x, "cuda") if x is not None and x.dim() == 4 else x.cuda() for x in p[:5]]
           for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(binding.paged_attention_decode(*dev[i]))
    torch.cuda.synchronize()
    for w, gs in zip(want, got):
        for g in gs:
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
    _ok()


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "address"])
def test_helpers_allocate_on_the_stream_of_the_call(lib, raw, monkeypatch):
    """What a call on a side stream allocates and lets go of is not given to the current one."""
    p = P.problem(15, B=4, K=2, G=8, T=1, H=128, lens=[900, 3000, 17, 64], page=16)
    want = _decode(p)
    q, table, lens = (p[i].cuda() for i in (0, 3, 4))
    caches = [P.to_device(x, "cuda") for x in p[1:3]]
    torch.cuda.synchronize()
    side, seen = torch.cuda.Stream(), []
    plain = binding.fa_paged_decode
    monkeypatch.setattr(binding, "fa_paged_decode",
                        lambda *a: (seen.append((a[7].data_ptr(), a[7].nbytes)), plain(*a))[1])
    got = binding.paged_attention_decode(q, *caches, table, lens,
                                         stream=side.cuda_stream if raw else side)
    (at, size), = seen
    others = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(8)]
    assert at not in [x.data_ptr() for x in others]
    steps = binding.paged_tables(_i32([3, 0]), _i32([1, 2]), _i32([0, 1]), _i32([0]),
                                 _i32([[2], [0]]), n_pages=3, page_size=4, max_tokens=4,
                                 stream=side.cuda_stream if raw else side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert steps[2].tolist() == [11, 0, 1, -1]
    _ok()


def test_empty_row_of_queries(lib):
    for shape in ((0, 2, 4, 1, 64), (2, 0, 4, 1, 64), (2, 2, 4, 0, 64)):
        q = torch.zeros(shape, dtype=BF16, device="cuda")
        c = torch.zeros((2, shape[1], 16, 64), dtype=BF16, device="cuda")
        o, lse = binding.paged_attention_decode(q, c, c, _i32(np.zeros((shape[0], 1), int)),
                                                _i32(np.zeros(shape[0], int)))
        assert o.shape == shape and lse.shape == shape[:4]
    _ok()


# ------------------------------------------------------- the three together

class _Server:
    """Requests on one paged cache, and beside it every key and value in order on the CPU."""

    def __init__(self, B, K, G, H, page, n_pages, cols, dtype, layout, seed):
        self.B, self.K, self.G, self.H, self.page, self.n_pages = B, K, G, H, page, n_pages
        self.gen = torch.Generator().manual_seed(seed)
        self.dtype = dtype
        shape = (n_pages, K, page, H) if layout == "head" else (n_pages, page, K, H)
        self.caches = []
        for _ in range(2):
            c = torch.zeros(shape, dtype=dtype, device="cuda")
            self.caches.append(c if layout == "head" else c.transpose(1, 2))
        self.scale = None if dtype == BF16 else [torch.full((K,), 0.02, device="cuda") for _ in range(2)]
        self.lens = _i32([0] * B)
        self.used = _i32([0])
        self.free = torch.randperm(n_pages, generator=self.gen).int().cuda()
        self.table = torch.full((B, cols), -1, dtype=torch.int32, device="cuda")
        self.history = [[torch.zeros(0, K, H) for _ in range(2)] for _ in range(B)]

    def inputs(self, new, T, pad):
        n = sum(new)
        kv = torch.randn((2, n + pad, self.K, self.H), generator=self.gen).bfloat16()
        q = (torch.randn((self.B, self.K, self.G, T, self.H), generator=self.gen)
             * self.H ** -0.5).bfloat16()
        at = 0
        for b, m in enumerate(new):
            for i in range(2):
                x = kv[i, at:at + m]
                if self.scale is not None:
                    x = _stored(x, self.scale[i].cpu()).float() * self.scale[i].cpu()[:, None]
                self.history[b][i] = torch.cat([self.history[b][i], x.float()])
            at += m
        return kv, q

    def step(self, kv, q, new, o, lse, ws, out):
        binding.fa_paged_tables(self.lens, new, self.free, self.used, self.table, self.lens,
                                out["starts"], out["slots"], out["pos"], self.used, self.n_pages,
                                self.page)
        binding.fa_paged_append(kv[0], kv[1], out["slots"], *self.caches, *(self.scale or ()))
        binding.fa_paged_decode(q, *self.caches, self.table, self.lens, o, lse, ws,
                                *(self.scale or ()))

    def check(self, q, o, lse):
        """Each request against the dense oracle on its history (the T newest tokens' rows)."""
        T = q.shape[3]
        for b, (k, v) in enumerate(self.history):
            n = k.shape[0]
            kk, vv = (x.transpose(0, 1)[None].numpy().astype(np.float64) for x in (k, v))
            if n == 0:
                assert (o[b] == 0).all() and torch.isneginf(lse[b]).all()
                continue
            ro, rl = oracle.attention_forward(q[b:b + 1].float().numpy().astype(np.float64), kk, vv,
                                              causal=True)
            # the tolerances of the dense kernels' parity tests
            assert np.abs(o[b].float().cpu().numpy() - ro[0]).max() <= 2e-2
            rl = rl[0]
            got = lse[b].cpu().numpy()
            assert np.array_equal(np.isinf(rl), np.isinf(got))
            assert np.abs(got - rl)[np.isfinite(rl)].max(initial=0) <= 1e-3


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("layout", ["head", "token"])
def test_serving_steps(lib, layout, dtype):
    """Prompts, then decode steps, a step without tokens for some, and drafted tokens."""
    s = _Server(5, 2, 4, 128, 16, 120, 24, dtype, layout, 0)
    for new, T in (([37, 0, 5, 150, 16], 1), ([1, 1, 1, 1, 1], 1), ([1, 1, 0, 1, 1], 1),
                   ([3, 3, 3, 3, 3], 3), ([1, 20, 1, 1, 1], 1)):
        pad = 7
        kv, q = s.inputs(new, T, pad)
        N = sum(new) + pad
        out = dict(starts=_i32([0] * 6), slots=torch.empty(N, dtype=torch.int64, device="cuda"),
                   pos=_i32([0] * N))
        o = torch.empty(q.shape, dtype=BF16, device="cuda")
        lse = torch.empty(q.shape[:4], device="cuda")
        n = binding.fa_paged_decode_workspace_size(*q.shape)
        ws = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
        s.step(kv.cuda(), q.cuda(), _i32(new), o, lse, ws, out)
        _ok()
        assert s.lens.tolist() == [h[0].shape[0] for h in s.history]
        s.check(q, o, lse)


def test_serving_step_captured_and_replayed(lib):
    """One decode step captured once, replayed while the lengths and pages grow; a second graph
    shares its workspace."""
    s = _Server(6, 2, 8, 128, 16, 400, 40, BF16, "token", 1)
    kv, q = s.inputs([300, 15, 16, 1, 0, 31], 1, 0)
    N = 363
    o = torch.empty(q.shape, dtype=BF16, device="cuda")
    lse = torch.empty(q.shape[:4], device="cuda")
    ws = torch.full((max(256, binding.fa_paged_decode_workspace_size(*q.shape)),), 255,
                    dtype=torch.uint8, device="cuda")
    big = dict(starts=_i32([0] * 7), slots=torch.empty(N, dtype=torch.int64, device="cuda"), pos=None)
    s.step(kv.cuda(), q.cuda(), _i32([300, 15, 16, 1, 0, 31]), o, lse, ws, big)
    _ok()
    out = dict(starts=_i32([0] * 7), slots=torch.empty(6, dtype=torch.int64, device="cuda"), pos=None)
    kv_in = torch.zeros((2, 6, 2, 128), dtype=BF16, device="cuda")
    q_in, new = torch.zeros_like(q, device="cuda"), _i32([1] * 6)
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    graphs = []
    for oo, ll in ((o, lse), (o2, lse2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.step(kv_in, q_in, new, oo, ll, ws, out)
        graphs.append((g, oo, ll))
    assert s.lens.tolist() == [300, 15, 16, 1, 0, 31]       # capturing runs nothing
    for i in range(20):
        kv, q = s.inputs([1] * 6, 1, 0)
        kv_in.copy_(kv)
        q_in.copy_(q)
        g, oo, ll = graphs[i % 2]
        g.replay()
        _ok()
        s.check(q, oo, ll)
    assert s.lens.tolist() == [320, 35, 36, 21, 20, 51]


def test_paged_decode_matches_the_dense_split_forward(lib):
    """The same keys in pages and in a dense cache: two kernels, one definition."""
    p = P.problem(20, B=2, K=2, G=8, T=1, H=128, lens=[1024, 1024], page=64)
    q, kc, vc, table, lens, *_ = p
    o, lse = _decode(p)
    k, v = (torch.stack([torch.cat([c[int(table[b, j])] for j in range(16)], 1) for b in range(2)])
            for c in (kc, vc))
    od, ld = binding.attention_forward_splitkv(q.cuda(), k.cuda(), v.cuda(), causal=True)
    _ok()
    assert (o.float() - od.float()).abs().max() <= 2e-2
    assert (lse - ld).abs().max() <= 1e-3


def test_paged_tables_helper(lib):
    case = _tables_case(3, 40, 16, 200, 30)
    want = P.tables(*case[:7])
    table = _i32(case[4])
    total, starts, slots, positions, used = binding.paged_tables(
        _i32(case[0]), _i32(case[1]), _i32(case[2]), _i32([case[3]]), table, n_pages=case[7],
        page_size=case[5], max_tokens=case[6])
    _ok()
    got = (table, total, starts, slots, positions, used)
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy().ravel(), np.asarray(w).ravel())


def test_serving_step_through_the_helpers(lib):
    """The helpers that allocate, as in the README: two steps from an empty cache."""
    B, K, G, H, page, n_pages = 3, 2, 4, 64, 16, 32
    gen = torch.Generator().manual_seed(3)
    caches = [torch.empty((n_pages, K, page, H), dtype=BF16, device="cuda") for _ in range(2)]
    lens, used, free = _i32([0] * B), _i32([0]), _i32(np.arange(n_pages)[::-1].copy())
    table = torch.zeros((B, 8), dtype=torch.int32, device="cuda")
    past = [torch.zeros((B, 0, K, H)) for _ in range(2)]
    for n in (21, 1):
        kv = torch.randn((2, B, n, K, H), generator=gen).bfloat16()
        q = (torch.randn((B, K, G, 1, H), generator=gen) / 8).bfloat16()
        past = [torch.cat([p, x.float()], 1) for p, x in zip(past, kv)]
        lens, starts, slots, positions, used = binding.paged_tables(
            lens, _i32([n] * B), free, used, table, n_pages=n_pages, page_size=page, max_tokens=B * n)
        k, v = (x.reshape(B * n, K, H).cuda() for x in kv)
        binding.fa_paged_append(k, v, slots, *caches)
        o, lse = binding.paged_attention_decode(q.cuda(), *caches, table, lens)
        _ok()
        ro, rl = oracle.attention_forward(q.double().numpy(), *(x.transpose(1, 2).double().numpy() for x in past))
        assert np.abs(o.float().cpu().numpy() - ro).max() <= 2e-2
        assert np.abs(lse.cpu().numpy() - rl).max() <= 1e-3
    assert lens.tolist() == [22] * B and used.tolist() == [6]


@pytest.mark.parametrize("wrong", range(11))
def test_binding_refuses_wrong_tables_tensors(lib, wrong):
    """Each tensor in turn of another type, another size, not contiguous, or on the CPU."""
    def good():
        return [_i32([1, 2]), _i32([1, 1]), _i32(range(8)), _i32([0]), _i32(np.zeros((2, 4), int)),
                _i32([0, 0]), _i32([0, 0, 0]), torch.zeros(4, dtype=torch.int64, device="cuda"),
                _i32([0] * 4), _i32([0])]
    if wrong == 10:
        binding.fa_paged_tables(*good(), 8, 16)
        return _ok()
    for spoil in (lambda t: t.float(), lambda t: torch.cat([t, t]) if wrong in (0, 1, 3, 4, 5, 6, 8, 9) else t.float(),
                  lambda t: torch.stack([t, t], -1)[..., 0] if t.numel() > 1 else t.float(), lambda t: t.cpu()):
        args = good()
        args[wrong] = spoil(args[wrong])
        with pytest.raises(ValueError):
            binding.fa_paged_tables(*args, 8, 16)
    _ok()


@pytest.mark.parametrize("what", ["lens", "table", "o", "dtype", "scale", "strides", "lse", "sizes",
                                  "apart", "cpu"])
def test_binding_refuses_wrong_gpu_tensors(lib, what):
    q = torch.zeros((2, 2, 4, 1, 64), dtype=BF16, device="cuda")
    kc = torch.zeros((3, 2, 16, 64), dtype=BF16, device="cuda")
    vc, table, lens, o, ks = kc.clone(), _i32([[0], [1]]), _i32([1, 1]), torch.empty_like(q), None
    lse = torch.empty((2, 2, 4, 1), device="cuda")
    if what == "lens":
        lens = lens.long()
    elif what == "table":
        table = _i32([[0]])
    elif what == "o":
        o = o[:1]
    elif what == "dtype":
        kc, vc = kc.half(), vc.half()
    elif what == "scale":
        ks = torch.ones(2, device="cuda")
    elif what == "lse":
        lse = lse.double()
    elif what == "sizes":
        lens = _i32([1, 1, 1])
    elif what == "apart":
        q = torch.stack([q, q], -1)[..., 0]
    elif what == "cpu":
        table = table.cpu()
    else:
        vc = vc.transpose(1, 2).contiguous().transpose(1, 2)
    with pytest.raises(ValueError):
        binding.fa_paged_decode(q, kc, vc, table, lens, o, lse, None, ks, ks)
    _ok()
