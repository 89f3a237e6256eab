"""The paged cache operators where they can go wrong: waits that run out, values at the ends of
their types, sizes at the limits of a launch, errors of other calls."""
import ctypes
import os
import struct
import subprocess
import sys
import threading

import pytest
import torch

from flash_attention_gqa_gb300 import binding
import _paged as P
from test_paged import BF16, E4M3, _append_case, _check, _decode, _ok, _stored

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


def _sinks(rows, H, n, B, spread=0.3):
    """An 8-bit cache whose requests have one key far above the others, with values of zero: kv
    heads 0 to 3 at the first position, 4 to 7 in the middle, 12 to 17 nats above."""
    G, T = rows
    p = P.problem(H, B=B, K=8, G=G, T=T, H=H, lens=[n] * B, page=16, dtype=E4M3)
    q, kc, vc, table, lens, ks, vs = p
    gap = torch.tensor([12.0, 14.0, 16.0, 17.0] * 2)
    q.mul_(spread)
    q[..., 0] = gap[:, None, None].bfloat16()
    kc.view(torch.uint8)[..., 0] = 0
    for b in range(B):
        for h in range(8):
            s = 0 if h < 4 else n // 2
            at = (int(table[b, s // 16]), h, s % 16)
            kc.view(torch.uint8)[at] = 0
            kc[at][0] = torch.tensor(32.0).to(E4M3)
            vc.view(torch.uint8)[at] = 0
    ks.fill_(1 / 32)
    return p


@pytest.mark.parametrize("H", [64, 128, 256])
@pytest.mark.parametrize("rows", [(8, 1), (4, 3), (24, 1), (40, 1), (16, 5)], ids=lambda r: "G%d_T%d" % r)
def test_decode_8bit_keys_far_below_the_largest(lib, rows, H):
    """Every other key weighs 2^-17 to 2^-25 of the largest, and is all of the result: the weights'
    f16 terms have to hold them as well as they hold large ones.  Requests done whole, by one CTA
    each, and split."""
    for B, n in ((40, 450), (24, 1500), (2, 6000)):
        _check(_sinks(rows, H, n, B))


@pytest.mark.parametrize("G", [8, 24, 64])
def test_decode_8bit_large_scores(lib, G):
    """Scores in the hundreds that grow along the keys: the base of the exponents moves."""
    for H in (64, 128, 256):
        p = P.problem(9, B=3, K=1, G=G, T=1, H=H, lens=[900, 64, 1], page=16, dtype=E4M3)
        q, kc, vc, table, lens, ks, vs = p
        grow = torch.ones(kc.shape[0])
        for j, page in enumerate(table[0][table[0] >= 0].tolist()):
            grow[page] = 0.05 + 0.05 * j
        kc.copy_((kc.float() * grow[:, None, None, None]).to(E4M3))
        _check(((q.float() * 40).bfloat16(), kc, vc, table, lens, ks, vs))


_TABLES_SIZES = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import numpy as np
import _paged as P
import test_paged as T
for B in {sizes}:
    for in_place in (False, True):
        case = T._tables_case(B, B, 16, 40, 2)
        for g, w in zip(T._run_tables(case, in_place), P.tables(*case[:7])):
            assert np.array_equal(g.ravel(), np.asarray(w).ravel()), B
T._ok()
"""


@pytest.mark.parametrize("sizes", [(4053, 4054, 4095), (4080,), (4096, 4095)], ids=str)
def test_tables_around_48_kb_of_shared_memory(lib, sizes):
    """In a process of their own: a call with more requests raises the launch's limit for later ones."""
    tests = os.path.dirname(os.path.abspath(__file__))
    code = _TABLES_SIZES.format(root=os.path.dirname(tests), tests=tests, sizes=sizes)
    run = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]


def _tables_state(B):
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    lens = i32([3] * B)
    return (lens, i32([1] * B), i32(range(B)), i32([0]), i32([[b] for b in range(B)]), torch.empty_like(lens),
            i32([0] * (B + 1)), torch.empty(B, dtype=torch.int64, device="cuda"), None, i32([0]), B, 16)


def _tables_done(args):
    B = args[0].numel()
    want = torch.arange(B, device="cuda")
    return torch.equal(args[7], want * 16 + 3) and (args[5] == 4).all() and torch.equal(args[6][:-1].long(), want)


def test_tables_of_different_sizes_in_two_threads(lib):
    """One thread's launch with fewer requests leaves the other's its shared memory (calls without
    the checks of the binding between them, so that the two meet)."""
    states = [_tables_state(8192), _tables_state(4096)]
    torch.cuda.synchronize()
    start, failed = threading.Barrier(2), []

    def work(args):
        stream = torch.cuda.Stream()
        c, n, f, u, t, total, starts, slots, _, out, n_pages, page = args
        B = n_pages
        record = struct.pack("17q", *(x.data_ptr() for x in (c, n, f)), B, u.data_ptr(), t.data_ptr(), 1,
                             *(x.data_ptr() for x in (total, starts, slots)), 0, B, out.data_ptr(), B, n_pages,
                             page, stream.cuda_stream)
        torch.cuda.set_device(0)
        start.wait()
        failed.append(sum(lib.fa_paged_tables_packed(record) for _ in range(40000)))

    threads = [threading.Thread(target=work, args=(s,)) for s in states]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert failed == [0, 0]
    _ok()
    assert all(_tables_done(s) for s in states)


def _three_calls(stream=None):
    """The three operators as calls that return their status, and a check of what they did."""
    tables = _tables_state(8)
    gen = torch.Generator().manual_seed(0)
    kv = torch.randn((2, 8, 2, 64), generator=gen).bfloat16().cuda()
    caches = [torch.zeros((8, 2, 16, 64), dtype=BF16, device="cuda") for _ in range(2)]
    slots = torch.arange(8, device="cuda") * 16
    p = P.problem(3, B=3, K=2, G=4, T=1, H=64, lens=[700, 3, 40], page=16)
    want = _check(p)
    q, table, lens = (p[i].cuda() for i in (0, 3, 4))
    pages = [P.to_device(c, "cuda") for c in p[1:3]]
    o, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    ws = torch.empty(binding.fa_paged_decode_workspace_size(3, 2, 4, 1, 64), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()

    def done():
        _ok()
        assert _tables_done(tables)
        assert all(torch.equal(c[:, :, 0], x) for c, x in zip(caches, kv))
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])

    return [lambda: binding.fa_paged_tables(*tables, stream=stream, check=False),
            lambda: binding.fa_paged_append(*kv, slots, *caches, stream=stream, check=False),
            lambda: binding.fa_paged_decode(q, *pages, table, lens, o, lse, ws, stream=stream, check=False)], done


def test_errors_of_earlier_calls_are_not_theirs(lib):
    """An error that another user of the runtime has left behind (here: a device that is none)."""
    calls, done = _three_calls()
    try:
        for call in calls:
            assert lib.cudaSetDevice(9999) != 0 and lib.cudaPeekAtLastError() != 0
            assert call() == binding.FA_OK
    finally:
        lib.cudaGetLastError()
    done()


def test_a_failed_call_leaves_no_error_behind(lib):
    """Launches into a capture that something has spoiled (a synchronisation) are refused by the
    runtime; the calls after it know nothing of that."""
    stream = torch.cuda.Stream()
    calls, done = _three_calls(stream)
    at, graph = ctypes.c_void_p(stream.cuda_stream), ctypes.c_void_p()
    for call in calls:
        assert lib.cudaStreamBeginCapture(at, 2) == 0
        assert lib.cudaStreamSynchronize(at) != 0
        lib.cudaGetLastError()
        rc, left = call(), lib.cudaPeekAtLastError()
        assert lib.cudaStreamEndCapture(at, ctypes.byref(graph)) != 0
        lib.cudaGetLastError()
        assert rc == binding.FA_ERR_CUDA and left == 0
    for call in calls:
        assert call() == binding.FA_OK
    done()


@pytest.mark.parametrize("G", [8, 12, 24, 40])
def test_decode_8bit_scores_at_the_ends_of_fp32(lib, G):
    """Queries and scales whose product, with what undoes the queries' scaling, leaves fp32: scores
    of nothing (masked keys stay masked, the kept ones weigh the same), and keys of zeros."""
    for H in (64, 128, 256):
        p = list(P.problem(17, B=3, K=3, G=G, T=1, H=H, lens=[300, 21, 40], page=16, dtype=E4M3))
        p[0][:, :2] = (p[0][:, :2].float() * 1e-30).bfloat16()
        p[5] = torch.tensor([1e-20, 1e-38, 1e3])
        p[0][:, 2] = 1e38
        p[1].view(torch.uint8)[:, 2] = 0
        _check(tuple(p))


@pytest.mark.parametrize("single", ["heads", "page size", "pages"])
def test_strides_of_single_dims_may_differ(lib, single):
    """A dimension of one has no stride that matters: a cache written as [pages, page size, K, H] is
    one written as [pages, K, page size, H] where K or the page size is one."""
    n_pages, K, page = dict(zip(("heads", "page size", "pages"), ((9, 1, 16), (60, 2, 1), (1, 2, 64))))[single]
    gen = torch.Generator().manual_seed(2)
    k, v = (torch.randn((n_pages, K, page, 64), generator=gen).bfloat16().cuda() for _ in range(2))
    if single == "pages":
        odd = v.as_strided(v.shape, (7, *v.stride()[1:]))
    else:
        odd = v.view(n_pages, page, K, 64).transpose(1, 2)
        assert torch.equal(odd, v)
    assert odd.stride() != k.stride()
    table = torch.arange(n_pages, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([min(60, n_pages * page)], dtype=torch.int32, device="cuda")
    q = torch.randn((1, K, 4, 1, 64), generator=gen).bfloat16().cuda() / 8
    want = binding.paged_attention_decode(q, k, v, table, lens)
    for caches in ((k, odd), (odd, v)):
        if caches[0] is odd:
            want = binding.paged_attention_decode(q, v, v, table, lens)
        o, lse = binding.paged_attention_decode(q, *caches, table, lens)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    new = torch.randn((1, K, 64), generator=gen).bfloat16().cuda()
    binding.fa_paged_append(new, new, torch.tensor([5], device="cuda"), k, odd)
    assert torch.equal(k[5 // page, :, 5 % page], new[0]) and torch.equal(v[5 // page, :, 5 % page], new[0])
    _ok()


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("shape", [(60001, 3, 64, 16, "token"), (8003, 5, 256, 32, "head"),
                                   (9999, 8, 128, 64, "head")], ids=lambda s: "N%d_K%d_H%d" % s[:3])
def test_append_of_many_tokens(lib, shape, dtype):
    """Four pairs of loads a thread: heads that do not divide a CTA's units, a last CTA with few
    tokens, padding and slots past the cache among the loads."""
    N, K, H, page, layout = shape
    k, v, slots, caches, scales = _append_case(N, N, K, H, page, dtype, layout, pad=32)
    past = torch.rand(N, generator=torch.Generator().manual_seed(N)) < 0.01
    n_slots = caches[0].shape[0] * page
    slots[past] = n_slots + slots[past].clamp(min=0)
    dev = [P.to_device(c, "cuda") for c in caches]
    binding.fa_paged_append(*(P.to_device(x, "cuda") for x in (k, v)), slots.cuda(), *dev,
                            *(x if x is None else x.cuda() for x in scales))
    assert binding.fa_check_status() == binding.FA_ERR_DEVICE_VALUE
    live = (slots >= 0) & (slots < n_slots)
    at = slots[live]
    bits = torch.int16 if dtype is BF16 else torch.uint8
    for x, want, got, scale in zip((k, v), caches, dev, scales):
        put = x if scale is None else _stored(x, scale)
        want.view(bits)[at // page, :, at % page] = put.contiguous().view(bits)[live]
        assert torch.equal(got.cpu().contiguous().view(bits), want.contiguous().view(bits))
    _ok()


@pytest.mark.parametrize("G", [8, 20, 40])
def test_decode_8bit_without_scales(lib, G):
    for H in (64, 128, 256):
        p = list(P.problem(23, B=3, K=2, G=G, T=1, H=H, lens=[700, 1, 90], page=16, dtype=E4M3))
        for c in p[1:3]:
            c.copy_((c.float() / 32).to(E4M3))
        for scales in ([None, None], [p[5] * 16, None], [None, p[6]]):
            p[5:] = scales
            _check(tuple(p))


@pytest.mark.parametrize("G", [1, 40])
@pytest.mark.parametrize("B,K", [(8191, 8), (257, 255)])
def test_decode_of_many_heads(lib, B, K, G):
    """Close to the limit of B * K; every 97th request is compared."""
    rng = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 41, (B,), generator=rng)
    lens[::97] = torch.arange(len(lens[::97])) % 60
    lens[5] = 3000
    p = P.problem(B, B=B, K=K, G=G, T=1, H=64, lens=lens.tolist(), page=16)
    o, lse = (x.cpu() for x in _decode(p))
    _ok()
    some = torch.cat([torch.arange(0, B, 97), torch.tensor([5, B - 1])])[:40 if K > 8 else None]
    q, kc, vc, table, n, *_ = p
    want = P.decode(q[some], kc, vc, table[some], n[some])
    P.check_decode(o[some], lse[some], want, 64, False, 3000)
