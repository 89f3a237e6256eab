"""Rotary positions, page management and the decode of shared prefixes without a GPU: argument checks of
the C ABI (fake pointers: every call is refused, or has nothing to do, before any launch) and of the
binding."""
import math
import struct

import pytest
import torch

from flash_attention_gqa_gb300 import binding
from test_boundary import clib  # noqa: F401  (fixture)

BAD, UNSUP, OK = binding.FA_ERR_INVALID_ARG, binding.FA_ERR_UNSUPPORTED, binding.FA_OK


def _both(lib, name, *args):
    """The status of a call with plain arguments, which its packed form has to give too."""
    rc = getattr(lib, name)(*args)
    bits = lambda x: 0 if x is None else struct.unpack("i", struct.pack("f", x))[0] if isinstance(x, float) else x  # noqa: E731
    assert getattr(lib, name + "_packed")(struct.pack(f"{len(args)}q", *map(bits, args))) == rc
    return rc


def _rotary(lib, q=16, qs=(65536, 4096, 128), qo=32, qos=(65536, 128, 2048), k=16, ks=(65536, 4096, 128), ko=32,
            kos=(65536, 128, 2048), pos=16, ps=(64, 16, 1), freq=16, axes=16, pairs=64, n_axes=2, adjacent=0,
            inverse=0, scale=0.5, B=4, T=16, qh=8, kh=2, H=128):
    return _both(lib, "fa_rotary", q, *qs, qo, *qos, k, *ks, ko, *kos, pos, *ps, freq, axes, pairs, n_axes, adjacent,
                 inverse, scale, B, T, qh, kh, H, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(q=None), BAD), (dict(q=24), BAD), (dict(qo=None), BAD), (dict(k=None), BAD), (dict(ko=8), BAD),
    (dict(pos=None), BAD), (dict(pos=18), BAD), (dict(freq=None), BAD), (dict(axes=2), BAD),
    (dict(qs=(65536, 4100, 128)), BAD), (dict(qos=(-8, 128, 2048)), BAD), (dict(ks=(65536, 4096, 1 << 41)), BAD),
    (dict(ps=(64, -1, 1)), BAD), (dict(q=32), BAD), (dict(k=32), BAD), (dict(adjacent=2), BAD),
    (dict(inverse=-1), BAD), (dict(scale=math.inf), BAD), (dict(scale=math.nan), BAD), (dict(B=-1), BAD),
    (dict(T=-1), BAD), (dict(qh=-1), BAD), (dict(kh=-1), BAD), (dict(H=-128), BAD), (dict(n_axes=0), BAD),
    (dict(pairs=-8), BAD), (dict(H=96), UNSUP), (dict(pairs=0), UNSUP), (dict(pairs=12), UNSUP),
    (dict(pairs=72), UNSUP), (dict(n_axes=17), UNSUP), (dict(B=1 << 16, T=1 << 15), UNSUP),
    (dict(qh=65000, kh=300), UNSUP), (dict(B=0, q=None), OK), (dict(T=0, pos=None), OK),
    (dict(qh=0, kh=0, freq=None), OK)])
def test_rotary_refusals(clib, kw, rc):  # noqa: F811
    assert _rotary(clib, **kw) == rc


def _append(lib, q=16, qt=4096, qhs=128, qo=32, qos=(4096, 4096, 128), k=16, kt=4096, khs=128, v=16, vt=4096,
            vhs=128, pos=16, ps=(64, 1), freq=16, axes=None, pairs=64, n_axes=1, adjacent=0, scale=0.5, slots=16,
            kc=16, vc=16, kind=0, ksc=None, vsc=None, sp=16384, sh=2048, st=128, B=4, T=1, qh=8, kh=8, H=128,
            n_pages=10, page=16):
    return _both(lib, "fa_paged_rotary_append", q, qt, qhs, qo, *qos, k, kt, khs, v, vt, vhs, pos, *ps, freq, axes,
                 pairs, n_axes, adjacent, scale, slots, kc, vc, kind, ksc, vsc, sp, sh, st, B, T, qh, kh, H, n_pages,
                 page, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(q=None), BAD), (dict(qo=8), BAD), (dict(k=None), BAD), (dict(v=24), BAD), (dict(pos=None), BAD),
    (dict(freq=2), BAD), (dict(slots=None), BAD), (dict(slots=4), BAD), (dict(kc=None), BAD), (dict(vc=8), BAD),
    (dict(kind=2), BAD), (dict(kind=0, ksc=16), BAD), (dict(kind=1, vsc=2), BAD), (dict(qt=4097), BAD),
    (dict(kt=-8), BAD), (dict(vhs=12), BAD), (dict(qos=(4096, 4096, 4)), BAD), (dict(ps=(64, -1)), BAD),
    (dict(T=1 << 29, B=1, kt=1 << 33), BAD), (dict(T=1 << 29, B=1, ps=(0, 1 << 33)), BAD), (dict(st=132), BAD),
    (dict(sp=-8), BAD), (dict(q=32, qhs=256), BAD), (dict(scale=math.nan), BAD), (dict(page=24), UNSUP),
    (dict(H=512), UNSUP), (dict(pairs=65), UNSUP), (dict(B=0), OK), (dict(qh=0, kh=0), OK)])
def test_rotary_append_refusals(clib, kw, rc):  # noqa: F811
    assert _append(clib, **kw) == rc


def _pool_args(lens=16, table=16, max_pages=8, shares=16, free=16, n_free=10, used=16):
    return lens, table, max_pages, shares, free, n_free, used


def _free(lib, rows=16, keep=16, N=3, lens_out=16, used_out=16, B=4, n_pages=100, page=16, **pool):
    lens, table, max_pages, shares, free, n_free, used = _pool_args(**pool)
    return _both(lib, "fa_paged_free", rows, keep, N, lens, table, max_pages, shares, free, n_free, used, lens_out,
                 used_out, B, n_pages, page, None)


def _fork(lib, parents=16, children=16, fork_lens=16, N=3, lens_out=16, copies=16, used_out=16, B=4, n_pages=100,
          page=16, **pool):
    lens, table, max_pages, shares, free, n_free, used = _pool_args(**pool)
    return _both(lib, "fa_paged_fork", parents, children, fork_lens, N, lens, table, max_pages, shares, free, n_free,
                 used, lens_out, copies, used_out, B, n_pages, page, None)


def _compact(lib, table_out=16, shares_out=16, free_out=16, moves=16, max_moves=7, B=4, n_pages=100, page=16, **pool):
    lens, table, max_pages, shares, free, n_free, used = _pool_args(**pool)
    return _both(lib, "fa_paged_compact", lens, table, max_pages, shares, free, n_free, used, table_out, shares_out,
                 free_out, moves, max_moves, B, n_pages, page, None)


POOL = [(dict(lens=None), BAD), (dict(table=None), BAD), (dict(shares=None), BAD), (dict(shares=2), BAD),
        (dict(free=None), BAD), (dict(used=None), BAD), (dict(used=2), BAD), (dict(B=-1), BAD),
        (dict(max_pages=-1), BAD), (dict(n_free=-1), BAD), (dict(n_pages=-1), BAD), (dict(page=0), BAD),
        (dict(page=24), UNSUP), (dict(page=1 << 17), UNSUP), (dict(B=8193), UNSUP),
        (dict(n_pages=(1 << 21) + 1), UNSUP), (dict(max_pages=1 << 27), UNSUP)]


@pytest.mark.parametrize("kw,rc", POOL + [
    (dict(rows=None), BAD), (dict(rows=2), BAD), (dict(keep=2), BAD), (dict(N=-1), BAD), (dict(N=8193), UNSUP),
    (dict(lens_out=None), BAD), (dict(used_out=None), BAD)])
def test_free_refusals(clib, kw, rc):  # noqa: F811
    assert _free(clib, **kw) == rc


@pytest.mark.parametrize("kw,rc", POOL + [
    (dict(parents=None), BAD), (dict(children=2), BAD), (dict(fork_lens=2), BAD), (dict(copies=None), BAD),
    (dict(N=-1), BAD), (dict(N=8193), UNSUP), (dict(lens_out=None), BAD), (dict(used_out=2), BAD)])
def test_fork_refusals(clib, kw, rc):  # noqa: F811
    assert _fork(clib, **kw) == rc


@pytest.mark.parametrize("kw,rc", POOL + [
    (dict(table_out=None), BAD), (dict(shares_out=2), BAD), (dict(free_out=None), BAD), (dict(moves=None), BAD),
    (dict(max_moves=-1), BAD)])
def test_compact_refusals(clib, kw, rc):  # noqa: F811
    assert _compact(clib, **kw) == rc


def _copy(lib, moves=16, N=4, kc=16, vc=16, kind=0, sl=1 << 20, sp=16384, sh=2048, st=128, layers=2, K=8, H=128,
          n_pages=10, page=16):
    return _both(lib, "fa_paged_copy", moves, N, kc, vc, kind, sl, sp, sh, st, layers, K, H, n_pages, page, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(moves=None), BAD), (dict(moves=2), BAD), (dict(kc=None), BAD), (dict(vc=8), BAD), (dict(kind=2), BAD),
    (dict(N=-1), BAD), (dict(layers=-1), BAD), (dict(K=-1), BAD), (dict(sl=4), BAD), (dict(sl=-16), BAD),
    (dict(sh=4), BAD), (dict(page=0), BAD), (dict(page=24), UNSUP), (dict(H=96), UNSUP), (dict(K=65536), UNSUP),
    (dict(layers=16385), UNSUP), (dict(K=65535, page=65536), UNSUP), (dict(K=4096, page=4096, N=1 << 20), UNSUP),
    (dict(N=0, moves=None), OK), (dict(layers=0), OK), (dict(K=0), OK)])
def test_copy_refusals(clib, kw, rc):  # noqa: F811
    assert _copy(clib, **kw) == rc


def _shared(lib, q=16, kc=16, vc=16, kind=0, ks=None, vs=None, sp=16384, sh=2048, st=128, table=16, lens=16,
            members=16, n_members=4, starts=16, prefix=16, n_groups=1, o=16, lse=16, ws=256, ws_bytes=1 << 40, B=4,
            K=8, G=4, T=1, H=128, n_pages=10, page=16, max_pages=8):
    return _both(lib, "fa_paged_decode_shared", q, kc, vc, kind, ks, vs, sp, sh, st, table, lens, members, n_members,
                 starts, prefix, n_groups, o, lse, ws, ws_bytes, B, K, G, T, H, n_pages, page, max_pages, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(q=None), BAD), (dict(q=8), BAD), (dict(o=None), BAD), (dict(lse=None), BAD), (dict(lens=2), BAD),
    (dict(table=None), BAD), (dict(kc=None), BAD), (dict(vc=8), BAD), (dict(kind=3), BAD), (dict(B=-1), BAD),
    (dict(n_members=-1), BAD), (dict(n_members=5), BAD), (dict(members=None), BAD), (dict(starts=None), BAD),
    (dict(prefix=None), BAD), (dict(prefix=2), BAD), (dict(n_groups=-1), BAD), (dict(n_groups=4097), UNSUP),
    (dict(ks=16), BAD), (dict(st=132), BAD), (dict(page=48), UNSUP), (dict(H=192), UNSUP), (dict(G=129), UNSUP),
    (dict(G=16, T=9), UNSUP), (dict(B=8193), UNSUP), (dict(B=8192, K=8), UNSUP), (dict(max_pages=1 << 27), UNSUP),
    (dict(ws=None), BAD), (dict(ws=128), BAD), (dict(ws_bytes=255), BAD), (dict(B=0, n_members=0), OK),
    (dict(T=0, q=None), OK)])
def test_shared_refusals(clib, kw, rc):  # noqa: F811
    assert _shared(clib, **kw) == rc


def test_shared_workspace_size(clib):  # noqa: F811
    size = binding.fa_paged_decode_shared_workspace_size
    assert size(0, 1, 1, 1, 128, 0, 0) == 0
    assert size(1, 1, 1, 1, 96, 1, 1) == 0
    assert size(4, 1, 1, 1, 128, 1, 5) == 0
    assert size(4, 1, 1, 1, 128, 4097, 4) == 0
    assert size(4, 1, 129, 1, 128, 1, 4) == 0
    assert 0 < size(4, 8, 4, 1, 128, 1, 4) < size(64, 8, 4, 1, 128, 1, 64)


@pytest.mark.parametrize("name,n", [("paged_free", 16), ("paged_fork", 18), ("paged_compact", 16), ("paged_copy", 15),
                                    ("rotary", 33), ("paged_rotary_append", 39), ("paged_decode_shared", 29)])
def test_packed_sizes_have_to_fit(clib, name, n):  # noqa: F811
    call = getattr(clib, f"fa_{name}_packed")
    for big in (2 ** 31, -2 ** 31 - 1):
        record = [0] * n
        record[-2] = big            # the last size
        assert call(struct.pack(f"{n}q", *record)) == BAD
    assert call(None) == BAD


def test_binding_refuses_wrong_tensors():
    # refused before the library is called: the tensors are on the CPU, or are not what they should be
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)      # noqa: E731
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)    # noqa: E731
    freq = torch.zeros(32)
    calls = [
        lambda: binding.fa_rotary(bf(1, 2, 3, 64), bf(1, 2, 3, 64), None, None, i32(1, 2), freq),
        lambda: binding.rotary_forward(bf(1, 2, 3, 64), bf(1, 2, 2, 64), i32(1, 2), freq),
        lambda: binding.rotary_backward(bf(1, 1, 3, 2, 64), bf(1, 1, 2, 64).float(), i32(1, 2), freq),
        lambda: binding.fa_paged_rotary_append(bf(2, 4, 64), bf(2, 2, 64), bf(2, 2, 64), i32(2), freq,
                                               torch.zeros(2, dtype=torch.int64), bf(2, 4, 64), bf(3, 2, 16, 64),
                                               bf(3, 2, 16, 64)),
        lambda: binding.fa_paged_free(i32(2), i32(4), i32(4, 5), i32(9), i32(9), i32(1), i32(4), i32(1), 16),
        lambda: binding.fa_paged_fork(i32(2), i32(2), i32(4), i32(4, 5), i32(9), i32(9), i32(1), i32(4), i32(2, 3),
                                      i32(1), 16),
        lambda: binding.fa_paged_compact(i32(4), i32(4, 5), i32(9), i32(9), i32(1), i32(4, 5), i32(9), i32(9),
                                         i32(2, 3), 16),
        lambda: binding.fa_paged_copy(i32(2, 3), bf(3, 2, 16, 64), bf(3, 2, 16, 64)),
        lambda: binding.fa_paged_decode_shared(bf(1, 4, 2, 1, 128), bf(3, 4, 16, 128), bf(3, 4, 16, 128), i32(1, 2),
                                               i32(1), i32(1), i32(2), i32(1), bf(1, 4, 2, 1, 128),
                                               torch.zeros(1, 4, 2, 1), None)]
    for call in calls:
        with pytest.raises(ValueError):
            call()
