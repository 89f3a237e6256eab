"""The paged cache operators without a GPU: argument checks of the C ABI (fake pointers: every
call is refused, or has nothing to do, before any launch) and of the binding."""
import ctypes
import os
import struct
import subprocess
import sys

import pytest
import torch

from flash_attention_gqa_gb300 import binding
from test_boundary import clib  # noqa: F401  (fixture)

BAD, UNSUP, OK = binding.FA_ERR_INVALID_ARG, binding.FA_ERR_UNSUPPORTED, binding.FA_OK


def _both(lib, name, *args):
    """The status of a call with plain arguments, which its packed form has to give too."""
    rc = getattr(lib, name)(*args)
    record = struct.pack(f"{len(args)}q", *(0 if x is None else x for x in args))
    assert getattr(lib, name + "_packed")(record) == rc
    return rc


def _tables(lib, cached=16, new=16, free=16, n_free=10, used=16, table=16, max_pages=8, total=16,
            starts=16, slots=16, positions=16, max_tokens=64, used_out=16, B=4, n_pages=100,
            page=16):
    return _both(lib, "fa_paged_tables", cached, new, free, n_free, used, table, max_pages, total, starts,
                 slots, positions, max_tokens, used_out, B, n_pages, page, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(cached=None), BAD), (dict(new=None), BAD), (dict(free=None), BAD), (dict(used=None), BAD),
    (dict(table=None), BAD), (dict(total=None), BAD), (dict(starts=None), BAD),
    (dict(slots=None), BAD), (dict(slots=20), BAD), (dict(positions=2), BAD),
    (dict(used_out=None), BAD), (dict(B=-1), BAD), (dict(n_free=-1), BAD), (dict(max_pages=-1), BAD),
    (dict(max_tokens=-1), BAD), (dict(n_pages=-1), BAD), (dict(page=0), BAD), (dict(page=-16), BAD),
    (dict(page=24), UNSUP), (dict(page=1 << 17), UNSUP), (dict(B=8193), UNSUP),
    (dict(max_pages=1 << 27), UNSUP), (dict(max_tokens=(1 << 30) + 1), UNSUP),
])
def test_tables_refusals(clib, kw, rc):  # noqa: F811
    assert _tables(clib, **kw) == rc


def _append(lib, k=16, v=16, kt=1024, kh=128, vt=1024, vh=128, slots=16, kc=16, vc=16, kind=0,
            ks=None, vs=None, sp=16384, sh=2048, st=128, N=4, K=8, H=128, n_pages=10, page=16):
    return _both(lib, "fa_paged_append", k, v, kt, kh, vt, vh, slots, kc, vc, kind, ks, vs, sp, sh, st, N, K,
                 H, n_pages, page, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(k=None), BAD), (dict(v=8), BAD), (dict(slots=None), BAD), (dict(slots=4), BAD),
    (dict(kc=None), BAD), (dict(vc=24), BAD), (dict(kind=2), BAD), (dict(kind=-1), BAD),
    (dict(kt=1023), BAD), (dict(vh=-128), BAD), (dict(sp=16388), BAD), (dict(kind=1, st=136), BAD),
    (dict(sh=-2048), BAD), (dict(ks=16), BAD), (dict(kind=1, vs=2), BAD), (dict(N=-1), BAD),
    (dict(n_pages=-1), BAD), (dict(page=0), BAD), (dict(page=12), UNSUP), (dict(H=96), UNSUP),
    (dict(H=512), UNSUP), (dict(K=65536), UNSUP), (dict(N=0, k=None, v=None), OK),
    (dict(K=0), OK),
])
def test_append_refusals(clib, kw, rc):  # noqa: F811
    assert _append(clib, **kw) == rc


def _decode(lib, q=16, kc=16, vc=16, kind=0, ks=None, vs=None, sp=16384, sh=2048, st=128, table=16,
            lens=16, window=0, o=16, lse=16, ws=256, ws_bytes=1 << 30, B=4, K=8, G=4, T=1, H=128,
            n_pages=10, page=16, max_pages=8):
    return _both(lib, "fa_paged_decode", q, kc, vc, kind, ks, vs, sp, sh, st, table, lens, window, o, lse,
                 ws, ws_bytes, B, K, G, T, H, n_pages, page, max_pages, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(q=None), BAD), (dict(q=8), BAD), (dict(o=None), BAD), (dict(lse=None), BAD),
    (dict(lens=None), BAD), (dict(lens=2), BAD), (dict(table=None), BAD), (dict(kc=None), BAD),
    (dict(vc=8), BAD), (dict(kind=3), BAD), (dict(window=-1), BAD), (dict(B=-1), BAD),
    (dict(T=-1), BAD), (dict(max_pages=-1), BAD), (dict(st=132), BAD), (dict(ks=16), BAD),
    (dict(kind=1, ks=2), BAD), (dict(page=48), UNSUP), (dict(H=192), UNSUP), (dict(G=129), UNSUP),
    (dict(G=16, T=9), UNSUP), (dict(B=8193), UNSUP), (dict(B=8192, K=8), UNSUP),
    (dict(max_pages=1 << 27), UNSUP), (dict(ws=None), BAD), (dict(ws=128), BAD),
    (dict(B=0), OK), (dict(T=0, q=None), OK),
    (dict(G=0), OK), (dict(K=0), OK),
])
def test_decode_refusals(clib, kw, rc):  # noqa: F811
    assert _decode(clib, **kw) == rc


def test_strides_of_single_dims_do_not_matter(clib):  # noqa: F811
    # one kv head, one page: their strides are never used, aligned or not (nothing to do: B = 0)
    assert _decode(clib, B=0, K=1, sh=3, n_pages=1, sp=5) == OK
    assert _append(clib, N=0, K=1, sh=3, kh=1, kt=1) == OK


def test_workspace_size_of_nothing(clib):  # noqa: F811
    size = binding.fa_paged_decode_workspace_size
    assert size(0, 1, 1, 1, 128) == 0
    assert size(1, 1, 1, 1, 96) == 0
    assert size(1, 1, 129, 1, 128) == 0
    assert size(8193, 1, 1, 1, 128) == 0


def test_status_string(clib):  # noqa: F811
    assert binding.status_string(binding.FA_ERR_DEVICE_VALUE) != binding.status_string(99)


def test_binding_refuses_wrong_tensors():
    # refused before the library is called: the tensors are on the CPU
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        binding.fa_paged_tables(i32(2), i32(2), i32(4), i32(1), i32(2, 4), i32(2), i32(3),
                                torch.zeros(8, dtype=torch.int64), None, i32(1), 8, 16)
    with pytest.raises(ValueError):
        binding.fa_paged_append(bf(2, 4, 128), bf(2, 4, 128), torch.zeros(2, dtype=torch.int64),
                                bf(3, 4, 16, 128), bf(3, 4, 16, 128))
    with pytest.raises(ValueError):
        binding.fa_paged_append(torch.zeros(2, 4, 128), bf(2, 4, 128),
                                torch.zeros(2, dtype=torch.int64), bf(3, 4, 16, 128),
                                bf(3, 4, 16, 128))
    with pytest.raises(ValueError):
        binding.fa_paged_decode(bf(1, 4, 2, 1, 128), bf(3, 4, 16, 128), bf(3, 4, 16, 128),
                                i32(1, 2), i32(1), bf(1, 4, 2, 1, 128), torch.zeros(1, 4, 2, 1), None)


@pytest.mark.parametrize("name,n", [("tables", 17), ("append", 21), ("decode", 25)])
def test_packed_sizes_have_to_fit(clib, name, n):  # noqa: F811
    # the second size argument from the end, past an int (and null pointers elsewhere)
    call = getattr(clib, f"fa_paged_{name}_packed")
    for big in (2 ** 31, 2 ** 32 + 1, -2 ** 31 - 1):
        record = [0] * n
        record[-3] = big
        assert call(struct.pack(f"{n}q", *record)) == BAD
    assert call(None) == BAD


def test_argument_types_are_plain(clib):  # noqa: F811
    for name in ("fa_paged_tables", "fa_paged_append", "fa_paged_decode"):
        assert binding.SIGNATURES[name][0] is ctypes.c_int


_WITHOUT_CUDA = """
import sys
sys.path.insert(0, {root!r})
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
from flash_attention_gqa_gb300 import binding
assert binding.FA_OK == 0 and "fa_paged_decode" in binding.SIGNATURES
lens = torch.zeros(2, dtype=torch.int32)
try:
    binding.fa_paged_tables(lens, lens, lens, lens[:1], lens[:, None], lens, lens, lens.long(), None,
                            lens[:1], 2, 16)
except ValueError as e:
    assert "CUDA" in str(e)
else:
    raise AssertionError("tensors on the CPU were taken")
"""


def test_binding_imports_with_a_torch_without_cuda():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", _WITHOUT_CUDA.format(root=root)], capture_output=True, text=True)
    assert run.returncode == 0, run.stderr
