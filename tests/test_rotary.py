"""Rotary positions on the GPU against their definition: angles as exact fractions of a turn, products in
64 bits.

Tolerance.  The kernel's angle is off by 2^-23.3 (a turn's fraction as fp32 in half turns, at most 2^-25 off,
times pi), cos and sin by 2^-23 beside it: together below 2^-22.  a cos - b sin takes three more fp32
roundings, the scale one: (|a| + |b|) scale (2^-22 + 4 * 2^-24) < (|a| + |b|) scale 2^-21.  Then the result
is rounded to its type once: bf16 2^-8; e4m3 2^-4 of it, or 2^-10 (half of its smallest step), and the
quotient before it 2^-24."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from flash_attention_gqa_gb300 import binding
import _paged as P

pytestmark = pytest.mark.gpu
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn
# 1 / (2 pi) to 60 digits
PER_TURN = Fraction("0.159154943091895335768883763372514362034459645740456448747667")


def _ok():
    torch.cuda.synchronize()
    assert binding.fa_check_status() == binding.FA_OK


def angles(pos, freq, axes):
    """[tokens, pairs] in float64, reduced exactly: pos [n_axes, tokens]."""
    step = [int(Fraction(float(f)) * PER_TURN * 2 ** 120) for f in freq.tolist()]
    out = np.zeros((pos.shape[1], len(step)))
    for i, s in enumerate(step):
        row = pos[int(axes[i]) if axes is not None else 0].numpy().astype(object)
        out[:, i] = ((row * s) % 2 ** 120 / 2 ** 120).astype(np.float64)
    return torch.from_numpy(out) * (2 * math.pi)


def turned(x, angle, adjacent, scale=1.0):
    """(result, |a| + |b| per value) of x [tokens, heads, H] in float64."""
    x = x.double()
    n = angle.shape[-1]
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if adjacent else (slice(0, n), slice(n, 2 * n))
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    out, size = x.clone(), x.abs()
    out[..., a], out[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    both = x[..., a].abs() + x[..., b].abs()
    size[..., a], size[..., b] = both, both
    return out * scale, size * abs(scale)


def close(got, want, size, name=""):
    err = (got.double() - want).abs() - 2.0 ** -8 * want.abs() - 2.0 ** -21 * size
    assert err.numel() == 0 or err.max().item() <= 0, f"{name} off by {err.max().item():.3g} more than its roundings"


def make(seed, B, T, heads, H, pairs, n_axes, mixed, far, strides):
    """(x [B, T, heads, H] with its strides, positions [n_axes, B, T], freq, axes)"""
    gen = torch.Generator().manual_seed(seed)
    x = [(torch.randn((B, T, h + 3, H + 8), generator=gen)).to(BF16) for h in heads]
    x = [v[:, :, 1:1 + h, :H] if strides else v[:, :, :h, :H].contiguous() for v, h in zip(x, heads)]
    pos = torch.randint(-5 if far else 0, max(far, 1000), (n_axes, B, T), generator=gen).to(torch.int32)
    freq = (10000.0 ** (-torch.arange(pairs).double() / pairs)).float()
    axes = None if n_axes == 1 else (torch.arange(pairs) % n_axes if mixed
                                     else torch.arange(pairs) * n_axes // pairs).to(torch.int32)
    return x, pos, freq, axes


CASES = [  # B, T, q heads, k heads, H, pairs, axes, mixed, adjacent, far, strided
    (1, 1, 1, 1, 64, 32, 1, False, False, 0, False), (2, 3, 5, 2, 64, 8, 2, True, True, 0, True),
    (3, 77, 8, 2, 128, 64, 1, False, False, 10 ** 6, True), (1, 300, 16, 2, 256, 128, 3, False, False, 0, False),
    (2, 129, 4, 4, 128, 40, 4, True, False, 2 ** 31 - 1, True), (1, 50, 3, 0, 256, 64, 3, True, True, 2 ** 30, True),
    (4, 11, 12, 3, 256, 8, 1, False, False, 0, True), (2, 500, 32, 8, 128, 64, 1, False, True, 0, False),
    (1, 3000, 1, 1, 64, 24, 2, False, False, 99999, False), (70, 1, 7, 7, 64, 32, 16, True, False, 0, True),
    (1, 9000, 40, 8, 128, 64, 3, False, False, 0, True), (1, 40000, 1, 0, 256, 128, 1, False, False, 0, False),
    (3, 20001, 1, 1, 64, 32, 2, True, True, 0, True)]
each_case = pytest.mark.parametrize("case", CASES, ids=lambda c: "B%d_T%d_h%d+%d_H%d_p%d_ax%d%s%s_%d%s" % (
    *c[:7], "m" if c[7] else "", "_adj" if c[8] else "", c[9], "_str" if c[10] else ""))


@pytest.mark.parametrize("inverse", [False, True], ids=["forward", "inverse"])
@each_case
def test_rotary(lib, case, inverse):
    B, T, qh, kh, H, pairs, n_axes, mixed, adjacent, far, strides = case
    xs, pos, freq, axes = make(B + T, B, T, (qh, kh), H, pairs, n_axes, mixed, far, strides)
    dev = [x.cuda() if not strides else P.to_device(x, "cuda") for x in xs]
    out = [torch.full((B, h + 1, T + 2, H + 16), 5.0, dtype=BF16, device="cuda") for h in (qh, kh)]
    view = [o[:, :h, 1:T + 1, 8:H + 8].transpose(1, 2) for o, h in zip(out, (qh, kh))]
    p = pos.cuda() if not strides else pos.permute(1, 2, 0).contiguous().cuda().permute(2, 0, 1)
    binding.fa_rotary(dev[0], view[0], dev[1] if kh else None, view[1] if kh else None, p, freq.cuda(),
                      None if axes is None else axes.cuda(), q_scale=H ** -0.5, adjacent=adjacent, inverse=inverse)
    _ok()
    angle = angles(pos.flatten(1), freq, axes) * (-1 if inverse else 1)
    for i, (x, o, v, h, scale) in enumerate(zip(xs, out, view, (qh, kh), (H ** -0.5, 1.0))):
        want, size = turned(x.reshape(B * T, h, H), angle, adjacent, scale)
        close(v.reshape(B * T, h, H).cpu(), want, size, "qk"[i])
        v.fill_(5.0)
        assert (o == 5.0).all()         # nothing beside the outputs was written


def test_rotary_in_place_and_no_heads(lib):
    xs, pos, freq, axes = make(3, 2, 40, (6, 2), 128, 64, 2, True, 0, True)
    dev = [P.to_device(x, "cuda") for x in xs]
    binding.fa_rotary(dev[0], dev[0], dev[1], dev[1], pos.cuda(), freq.cuda(), axes.cuda())
    angle = angles(pos.flatten(1), freq, axes)
    for x, d in zip(xs, dev):
        close(d.reshape(80, -1, 128).cpu(), *turned(x.reshape(80, -1, 128), angle, False))
    with pytest.raises(binding.FAError):    # in place with other strides
        binding.fa_rotary(dev[0], dev[0].as_strided(dev[0].shape, (8000, 400, 128, 1), dev[0].storage_offset()),
                          None, None, pos.cuda(), freq.cuda(), axes.cuda())
    empty = torch.empty((2, 0, 6, 128), dtype=BF16, device="cuda")
    binding.fa_rotary(empty, empty, None, None, torch.empty((2, 0), dtype=torch.int32, device="cuda"), freq.cuda())
    _ok()


def test_rotary_one_axis_without_its_dim(lib):
    xs, pos, freq, _ = make(4, 3, 5, (4, 1), 64, 32, 1, False, 0, False)
    a, b = ([torch.empty_like(x, device="cuda") for x in xs] for _ in range(2))
    dev = [x.cuda() for x in xs]
    binding.fa_rotary(dev[0], a[0], dev[1], a[1], pos.cuda(), freq.cuda())
    binding.fa_rotary(dev[0], b[0], dev[1], b[1], pos[0].cuda(), freq.cuda(), torch.zeros(32, dtype=torch.int32).cuda())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    _ok()


def test_rotary_frequencies_of_every_size(lib):
    """From the smallest number to 2^40, negative ones and zero, at the ends of the positions."""
    freq = torch.tensor([2.0 ** -149, -(2.0 ** -130), 2.0 ** -60, 1e-9, -0.3, 1.0, 3.1415927, 2.0 ** 23 + 1,
                         2.0 ** 24 + 2, 1e9, 2.0 ** 40, 0.0, -0.0, 6.2831855, 0.5, -7777.7])
    pos = torch.tensor([[-2 ** 31, 2 ** 31 - 1, 0, 1, -1, 123456789]], dtype=torch.int32)
    x = torch.randn((1, 6, 2, 64), generator=torch.Generator().manual_seed(1)).bfloat16()
    y = torch.empty_like(x, device="cuda")
    binding.fa_rotary(x.cuda(), y, None, None, pos[:, None].cuda(), freq.cuda())
    close(y[0].cpu(), *turned(x[0], angles(pos, freq, None), False))
    _ok()


def test_rotary_values_that_are_not_finite_stay_in_their_pair(lib):
    x = torch.ones((1, 4, 1, 64), dtype=BF16)
    x[0, 1, 0, 3], x[0, 2, 0, 40] = math.inf, math.nan
    freq = torch.full((16,), 0.3)
    y = torch.empty_like(x, device="cuda")
    binding.fa_rotary(x.cuda(), y, None, None, torch.ones((1, 4), dtype=torch.int32).cuda(), freq.cuda())
    bad = ~torch.isfinite(y.cpu())[0, :, 0]
    assert bad[0].sum() == 0 and bad[1].nonzero()[:, 0].tolist() == [3, 19]
    assert bad[2].nonzero()[:, 0].tolist() == [40] and bad[3].sum() == 0
    _ok()


def test_rotary_odd_tables(lib):
    """An axis out of range counts as 0 and a frequency that is no number as 0; both are reported."""
    xs, pos, freq, axes = make(4, 1, 5, (2, 1), 64, 16, 2, True, 0, False)
    dev = [x.cuda() for x in xs]
    for fault in range(4):
        f, ax = freq.clone(), axes.clone()
        if fault < 2:
            ax[5] = (2, -1)[fault]
            want_axes = ax.clone()
            want_axes[5] = 0
            want = angles(pos.flatten(1), f, want_axes)
        else:
            f[7] = (math.inf, math.nan)[fault - 2]
            zero = f.clone()
            zero[7] = 0
            want = angles(pos.flatten(1), zero, ax)
        out = [torch.empty_like(x) for x in dev]
        binding.fa_rotary(dev[0], out[0], dev[1], out[1], pos.cuda(), f.cuda(), ax.cuda())
        torch.cuda.synchronize()
        assert binding.fa_check_status() == binding.FA_ERR_DEVICE_VALUE
        close(out[0].reshape(5, 2, 64).cpu(), *turned(xs[0].reshape(5, 2, 64), want, False))
    _ok()


@pytest.mark.parametrize("adjacent", [False, True])
def test_rotary_gradient(lib, adjacent):
    """The inverse call gives the formula's gradient, torch's of the plain form, and its differences."""
    B, T, K, G, H, pairs = 2, 9, 2, 3, 64, 24
    xs, pos, freq, axes = make(7, B, T, (K * G, K), H, pairs, 3, True, 0, False)
    angle = angles(pos.flatten(1), freq, axes)
    q, k = (x.cuda() for x in xs)
    turn = (pos.cuda(), freq.cuda(), axes.cuda())
    qo, ko = binding.rotary_forward(q, k, *turn, adjacent=adjacent)
    assert qo.shape == (B, K, G, T, H) and ko.shape == (B, K, T, H) and qo.is_contiguous() and ko.is_contiguous()
    close(ko.transpose(1, 2).reshape(B * T, K, H).cpu(), *turned(xs[1].reshape(B * T, K, H), angle, adjacent))
    gen = torch.Generator().manual_seed(2)
    dq, dk = (torch.randn(x.shape, generator=gen).bfloat16() for x in (qo, ko))
    gq, gk = binding.rotary_backward(dq.cuda(), dk.cuda(), *turn, adjacent=adjacent)
    assert gq.shape == q.shape and gk.shape == k.shape
    for x, d, g, h, scale in ((xs[0], dq.flatten(1, 2), gq, K * G, H ** -0.5), (xs[1], dk, gk, K, 1.0)):
        leaf = x.reshape(B * T, h, H).double().requires_grad_()
        # differentiable: the plain form without its writes in place
        c, s = angle.cos()[:, None], angle.sin()[:, None]
        a, b = (leaf[..., 0:2 * pairs:2], leaf[..., 1:2 * pairs:2]) if adjacent else (
            leaf[..., :pairs], leaf[..., pairs:2 * pairs])
        y = [a * c - b * s, b * c + a * s]
        y = torch.stack(y, -1).flatten(-2) if adjacent else torch.cat(y, -1)
        y = torch.cat([y, leaf[..., 2 * pairs:]], -1) * scale
        up = d.transpose(1, 2).reshape(B * T, h, H).double()
        y.backward(up)
        _, size = turned(up, -angle, adjacent, scale)
        close(g.reshape(B * T, h, H).cpu(), leaf.grad, size)
        # the form is linear: a difference of any size gives the derivative
        for i in range(3):
            at = torch.zeros(B * T, h, H, dtype=torch.float64)
            at[i * 5, h - 1, (i * 17) % H] = 1
            moved = turned(leaf.detach() + at, angle, adjacent, scale)[0] - turned(leaf.detach(), angle, adjacent, scale)[0]
            want = (moved * up).sum()
            got = g.reshape(B * T, h, H)[i * 5, h - 1, (i * 17) % H].double().cpu()
            assert abs(got - want) <= 2.0 ** -8 * abs(want) + 2.0 ** -21 * size[i * 5, h - 1].max() + 1e-12
    _ok()


# ----------------------------------------------------------- into the cache

APPENDS = [  # B, T, pad, K, G, H, pairs, axes, page, layout, far
    (1, 1, 0, 1, 1, 64, 32, 1, 1, "head", 0), (64, 1, 0, 8, 4, 128, 64, 1, 16, "token", 10 ** 6),
    (3, 5, 0, 2, 8, 256, 128, 3, 8, "head", 0), (1, 333, 9, 2, 3, 128, 24, 2, 64, "head", 0),
    (1, 2000, 77, 4, 5, 64, 32, 3, 256, "token", 2 ** 31 - 1), (1, 5000, 0, 8, 8, 128, 64, 1, 16, "head", 0)]


def _append(case, dtype, adjacent=False, seed=0):
    B, T, pad, K, G, H, pairs, n_axes, page, layout, far = case
    N = B * T + pad
    gen = torch.Generator().manual_seed(seed + N)
    (q, kv), pos, freq, axes = make(N, 1, N, (K * G, 2 * K), H, pairs, n_axes, True, far, True)
    q, k, v = q[0], kv[0][:, :K], kv[0][:, K:]
    n_pages = P.up(N, page) + 3
    slots = torch.randperm(n_pages * page, generator=gen)[:N]
    slots[B * T:] = -1
    caches = [P.cache(n_pages, K, page, H, dtype, layout, gen, fill=1.5, pad=32) for _ in range(2)]
    scales = [torch.rand(K, generator=gen) / 10 + 0.01 for _ in range(2)] if dtype == E4M3 else [None, None]
    shape = (1, K, G, N, H) if pad else (B, K, G, T, H)
    return q, k, v, pos[:, 0], freq, axes, slots, caches, scales, torch.full(shape, 7.0, dtype=BF16)


def _check_append(case, dtype, adjacent, data, q_out, dev):
    B, T, pad, K, G, H, pairs, n_axes, page, layout, far = case
    q, k, v, pos, freq, axes, slots, caches, scales, _ = data
    N = B * T + pad
    angle = angles(pos, freq, axes)
    want, size = turned(q, angle, adjacent, H ** -0.5)
    got = q_out.permute(0, 3, 1, 2, 4).reshape(N, K * G, H).cpu()
    live = slots >= 0
    close(got[live], want[live], size[live], "q")
    assert (got[~live] == 7.0).all()
    for (x, size), before, after, scale in zip((turned(k, angle, adjacent), (v.double(), 0 * v.double())), caches,
                                               dev, scales):
        at = slots[live]
        old = before.contiguous().view(torch.uint8)
        new = after.cpu().contiguous().view(torch.uint8)
        rows = after.cpu()[at // page, :, at % page] if dtype == BF16 else (
            new[at // page, :, at % page].view(E4M3).float())
        if scale is None:
            close(rows, x[live], size[live], "cache")
        else:
            s = scale.double()[:, None]
            ref, slack = (x[live] / s).clamp(-448, 448), size[live] / s
            err = (rows.double() - ref).abs()
            tol = torch.maximum(2.0 ** -4 * ref.abs(), torch.tensor(2.0 ** -10).double())
            assert (err <= tol * (1 + 2.0 ** -20) + 2.0 ** -21 * slack).all()
        # other slots are as they were
        rest = torch.ones(before.shape[0] * page, dtype=torch.bool)
        rest[at] = False
        for t in (old, new):
            t[at // page, :, at % page] = 0
        assert torch.equal(old, new)


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("adjacent", [False, True], ids=["halves", "adjacent"])
@pytest.mark.parametrize("case", APPENDS, ids=lambda c: "B%d_T%d_pad%d_K%d_G%d_H%d_p%d_ax%d_page%d_%s_%d" % c)
def test_rotary_append(lib, case, adjacent, dtype):
    data = _append(case, dtype, adjacent)
    q, k, v, pos, freq, axes, slots, caches, scales, q_out = data
    dev = [P.to_device(c, "cuda") for c in caches]
    on = lambda x: None if x is None else x.cuda()          # noqa: E731
    wide = torch.cat([q, k, v], 1).cuda()                   # a fused projection's output
    h = q.shape[1]
    q_out = q_out.cuda()
    binding.fa_paged_rotary_append(wide[:, :h], wide[:, h:h + k.shape[1]], wide[:, h + k.shape[1]:], on(pos),
                                   on(freq), on(slots), q_out, *dev, on(axes), on(scales[0]), on(scales[1]),
                                   q_scale=case[5] ** -0.5, adjacent=adjacent)
    _ok()
    _check_append(case, dtype, adjacent, data, q_out, dev)
    flat = torch.empty((q.shape[0], h, case[5]), dtype=BF16, device="cuda")     # q_out as [N, heads, H]
    binding.fa_paged_rotary_append(on(q), on(k), on(v), on(pos), on(freq), on(slots), flat, *dev, on(axes),
                                   on(scales[0]), on(scales[1]), q_scale=case[5] ** -0.5, adjacent=adjacent)
    live = slots >= 0
    B, K, G, T, H = q_out.shape
    assert torch.equal(flat.cpu()[live], q_out.permute(0, 3, 1, 2, 4).reshape(-1, h, H).cpu()[live])
    _ok()


@pytest.mark.parametrize("scale", [1e-39, 2e-38, 1e38, 3e38])
def test_rotary_append_scales_at_the_ends_of_their_range(lib, scale):
    # positions of zero: keys stay as they are, and only the scale and e4m3 are left
    case = (1, 40, 0, 2, 1, 64, 32, 1, 8, "head", 0)
    data = list(_append(case, E4M3))
    k, v = data[1].contiguous(), data[2].contiguous()
    big = scale * 20 if scale < 1 else 3e38
    for x in (k, v):
        x.copy_((x.float() * big / 4).clamp(-3e38, 3e38))
        x[::3, :, ::2] = 0
    scales = torch.full((2,), scale)
    dev = [P.to_device(c, "cuda") for c in data[7]]
    binding.fa_paged_rotary_append(data[0].cuda(), k.cuda(), v.cuda(), torch.zeros_like(data[3]).cuda(),
                                   data[4].cuda(), data[6].cuda(), data[9].cuda(), *dev, None, scales.cuda(),
                                   scales.cuda())
    _ok()
    at = data[6]
    for x, c in zip((k, v), dev):
        rows = c.cpu().contiguous().view(torch.uint8)[at // 8, :, at % 8].view(E4M3).double()
        ref = (x.double() / scales.double()[0]).clamp(-448, 448)
        tol = torch.maximum(2.0 ** -4 * ref.abs(), torch.tensor(2.0 ** -10).double())
        assert ((rows - ref).abs() <= tol * (1 + 2.0 ** -20)).all()


def test_rotary_append_slots_past_the_cache(lib):
    case = (1, 20, 0, 2, 2, 64, 32, 1, 8, "head", 0)
    data = list(_append(case, BF16))
    slots, caches = data[6], data[7]
    slots[3], slots[7] = caches[0].shape[0] * 8, 2 ** 45
    dev = [P.to_device(c, "cuda") for c in caches]
    q_out = data[9].cuda()
    binding.fa_paged_rotary_append(*(x.cuda() for x in data[:3]), data[3].cuda(), data[4].cuda(), slots.cuda(),
                                   q_out, *dev, q_scale=0.125)
    torch.cuda.synchronize()
    assert binding.fa_check_status() == binding.FA_ERR_DEVICE_VALUE
    angle = angles(data[3], data[4], None)
    close(q_out[0].permute(2, 0, 1, 3).reshape(20, 4, 64).cpu(), *turned(data[0], angle, False, 0.125))
    kept = slots.clone()
    kept[3] = kept[7] = -1
    for c, d in zip(caches, dev):
        changed = (c.contiguous() != d.cpu().contiguous()).any(-1).any(1).flatten().nonzero()[:, 0]
        assert set(changed.tolist()) <= set(kept[kept >= 0].tolist())
    _ok()


def test_rotary_on_a_side_stream_and_in_a_graph(lib):
    xs, pos, freq, axes = make(9, 2, 33, (8, 2), 128, 64, 3, False, 0, False)
    q, k = (x.cuda() for x in xs)
    p, f, ax = pos.cuda(), freq.cuda(), axes.cuda()
    out = [torch.zeros_like(q), torch.zeros_like(k)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            binding.fa_rotary(q, out[0], k, out[1], p, f, ax)
    p += 100
    torch.cuda.synchronize()
    graph.replay()
    binding.fa_rotary(q, q, None, None, p, f, ax, stream=side)
    torch.cuda.synchronize()
    angle = angles((pos + 100).flatten(1), freq, axes)
    for o, x in zip(out, xs):
        close(o.reshape(66, -1, 128).cpu(), *turned(x.reshape(66, -1, 128), angle, False))
    assert torch.equal(q, out[0])
    _ok()
