"""Plain 64-bit forms of the paged cache operators, and inputs for their tests.

Everything here runs on the CPU in float64 loops over requests and queries; it
shares no code with the kernels."""
import math

import numpy as np
import torch


def up(n, m):
    return -(-n // m)


def tables(cached, new, free, used, table, page, max_tokens):
    """(table, total, starts, slots, positions, used) by a loop over tokens."""
    table, free = table.copy(), list(free)
    starts, slots, positions = [0], [], []
    for b, (c, n) in enumerate(zip(cached, new)):
        for j in range(up(c, page), up(c + n, page)):
            table[b, j] = free[used]
            used += 1
        for pos in range(c, c + n):
            slots.append(int(table[b, pos // page]) * page + pos % page)
            positions.append(pos)
        starts.append(len(slots))
    pad = [-1] * (max_tokens - len(slots))
    return (table, np.array(cached) + np.array(new), np.array(starts), np.array(slots + pad),
            np.array(positions + pad), used)


def cache(n_pages, K, page, H, dtype, layout, gen, fill=None, pad=0):
    """A cache [n_pages, K, page, H] stored head-major or token-major, `pad` unused elements
    behind each page; N(0, 1) values, or `fill` everywhere."""
    inner = (K, page) if layout == "head" else (page, K)
    per = K * page * H
    raw = torch.full((n_pages, per + pad), float("nan") if fill is None else fill)
    x = torch.randn((n_pages, per), generator=gen) if fill is None else raw[:, :per]
    raw[:, :per] = x
    raw = raw.to(dtype)
    view = raw.as_strided((n_pages, *inner, H), (per + pad, inner[1] * H, H, 1))
    return view if layout == "head" else view.transpose(1, 2)


def to_device(c, device):
    """A copy on `device` with the same strides."""
    store = torch.empty(0, dtype=torch.uint8).set_(c.untyped_storage()).to(device, copy=True)
    return store.view(c.dtype).as_strided(c.shape, c.stride(), c.storage_offset())


def values(c):
    """A cache's values in float64."""
    return c.float().double()


def decode(q, k_cache, v_cache, table, lens, ks=None, vs=None, window=0):
    """(o, lse, bound): the definition in float64, and per output element the sizes that its
    rounding errors scale with: sum p |v| and, per row, the largest sum |q||k|."""
    B, K, G, T, H = q.shape
    page = k_cache.shape[2]
    qd, kc, vc = q.double(), values(k_cache), values(v_cache)
    o = torch.zeros(q.shape, dtype=torch.float64)
    size = torch.zeros(q.shape, dtype=torch.float64)
    reach = torch.zeros(q.shape[:4], dtype=torch.float64)
    lse = torch.full(q.shape[:4], -math.inf, dtype=torch.float64)
    for b in range(B):
        n = int(lens[b])
        ids = torch.tensor([int(table[b, s // page]) for s in range(n)], dtype=torch.long)
        off = torch.arange(n) % page
        for h in range(K):
            k = kc[ids, h, off] * (1.0 if ks is None else float(ks[h]))
            v = vc[ids, h, off] * (1.0 if vs is None else float(vs[h]))
            for t in range(T):
                hi = n - T + t + 1
                lo = max(0, hi - window) if window else 0
                if hi <= lo:
                    continue
                kk, vv = k[lo:hi], v[lo:hi]
                x = qd[b, h, :, t] @ kk.T
                top = x.max(-1, keepdim=True).values
                w = (x - top).exp()
                l = w.sum(-1, keepdim=True)
                o[b, h, :, t] = w @ vv / l
                size[b, h, :, t] = w @ vv.abs() / l
                lse[b, h, :, t] = (top + l.log())[:, 0]
                reach[b, h, :, t] = (qd[b, h, :, t].abs() @ kk.abs().T).max(-1).values
    return o, lse, (size, reach)


def check_decode(o, lse, want, H, e4m3, n):
    """Element by element.  The score of a key is an fp32 sum of H products, off by at most
    H * 2^-24 * sum |q||k|; a weight's relative error is the score's, plus 2^-21 for the
    exponential and its argument, plus the rounding of the weights for the product with v
    (2^-11 in fp16, for 8-bit caches; 2^-16 as two bf16 terms); weights enter the numerator and
    the denominator; fp32 sums over n keys add n * 2^-24.  The result is rounded to bf16 once."""
    ro, rl, (size, reach) = want
    rel = H * 2.0 ** -24 * reach + 2.0 ** -21 + n * 2.0 ** -24
    tol = 2.0 ** -8 * ro.abs() + (2 * rel[..., None] + (2.0 ** -11 if e4m3 else 2.0 ** -16)) * size
    err = (o.double() - ro).abs()
    worst = (err - tol).max().item() if err.numel() else 0.0
    assert worst <= 1e-30, f"o off by {worst:.3g} more than its roundings"
    fine = torch.isfinite(rl)
    assert torch.equal(torch.isinf(lse), ~fine), "empty rows"
    dl = (lse.double() - rl)[fine].abs()
    assert (dl <= (rel + 2.0 ** -22 * rl.abs())[fine]).all(), f"lse off by {dl.max().item():.3g}"


def problem(seed, *, B, K, G, T, H, lens, page, dtype=torch.bfloat16, layout="head", pad=0,
            spare=3, extra_cols=2):
    """Inputs of a decode whose pages are shuffled and whose unowned slots hold NaN."""
    gen = torch.Generator().manual_seed(seed)
    held = [up(n, page) for n in lens]
    n_pages = sum(held) + spare
    perm = torch.randperm(n_pages, generator=gen)
    table = torch.full((B, max(held + [0]) + extra_cols), -1, dtype=torch.int32)
    at, owned = 0, torch.zeros(n_pages, page, dtype=torch.bool)
    for b, n in enumerate(lens):
        for j in range(held[b]):
            table[b, j] = perm[at]
            owned[perm[at], :min(page, n - j * page)] = True
            at += 1
    q = (torch.randn((B, K, G, T, H), generator=gen) * H ** -0.5).bfloat16()
    caches = []
    for _ in range(2):
        c = cache(n_pages, K, page, H, torch.float32, layout, gen, pad=pad)
        if dtype == torch.float8_e4m3fn:
            c.mul_(32)
        c.copy_(torch.where(owned[:, None, :, None], c, torch.tensor(float("nan"))))
        raw = c.as_strided((c.untyped_storage().nbytes() // 4,), (1,)).to(dtype)
        caches.append(raw.as_strided(c.shape, c.stride()))
    scales = [None, None]
    if dtype == torch.float8_e4m3fn:
        scales = [(torch.rand(K, generator=gen) + 0.5) / 32 for _ in range(2)]
    return q, *caches, table, torch.tensor(lens, dtype=torch.int32), *scales
