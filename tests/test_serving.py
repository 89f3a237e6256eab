"""The paged operators together, as a server runs them: prompts turned and written into pages, forked into
samples that share them, decoded with the prefixes read once, cut after drafted tokens, compacted, and
decoded on."""
import numpy as np
import pytest
import torch

from flash_attention_gqa_gb300 import binding
import _paged as P
from test_rotary import angles, close, turned

pytestmark = pytest.mark.gpu
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_serving(lib, dtype):
    B, K, G, H, page, n_pages, cols = 10, 2, 4, 128, 16, 2000, 8192     # (wide tables: the groups are used)
    gen = torch.Generator(device="cuda").manual_seed(5)
    rng = np.random.default_rng(5)
    caches = [torch.full((n_pages, K, page, H), float("nan"), device="cuda").to(dtype) for _ in range(2)]
    scales = {}
    if dtype == E4M3:
        scales = dict(k_scale=torch.full((K,), 0.02, device="cuda"), v_scale=torch.full((K,), 0.03, device="cuda"))
    lens, table = _i32(np.zeros(B)), _i32(np.full((B, cols), -1))
    free, used, shares = _i32(rng.permutation(n_pages)), _i32([0]), _i32(np.zeros(n_pages))
    freq = (10000.0 ** (-torch.arange(H // 2).double() / (H // 2))).float().cuda()
    texts = [[] for _ in range(B)]          # (key, value) of every token, before the rotation

    def grow(new, T=None):
        """New tokens of every request into the cache; their queries, turned ([B, K, G, T, H] if T)."""
        nonlocal lens, used
        total = int(sum(new))
        before = lens.tolist()
        lens, starts, slots, positions, used = binding.paged_tables(
            lens, _i32(new), free, used, table, n_pages=n_pages, page_size=page, max_tokens=total)
        qkv = torch.randn((total, (G + 2) * K, H), generator=gen, device="cuda").to(BF16)
        shape = (B, K, G, T, H) if T else (total, K * G, H)
        q = torch.empty(shape, dtype=BF16, device="cuda")
        binding.fa_paged_rotary_append(qkv[:, :K * G], qkv[:, K * G:-K], qkv[:, -K:], positions, freq, slots, q,
                                       *caches, q_scale=H ** -0.5, **scales)
        want = [n + j for n, m in zip(before, new) for j in range(m)]
        assert positions.tolist() == want
        at = 0
        for b, m in enumerate(new):
            texts[b] = texts[b] + list(qkv[at:at + m, K * G:].cpu())
            at += m
        flat = q.permute(0, 3, 1, 2, 4).reshape(total, K * G, H) if T else q
        close(flat.cpu(), *turned(qkv[:, :K * G].cpu(), angles(positions.cpu()[None], freq.cpu(), None), False,
                                  H ** -0.5))
        return q

    def check(q, members, starts, prefix):
        o, lse = binding.paged_attention_decode_shared(q, *caches, table, lens, _i32(members), _i32(starts),
                                                       _i32(prefix), **scales)
        torch.cuda.synchronize()
        assert binding.fa_check_status() == binding.FA_OK
        host = [c.cpu() for c in caches]
        ks, vs = (scales[n].cpu() if scales else None for n in ("k_scale", "v_scale"))
        want = P.decode(q.cpu(), *host, table.cpu(), lens.cpu(), ks, vs)
        P.check_decode(o.cpu(), lse.cpu(), want, H, dtype == E4M3, int(lens.max()) + 16)
        plain, _ = binding.paged_attention_decode(q, *caches, table, lens, **scales)
        assert (plain.float() - o.float()).abs().max() <= 2.0 ** -6 * plain.float().abs().max()

    def check_cache():
        """Every request's pages hold its own tokens, turned."""
        for b, text in enumerate(texts):
            assert int(lens[b]) == len(text)
            if not text:
                continue
            rows = torch.stack(text)
            pos = torch.arange(len(text))
            ids = table[b].cpu()[pos // page].long()
            k, size = turned(rows[:, :K], angles(pos[None], freq.cpu(), None), False)
            for c, want, slack, s in ((caches[0], k, size, scales.get("k_scale")),
                                      (caches[1], rows[:, K:].double(), 0 * size, scales.get("v_scale"))):
                got = c.cpu().float()[ids, :, pos % page]
                if s is None:
                    close(got, want, slack)
                else:
                    s = s.cpu().double()[None, :, None]
                    tol = torch.maximum(2.0 ** -4 * (want / s).abs(), torch.tensor(2.0 ** -10).double())
                    assert ((got.double() - want / s).abs() <= tol * (1 + 2.0 ** -20) + 2.0 ** -21 * slack / s).all()

    # two prompts, samples of each
    grow([150, 0, 0, 0, 0, 83, 0, 0, 0, 0])
    copies = binding.paged_fork(_i32([0, 0, 0, 5, 5, 5, -1]), _i32([1, 2, 3, 6, 7, 8, 0]), lens, table, shares, free, used,
                                page_size=page)
    binding.fa_paged_copy(copies, *caches)
    for p, c in ((0, 1), (0, 2), (0, 3), (5, 6), (5, 7), (5, 8)):
        texts[c] = list(texts[p])
    members, starts, prefix = [3, 0, 1, 2, 8, 5, 7, 6], [0, 4, 8], [150 // page * page, 83 // page * page]
    for _ in range(3):
        q = grow([1] * B, T=1)
        check(q, members, starts, prefix)
    check_cache()
    # four drafted tokens each, of which some are taken
    q = grow([4] * B, T=4)
    check(q, members, starts, prefix)
    keep = [int(n) - int(rng.integers(0, 5)) for n in lens.tolist()]
    binding.paged_free(_i32(list(range(B))), lens, table, shares, free, used, page_size=page, keep=_i32(keep))
    texts[:] = [t[:n] for t, n in zip(texts, keep)]
    # one sample ends, another goes on from a third one's start; the pool is made dense
    binding.paged_free(_i32([2, 7]), lens, table, shares, free, used, page_size=page)
    copies = binding.paged_fork(_i32([1]), _i32([2]), lens, table, shares, free, used, page_size=page,
                                fork_lens=_i32([149]))
    binding.fa_paged_copy(copies, *caches)
    texts[2], texts[7] = texts[1][:149], []
    moves = binding.paged_compact(lens, table, shares, free, used, page_size=page, max_moves=n_pages)
    binding.fa_paged_copy(moves, *caches)
    torch.cuda.synchronize()
    held = {int(p) for b, t in enumerate(texts) for p in table[b, :P.up(len(t), page)]}
    assert held == set(range(len(held))) and (moves[:, 0] >= 0).any()
    check_cache()
    q = grow([1] * B, T=1)
    check(q, [0, 1, 2, 3, 8, 5, 6], [0, 4, 7], [144, 80])
    check_cache()
    # everything ends: no page is lost
    binding.paged_free(_i32(list(range(B))), lens, table, shares, free, used, page_size=page)
    torch.cuda.synchronize()
    assert used.item() == 0 and sorted(free.tolist()) == list(range(n_pages)) and not shares.any()
    assert binding.fa_check_status() == binding.FA_OK


def test_training_step(lib):
    """A projection's queries and keys turned, attended to, and their gradients turned back: against the
    same in 64 bits with torch's gradients."""
    B, T, K, G, H, pairs = 2, 96, 2, 2, 128, 32
    gen = torch.Generator().manual_seed(3)
    q, k = ((torch.randn((B, T, n, H), generator=gen) * 0.7).to(BF16) for n in (K * G, K))
    v = torch.randn((B, K, T, H), generator=gen).to(BF16)
    pos = torch.stack([torch.arange(T) // 8, torch.arange(T) % 8])[:, None].expand(2, B, T).contiguous().int()
    freq = (100.0 ** (-torch.arange(pairs).double() / pairs)).float()
    axes = (torch.arange(pairs) % 2).int()
    turn = (pos.cuda(), freq.cuda(), axes.cuda())
    qr, kr = binding.rotary_forward(q.cuda(), k.cuda(), *turn)
    o, lse = binding.attention_forward(qr, kr, v.cuda(), causal=True)
    dO = torch.randn(o.shape, generator=gen).to(BF16)
    dqr, dkr, _ = binding.attention_backward(qr, kr, v.cuda(), o, lse, dO.cuda(), causal=True)
    dq, dk = binding.rotary_backward(dqr, dkr, *turn)
    torch.cuda.synchronize()
    assert binding.fa_check_status() == binding.FA_OK
    angle = angles(pos.flatten(1), freq, axes).view(B, T, 1, pairs)
    leaves = [x.double().requires_grad_() for x in (q, k)]

    def spin(x):
        a, b, rest = x[..., :pairs], x[..., pairs:2 * pairs], x[..., 2 * pairs:]
        return torch.cat([a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin(), rest], -1)

    qx = (spin(leaves[0]) * H ** -0.5).transpose(1, 2).unflatten(1, (K, G))
    x = torch.einsum("bkgth,bksh->bkgts", qx, spin(leaves[1]).transpose(1, 2))
    x = x.masked_fill(torch.ones(T, T).triu(1).bool(), -torch.inf)
    out = torch.softmax(x, -1) @ v.double()[:, :, None]
    out.backward(dO.double())
    rel = lambda a, b: ((a.double().cpu() - b).norm() / b.norm()).item()    # noqa: E731
    # (the attention's own bounds: 5e-3 and 1e-2 in the 2-norm, of inputs rounded to bf16 once more here,
    # 2^-8 / sqrt(3) of them in the mean: 2.3e-3)
    assert rel(o, out.detach()) <= 5e-3 + 2.3e-3
    assert rel(dq, leaves[0].grad) <= 1e-2 + 2 * 2.3e-3 and rel(dk, leaves[1].grad) <= 1e-2 + 2 * 2.3e-3
