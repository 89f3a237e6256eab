"""Rotary positions, page management and shared-prefix attention, as cases to measure.

Three sets of operators around the paged key-value cache and the dense attention:
  rotary   queries and keys turned by positions of several axes: into the attention's
           layout (training), its gradient, and into the cache's pages (serving)
  pages    requests forked, freed and cut, their pages copied and compacted
  shared   attention of requests with a common prefix, its pages read once for all

``run`` computes them in a plain form (elementary torch operations in 32 bits, angles in
64); with ``own`` set it calls the library.  ``exact`` is the definition in 64 bits.
Caches are [layers,] [pages, kv heads, page size, head dim], read through their strides:
"head" layouts store them in that order, "token" layouts with the page's tokens outside
the heads.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
GOLDEN = 0.6180339887498949
SCRATCH = 256 << 20     # the workspace that a serving program sets aside at its start
BASE = 10000.0          # of the frequencies, BASE^(-i / pairs)


def listed():
    return [
        # Forward of the packed-document workload: queries and keys of a fused projection, turned
        # and laid out for the attention.
        dict(name="rotary_forward", op="rotary", B=4, T=4096, K=8, G=4, H=128, rot=128, axes=1,
             mixed=False, adjacent=False, inverse=False, far=0),
        # Gradients of images and video back through it: three axes, half of the dims, head dim 256.
        dict(name="rotary_backward", op="rotary", B=1, T=8191, K=2, G=8, H=256, rot=128, axes=3,
             mixed=True, adjacent=True, inverse=True, far=0),
        # One decode step of 64 requests: a token each, at far positions.
        dict(name="rotary_step", op="append", B=64, T=1, pad=0, K=8, G=4, H=128, rot=128, axes=1,
             mixed=False, adjacent=False, page=16, dtype="bf16", layout="token", far=131072),
        # Prompts with video frames into an 8-bit cache.
        dict(name="rotary_prompts", op="append", B=1, T=8000, pad=192, K=8, G=8, H=128, rot=128,
             axes=3, mixed=False, adjacent=False, page=64, dtype="e4m3", layout="head", far=0),
        # Verification of 8 drafted tokens: 256 requests drop those that were not taken.
        dict(name="pages_reject", op="release", B=256, lo=8, hi=4096, drop=8, page=16, pool=0.7),
        # A step of a beam search: half of 64 requests take over another one's tokens.
        dict(name="pages_beam", op="turnover", parents=32, children=32, lo=100, hi=2048, L=4, K=8,
             H=128, page=64, dtype="bf16", layout="head", pool=0.7),
        # 128 samples of one long prompt.
        dict(name="pages_samples", op="turnover", parents=1, children=128, lo=32750, hi=32750, L=2,
             K=8, H=128, page=64, dtype="bf16", layout="token", pool=0.7),
        # A pool of which a third is held, its pages everywhere, made dense.
        dict(name="pages_compact", op="compact", B=128, lo=16, hi=4096, L=2, K=8, H=128, page=16,
             dtype="bf16", layout="head", pool=0.33, most=4096),
        # Four samples of a short prompt: latency.
        dict(name="shared_one", op="shared", groups=1, members=4, K=2, G=8, T=1, H=256, lo=512,
             hi=512, tail=40, page=16, dtype="bf16", layout="head"),
        # 64 samples of one prompt.
        dict(name="shared_samples", op="shared", groups=1, members=64, K=8, G=8, T=1, H=128,
             lo=8192, hi=8192, tail=512, page=64, dtype="bf16", layout="head"),
        # A batch of several prompts, an 8-bit cache, samples of each.
        dict(name="shared_prompts", op="shared", groups=16, members=8, K=8, G=4, T=1, H=128,
             lo=256, hi=8192, tail=1024, page=32, dtype="e4m3", layout="token"),
        # A long document that 32 requests ask about, four drafted tokens each.
        dict(name="shared_document", op="shared", groups=1, members=32, K=2, G=8, T=4, H=256,
             lo=32768, hi=32768, tail=256, page=64, dtype="bf16", layout="head"),
    ]


def draw(rng):
    """A case of the same ranges: logarithmic sizes, odd ones among them."""
    def log(lo, hi):
        return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))

    op = rng.choice(["rotary", "append", "release", "turnover", "compact", "shared", "shared",
                     "shared"])
    page = 1 << rng.randrange(3, 9)
    K, H = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128, 256])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    dtype, layout = rng.choice(["bf16", "bf16", "e4m3"]), rng.choice(["head", "token"])
    if op in ("rotary", "append"):
        turn = dict(rot=rng.choice([H, H, H // 2, H // 4, 16 * rng.randrange(1, H // 16 + 1)]),
                    axes=rng.choice([1, 1, 2, 3, 4]), mixed=rng.random() < 0.5,
                    adjacent=rng.random() < 0.5, far=rng.choice([0, 0, log(1000, 1 << 29)]))
        B, T = log(1, 256), log(1, 16384)
        while B * T * K * G * H > 16384 * 4096:
            B, T = (B, T // 2) if T > 1 else (B // 2, T)
        if op == "rotary":
            return dict(op=op, B=B, T=T, K=K, G=G, H=H, inverse=rng.random() < 0.5, **turn)
        return dict(op=op, B=B, T=T, pad=rng.choice([0, rng.randrange(0, 64)]) if B == 1 else 0,
                    K=K, G=G, H=H, page=page, dtype=dtype, layout=layout, **turn)
    if op == "release":
        B = log(1, 512)
        hi = log(8, 32768)
        while B * hi > 1 << 22:
            hi //= 2
        return dict(op=op, B=B, lo=min(hi, 8), hi=hi, drop=rng.choice([0, 1, 8, log(1, hi)]),
                    page=page, pool=rng.choice([0.3, 0.7, 0.95]))
    if op == "turnover":
        parents, children, hi = log(1, 128), log(1, 256), log(8, 32768)
        L = rng.choice([1, 2, 4])
        while parents * hi > 40000 or (parents * (hi + page) + children * page) * L * K * H > 1 << 27:
            if L > 1:
                L //= 2
            elif parents > 1:
                parents //= 2
            else:
                hi, children = max(hi // 2, 8), max(children // 2, 1)
        return dict(op=op, parents=parents, children=children, lo=rng.choice([1, hi]), hi=hi, L=L,
                    K=K, H=H, page=page, dtype=dtype, layout=layout, pool=rng.choice([0.4, 0.8]))
    if op == "compact":
        B, hi, pool = log(1, 256), log(8, 8192), rng.choice([0.2, 0.33, 0.6, 0.9])
        L = rng.choice([1, 2])
        while B * (hi // 2 + page) * L * K * H / pool > 1 << 28 or B * hi > 1 << 18:
            B, hi = (B // 2, hi) if B > 1 else (B, max(hi // 2, 8))
            K = max(1, K // 2)
        return dict(op=op, B=B, lo=min(hi, 8), hi=hi, L=L, K=K, H=H, page=page, dtype=dtype,
                    layout=layout, pool=pool, most=log(1, 4096))
    T = rng.choice([1, 1, 1, rng.randrange(2, 9)])
    groups, members = log(1, 32), log(1, 64)
    hi, tail = log(page, 65536), log(1, 1024)
    while (groups * members * (hi + tail) * K * H > 64 * 8704 * 1024
           or groups * members * (hi + tail) * K * G * T > 1 << 28
           or groups * members * K * G * T * H > 1 << 24):
        if groups > 1:
            groups //= 2
        elif members > 2:
            members //= 2
        else:
            hi = max(page, hi // 2)
            tail = max(1, tail // 2)
            K = max(1, K // 2)
    return dict(op="shared", groups=groups, members=members, K=K, G=G, T=T, H=H,
                lo=rng.choice([min(page, hi), hi]), hi=hi, tail=tail, page=page, dtype=dtype,
                layout=layout)


# ------------------------------------------------------------------- sizes

def _lengths(n, lo, hi, phase=0.0):
    """n lengths spread over [lo, hi] by their logarithm: the case's, whatever the seed."""
    return [max(lo, min(hi, int(round(lo * (hi / lo) ** (((i + 0.5) * GOLDEN + phase) % 1.0)))))
            for i in range(n)]


def _pages(n, page):
    return -(-n // page)


def _shared_sizes(case):
    """(prefix of each group, tokens of each request behind its group's prefix)."""
    page, T = case["page"], case["T"]
    prefix = [max(page, n // page * page) for n in _lengths(case["groups"], case["lo"], case["hi"])]
    tails = _lengths(case["groups"] * case["members"], T, max(T, case["tail"]), 0.37)
    return prefix, tails


def _dropped(case):
    """(tokens, tokens kept) of each request of a release."""
    lens = _lengths(case["B"], case["lo"], case["hi"])
    if case["drop"] == 0:                                   # the requests end
        return lens, [0] * len(lens)
    return lens, [max(0, n - i * 7 % (case["drop"] + 1)) for i, n in enumerate(lens)]


def work(case):
    op = case["op"]
    e = 1 if case.get("dtype") == "e4m3" else 2
    if op in ("rotary", "append"):
        tokens = case["B"] * case["T"]
        q = tokens * case["K"] * case["G"] * case["H"]
        kv = tokens * case["K"] * case["H"]
        turned = (q + kv) * case["rot"] / case["H"]
        small = 4.0 * tokens * case["axes"] + 4.0 * case["rot"]
        if op == "rotary":
            return dict(bytes=4.0 * (q + kv) + small, flops=3.0 * turned)
        return dict(bytes=4.0 * q + 2.0 * kv * (2 + e) + small + 8.0 * tokens, flops=3.0 * turned)
    if op == "release":
        lens, keep = _dropped(case)
        gone = sum(_pages(a, case["page"]) - _pages(b, case["page"]) for a, b in zip(lens, keep))
        return dict(bytes=16.0 * case["B"] + 12.0 * gone + 8.0, flops=0.0)
    row = 2.0 * case.get("L", 1) * case["K"] * case["H"] * e    # bytes of a token's keys and values
    if op == "turnover":
        lens, page = _lengths(case["parents"], case["lo"], case["hi"]), case["page"]
        of = [lens[i % len(lens)] for i in range(case["children"])]
        held = sum(_pages(n, page) for n in lens)
        entries = sum(_pages(n, page) for n in of)
        moved = sum(n % page for n in of)
        return dict(bytes=2 * moved * row + 12.0 * held + 8.0 * entries + 40.0 * len(of), flops=0.0)
    if op == "compact":
        held = [_pages(n, case["page"]) for n in _lengths(case["B"], case["lo"], case["hi"])]
        n_pages = _pool(case, sum(held))
        moves = min(case["most"], int(sum(held) * (1 - sum(held) / n_pages)))
        return dict(bytes=2.0 * moves * case["page"] * row + 8.0 * sum(held) + 16.0 * n_pages
                    + 12.0 * case["most"], flops=0.0)
    prefix, tails = _shared_sizes(case)
    per = case["G"] * case["T"]
    once = sum(prefix) + sum(tails)
    met = sum(prefix) * case["members"] + sum(tails)
    rows = len(tails) * case["K"] * per
    return dict(bytes=once * 2.0 * case["K"] * case["H"] * e + rows * (4.0 * case["H"] + 4.0)
                + 4.0 * once / case["page"] + 8.0 * len(tails),
                flops=4.0 * met * case["K"] * per * case["H"])


def _pool(case, held):
    return int(held / case["pool"]) + 8


# ------------------------------------------------------------------ inputs

def _cache(case, n_pages, gen, layers=0):
    """A cache, filled, as the view [layers,] [pages, kv heads, page size, head dim]."""
    shape = (n_pages, case["K"], case["page"], case["H"])
    if case["layout"] == "token":
        shape = (shape[0], shape[2], shape[1], shape[3])
    if layers:
        shape = (layers, *shape)
    c = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
    if case["dtype"] == "e4m3":     # values over their scale: N(0, 1) over 1/64 or so
        c = (c * 64).to(torch.float8_e4m3fn)
    return c.transpose(-3, -2) if case["layout"] == "token" else c


def _scale(case, gen):
    if case["dtype"] == "bf16":
        return None
    return (torch.rand(case["K"], generator=gen, device="cuda") + 0.5) / 64


def _positions(case, total, order):
    """[axes, total] positions: a stretch of text, or frames of height x width patches."""
    n = torch.arange(total, device="cuda")
    t = n % case["T"] if case["op"] == "rotary" else n
    if case["far"]:
        t = (t * 7919 + order.randrange(case["far"])) % case["far"]
    w = 1 + int(case["T"] ** 0.5 / 2)
    rows = [t, t // w % w + order.randrange(8), t % w, t // (w * w)]
    return torch.stack(rows[:case["axes"]]).to(torch.int32)


def _turning(case):
    """(frequencies, axis of each pair or None) of a model's configuration."""
    pairs = case["rot"] // 2
    i = torch.arange(pairs, device="cuda", dtype=torch.float64)
    freq = (BASE ** (-i / pairs)).float()
    if case["axes"] == 1:
        return freq, None
    j = torch.arange(pairs, device="cuda")
    axis = j % case["axes"] if case["mixed"] else j * case["axes"] // pairs
    return freq, axis.to(torch.int32)


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _table(held, perm, width):
    """Rows of page ids, the requests' `held` pages one after the other from perm."""
    j = torch.arange(width, device="cuda")[None]
    first = _ints([sum(held[:i]) for i in range(len(held))], torch.int64)[:, None]
    ids = perm[(first + j).clamp(max=len(perm) - 1)]
    return torch.where(j < _ints(held)[:, None], ids, -1).contiguous()


def _prepare_rotary(case, gen, order):
    B, T, K, G, H = (case[x] for x in "BTKGH")
    freq, axis = _turning(case)
    s = dict(case=case, freq=freq, axis=axis)
    if case["op"] == "rotary":
        pos = _positions(case, B * T, order).unflatten(1, (B, T))
        fused = torch.randn((B, T, (G + 2) * K, H), generator=gen, device="cuda")
        fused = fused.to(torch.bfloat16)
        laid = [torch.empty((B, n, T, H), dtype=torch.bfloat16, device="cuda").transpose(1, 2)
                for n in (K * G, K)]
        flat = [fused[:, :, :G * K], fused[:, :, G * K:(G + 1) * K]]
        if case["inverse"]:     # from the attention's layout to the projection's
            for x in laid:
                x.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
            flat, laid = laid, [torch.empty_like(x) for x in flat]
        s.update(positions=pos, q=flat[0], k=flat[1], q_out=laid[0], k_out=laid[1])
        return s
    total = B * T + case["pad"]
    page = case["page"]
    runs, run = (B, 1) if T < 16 else (B, T)
    per = _pages(run if T >= 16 else page, page) if T >= 16 else 1
    n_pages = (runs if T >= 16 else B * T) * per + 3
    perm = torch.randperm(n_pages, generator=gen, device="cuda")
    i = torch.arange(B * T, device="cuda")
    at = i % run if T >= 16 else i * 0 + order.randrange(page)
    slots = perm[(i // run) * per + at // page * (T >= 16)] * page + at % page
    pad = torch.full((case["pad"],), -1, dtype=torch.int64, device="cuda")
    heads = (G + 2) * K
    qkv = torch.randn((total, heads, H), generator=gen, device="cuda").to(torch.bfloat16)
    split = (1, total) if case["pad"] else (B, T)
    q_out = torch.zeros((split[0], K, G, split[1], H), dtype=torch.bfloat16, device="cuda")
    s.update(positions=_positions(case, total, order), slots=torch.cat([slots, pad]), page=page,
             q=qkv[:, :G * K], k=qkv[:, G * K:(G + 1) * K], v=qkv[:, (G + 1) * K:], q_out=q_out,
             k_cache=_cache(case, n_pages, gen), v_cache=_cache(case, n_pages, gen),
             k_scale=_scale(case, gen), v_scale=_scale(case, gen))
    return s


def _prepare_release(case, gen, order):
    both = list(zip(*_dropped(case)))
    order.shuffle(both)
    lens, keep = [a for a, _ in both], [b for _, b in both]
    page = case["page"]
    held = [_pages(n, page) for n in lens]
    n_pages = _pool(case, sum(held))
    perm = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    rows = list(range(case["B"]))
    order.shuffle(rows)
    used = sum(held)
    return dict(case=case, page=page, lens=_ints(lens), rows=_ints(rows),
                keep=_ints([keep[r] for r in rows]) if case["drop"] else None,
                block_table=_table(held, perm, max(held) + 2), free_pages=perm.clone(),
                shares=torch.zeros(n_pages, dtype=torch.int32, device="cuda"),
                free_used=_ints([used]), lens_out=torch.empty_like(_ints(lens)),
                free_used_out=_ints([0]))


def _prepare_turnover(case, gen, order):
    page, P, C = case["page"], case["parents"], case["children"]
    lens = _lengths(P, case["lo"], case["hi"])
    order.shuffle(lens)
    of = [i % P for i in range(C)]
    order.shuffle(of)
    held = [_pages(n, page) for n in lens] + [1 if lens[p] % page else 0 for p in of]
    n_pages = _pool(case, sum(held))
    perm = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    width = max(held) + 2
    table = _table(held, perm, width)
    full = _ints([lens[p] // page for p in of], torch.int64)[:, None]
    own_page = table[P:, :1]
    j = torch.arange(width, device="cuda")[None]
    up = table[_ints(of, torch.int64)]      # the children hold their parent's pages already
    table[P:] = torch.where(j < full, up, torch.where(j == full, own_page, -1))
    shares = torch.zeros(n_pages + 1, dtype=torch.int32, device="cuda")
    ids = torch.where(j < full, up, n_pages).flatten().long()
    shares.index_add_(0, ids, torch.ones_like(ids, dtype=torch.int32))
    return dict(case=case, page=page, parents=_ints(of), children=_ints(list(range(P, P + C))),
                lens=_ints(lens + [lens[p] for p in of]), block_table=table.contiguous(),
                shares=shares[:n_pages].clone(), free_pages=perm.clone(),
                free_used=_ints([sum(held)]), copies=torch.empty((C, 3), dtype=torch.int32, device="cuda"),
                k_cache=_cache(case, n_pages, gen, case["L"]), v_cache=_cache(case, n_pages, gen, case["L"]))


def _prepare_compact(case, gen, order):
    page = case["page"]
    lens = _lengths(case["B"], case["lo"], case["hi"])
    order.shuffle(lens)
    held = [_pages(n, page) for n in lens]
    n_pages = _pool(case, sum(held))
    perm = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    table = _table(held, perm, max(held) + 2)
    empty = lambda x: torch.zeros_like(x)                   # noqa: E731
    shares = torch.randint(0, 3, (n_pages,), generator=gen, device="cuda", dtype=torch.int32)
    shares[perm[sum(held):].long()] = 0
    return dict(case=case, page=page, lens=_ints(lens), block_table=table, shares=shares,
                free_pages=perm, free_used=_ints([sum(held)]), block_table_out=empty(table),
                shares_out=empty(shares), free_pages_out=empty(perm),
                moves=torch.empty((case["most"], 3), dtype=torch.int32, device="cuda"),
                k_cache=_cache(case, n_pages, gen, case["L"]), v_cache=_cache(case, n_pages, gen, case["L"]))


def _prepare_shared(case, gen, order):
    K, G, T, H, page, M = (case[x] for x in ("K", "G", "T", "H", "page", "members"))
    prefix, tails = _shared_sizes(case)
    B = len(tails)
    order.shuffle(tails)
    rows = list(range(B))
    order.shuffle(rows)                     # member i of the groups is request rows[i]
    group = [0] * B
    for i, b in enumerate(rows):
        group[b] = i // M
    lens = [prefix[group[b]] + tails[b] for b in range(B)]
    own_pages = [_pages(t, page) for t in tails]
    head = [p // page for p in prefix]
    n_pages = sum(own_pages) + sum(head) + 5
    perm = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    width = max(h + o for h, o in zip((head[g] for g in group), own_pages))
    first = [sum(head[:g]) for g in range(len(head))]
    at, table = sum(head), []
    j = torch.arange(width, device="cuda")
    for b in range(B):
        h, g = head[group[b]], group[b]
        i = torch.where(j < h, first[g] + j, at + j - h).clamp(max=n_pages - 1)
        table.append(torch.where(j < h + own_pages[b], perm[i], -1))
        at += own_pages[b]
    q = torch.randn((B, K, G, T, H), generator=gen, device="cuda") * H ** -0.5
    return dict(case=case, page=page, q=q.to(torch.bfloat16), k_cache=_cache(case, n_pages, gen),
                v_cache=_cache(case, n_pages, gen), k_scale=_scale(case, gen),
                v_scale=_scale(case, gen), block_table=torch.stack(table).contiguous(),
                lens=_ints(lens), members=_ints(rows),
                group_starts=_ints([i * M for i in range(len(prefix) + 1)]),
                prefix_lens=_ints(prefix),
                o=torch.empty((B, K, G, T, H), dtype=torch.bfloat16, device="cuda"),
                lse=torch.empty((B, K, G, T), device="cuda"),
                workspace=torch.empty(SCRATCH, dtype=torch.uint8, device="cuda"))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    order = random.Random(seed)
    return dict(rotary=_prepare_rotary, append=_prepare_rotary, release=_prepare_release,
                turnover=_prepare_turnover, compact=_prepare_compact,
                shared=_prepare_shared)[case["op"]](case, gen, order)


# -------------------------------------------------------------- plain forms

def _turned(x, angle, adjacent, scale):
    """x [..., heads, H] in 32 bits, its first 2 * pairs dims turned by angle [..., 1, pairs]."""
    x = x.float()
    pairs = angle.shape[-1]
    c, s = angle.cos().float(), angle.sin().float()
    head, rest = x[..., :2 * pairs], x[..., 2 * pairs:]
    a, b = ((head[..., 0::2], head[..., 1::2]) if adjacent
            else (head[..., :pairs], head[..., pairs:]))
    a, b = a * c - b * s, b * c + a * s
    head = torch.stack([a, b], -1).flatten(-2) if adjacent else torch.cat([a, b], -1)
    return torch.cat([head, rest], -1) * scale


def _angles(s):
    """[..., 1, pairs] in 64 bits, of positions [axes, ...]."""
    pos, freq = s["positions"].double(), s["freq"].double()
    at = pos[s["axis"].long()] if s["axis"] is not None else pos[0][None].expand(len(freq), *pos.shape[1:])
    return (at.movedim(0, -1) * freq)[..., None, :]


def _plain_rotary(s):
    c = s["case"]
    angle = -_angles(s) if c["inverse"] else _angles(s)
    s["q_out"].copy_(_turned(s["q"], angle, c["adjacent"], c["H"] ** -0.5))
    s["k_out"].copy_(_turned(s["k"], angle, c["adjacent"], 1.0))
    return dict(q=s["q_out"], k=s["k_out"])


def _plain_append(s):
    c = s["case"]
    angle = _angles(s)
    live = s["slots"] >= 0
    at = s["slots"][live]
    q = _turned(s["q"], angle, c["adjacent"], c["H"] ** -0.5).to(torch.bfloat16)
    out = s["q_out"].permute(0, 3, 1, 2, 4)                 # [B, T, K, G, H]
    keep = live.view(out.shape[:2])[..., None, None, None]
    out.copy_(torch.where(keep, q.view(out.shape), out))
    for x, cache, scale in ((_turned(s["k"], angle, c["adjacent"], 1.0), s["k_cache"], s["k_scale"]),
                            (s["v"].float(), s["v_cache"], s["v_scale"])):
        x = x[live]
        if scale is not None:
            x = (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
            x, cache = x.view(torch.uint8), cache.view(torch.uint8)
        else:
            x = x.to(torch.bfloat16)
        cache[at // s["page"], :, at % s["page"]] = x
    return dict(q=s["q_out"], k_cache=s["k_cache"], v_cache=s["v_cache"])


def _release(rows, keep, lens, table, shares, free, used, page):
    """(lens, used) after the rows keep their first tokens; shares and free are updated."""
    rows = rows.long()
    n, n_free = len(shares), len(free)
    held, kept = (lens[rows] + page - 1) // page, (keep + page - 1) // page
    j = torch.arange(table.shape[1], device=table.device)[None]
    gone = (j >= kept[:, None]) & (j < held[:, None])
    ids = torch.where(gone, table[rows], n).flatten().long()
    less = torch.zeros(n + 1, dtype=torch.int32, device=table.device)
    less.index_add_(0, ids, torch.ones_like(ids, dtype=torch.int32))
    left = shares - less[:n]
    out = (less[:n] > 0) & (left < 0)
    shares.copy_(left.masked_fill(out, 0))
    rank, total = out.cumsum(0) - 1, out.sum()
    full = torch.cat([free, free[:1]])
    full.index_copy_(0, torch.where(out, used.long() - total + rank, n_free),
                     torch.arange(n, device=free.device, dtype=torch.int32))
    free.copy_(full[:n_free])
    return lens.index_copy(0, rows, keep), (used - total).to(torch.int32)


def _plain_release(s):
    keep = s["keep"] if s["keep"] is not None else torch.zeros_like(s["rows"])
    lens, used = _release(s["rows"], keep, s["lens"], s["block_table"], s["shares"],
                          s["free_pages"], s["free_used"], s["page"])
    s["lens_out"].copy_(lens)
    s["free_used_out"].copy_(used)
    return _released(s)


def _released(s):
    return dict(lens=s["lens_out"], used=s["free_used_out"], free=s["free_pages"], shares=s["shares"])


def _plain_copy(moves, *caches):
    moves = moves[moves[:, 0] >= 0].long()
    src, dst, n = moves.unbind(1)
    for cache in caches:
        bits = cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache
        live = torch.arange(cache.shape[3], device=cache.device) < n[:, None]   # [moves, page]
        bits[:, dst] = torch.where(live[:, None, :, None], bits[:, src], bits[:, dst])


def _plain_turnover(s):
    page, table, shares = s["page"], s["block_table"], s["shares"]
    lens, used = _release(s["children"], torch.zeros_like(s["children"]), s["lens"], table, shares,
                          s["free_pages"], s["free_used"], page)
    up, to = s["parents"].long(), s["children"].long()
    n = lens[up]
    full, part = n // page, n % page
    j = torch.arange(table.shape[1], device=table.device)[None]
    ids = table[up]
    whole = j < full[:, None]
    add = torch.where(whole, ids, len(shares)).flatten().long()
    more = torch.zeros(len(shares) + 1, dtype=torch.int32, device=table.device)
    shares += more.index_add_(0, add, torch.ones_like(add, dtype=torch.int32))[:-1]
    need = (part > 0).long()
    fresh = s["free_pages"][used.long() + need.cumsum(0) - need]
    opened = (j == full[:, None]) & (part > 0)[:, None]
    table[to] = torch.where(whole, ids, torch.where(opened, fresh[:, None], table[to]))
    src = ids.gather(1, full[:, None].long())[:, 0]
    none = part == 0
    s["copies"].copy_(torch.stack([src.masked_fill(none, -1), fresh.masked_fill(none, -1), part], 1))
    s["lens"].copy_(lens.index_copy(0, to, n))
    s["free_used"].copy_(used + need.sum())
    _plain_copy(s["copies"], s["k_cache"], s["v_cache"])
    return _turned_over(s)


def _turned_over(s):
    return dict(block_table=s["block_table"], lens=s["lens"], shares=s["shares"], free=s["free_pages"],
                used=s["free_used"], copies=s["copies"], k_cache=s["k_cache"], v_cache=s["v_cache"])


def _plain_compact(s):
    table, shares, free, page = s["block_table"], s["shares"], s["free_pages"], s["page"]
    n, most = len(shares), len(s["moves"])
    ids = torch.arange(n, device=table.device, dtype=torch.int32)
    j = torch.arange(table.shape[1], device=table.device)[None]
    live = j < ((s["lens"] + page - 1) // page)[:, None]
    held = torch.zeros(n + 1, dtype=torch.bool, device=table.device)
    held[torch.where(live, table, n).long()] = True
    spare = torch.zeros_like(held)
    spare[torch.where(torch.arange(len(free), device=free.device) >= s["free_used"], free, n).long()] = True
    held, spare = held[:n], spare[:n]
    above = held.flip(0).cumsum(0).flip(0) - held.long()    # held pages behind this one
    below = spare.cumsum(0) - spare.long()                  # free ones before it
    goes = held & (below > above) & (above < most)
    takes = spare & (above > below) & (below < most)
    src, dst = (torch.full((most + 1,), -1, dtype=torch.int32, device=table.device) for _ in range(2))
    src[torch.where(goes, above, most)] = ids
    dst[torch.where(takes, below, most)] = ids
    src, dst = src[:most], dst[:most]
    tokens = torch.where(src >= 0, page, 0).to(torch.int32)
    s["moves"].copy_(torch.stack([src, dst, tokens], 1))
    to = torch.where(goes, dst[above.clamp(max=most - 1)], ids)
    s["block_table_out"].copy_(torch.where(live, to[table.clamp(min=0).long()], table))
    back = src[below.clamp(max=most - 1)].clamp(min=0).long()
    s["shares_out"].copy_(torch.where(takes, shares[back], shares.masked_fill(goes, 0)))
    now = spare & ~takes | goes
    at = torch.where(now, s["free_used"] + now.cumsum(0) - 1, len(free))
    out = torch.cat([s["free_pages_out"], free[:1]])
    out[at] = ids
    s["free_pages_out"].copy_(out[:len(free)])
    _plain_copy(s["moves"], s["k_cache"], s["v_cache"])
    return _compacted(s)


def _compacted(s):
    return dict(block_table=s["block_table_out"], shares=s["shares_out"], free=s["free_pages_out"],
                moves=s["moves"], k_cache=s["k_cache"], v_cache=s["v_cache"])


def _gathered(cache, scale, table):
    """A request's keys in order, [B, K, columns * page size, H] in 32 bits."""
    bits = cache.view(torch.uint8) if scale is not None else cache
    x = bits[table.long().clamp(min=0)]                     # [B, columns, K, page, H]
    x = x.view(torch.float8_e4m3fn).float() * scale[:, None, None] if scale is not None else x.float()
    return x.transpose(1, 2).flatten(2, 3)


def _plain_shared(s):
    B, K, G, T, H = s["q"].shape
    q = s["q"].float().flatten(2, 3)
    k = _gathered(s["k_cache"], s["k_scale"], s["block_table"])
    x = q @ k.transpose(-1, -2)                             # [B, K, G * T, keys]
    del k
    key = torch.arange(x.shape[-1], device=x.device)
    last = (s["lens"].long()[:, None] - T + torch.arange(T, device=x.device))[:, :, None]
    keep = (key <= last)[:, None, None].expand(B, K, G, T, -1).flatten(2, 3)
    x = x.masked_fill(~keep, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = (x - top.masked_fill(top == -math.inf, 0)).exp()
    del x, keep
    total = p.sum(-1, keepdim=True)
    v = _gathered(s["v_cache"], s["v_scale"], s["block_table"])
    o = p @ v / total.masked_fill(total == 0, 1)
    lse = (top + total.log()).squeeze(-1)
    return dict(o=o.to(torch.bfloat16).unflatten(2, (G, T)), lse=lse.unflatten(2, (G, T)))


def run(s):
    op = s["case"]["op"]
    if own:
        from flash_attention_gqa_gb300 import binding
        c = s["case"]
        if op == "rotary":
            binding.fa_rotary(s["q"], s["q_out"], s["k"], s["k_out"], s["positions"], s["freq"],
                              s["axis"], q_scale=c["H"] ** -0.5, adjacent=c["adjacent"],
                              inverse=c["inverse"])
            return dict(q=s["q_out"], k=s["k_out"])
        if op == "append":
            binding.fa_paged_rotary_append(
                s["q"], s["k"], s["v"], s["positions"], s["freq"], s["slots"], s["q_out"],
                s["k_cache"], s["v_cache"], s["axis"], s["k_scale"], s["v_scale"],
                q_scale=c["H"] ** -0.5, adjacent=c["adjacent"])
            return dict(q=s["q_out"], k_cache=s["k_cache"], v_cache=s["v_cache"])
        if op == "release":
            binding.fa_paged_free(s["rows"], s["lens"], s["block_table"], s["shares"],
                                  s["free_pages"], s["free_used"], s["lens_out"],
                                  s["free_used_out"], s["page"], s["keep"])
            return _released(s)
        if op == "turnover":
            binding.fa_paged_free(s["children"], s["lens"], s["block_table"], s["shares"],
                                  s["free_pages"], s["free_used"], s["lens"], s["free_used"],
                                  s["page"])
            binding.fa_paged_fork(s["parents"], s["children"], s["lens"], s["block_table"],
                                  s["shares"], s["free_pages"], s["free_used"], s["lens"],
                                  s["copies"], s["free_used"], s["page"])
            binding.fa_paged_copy(s["copies"], s["k_cache"], s["v_cache"])
            return _turned_over(s)
        if op == "compact":
            binding.fa_paged_compact(s["lens"], s["block_table"], s["shares"], s["free_pages"],
                                     s["free_used"], s["block_table_out"], s["shares_out"],
                                     s["free_pages_out"], s["moves"], s["page"])
            binding.fa_paged_copy(s["moves"], s["k_cache"], s["v_cache"])
            return _compacted(s)
        binding.fa_paged_decode_shared(s["q"], s["k_cache"], s["v_cache"], s["block_table"],
                                       s["lens"], s["members"], s["group_starts"],
                                       s["prefix_lens"], s["o"], s["lse"], s["workspace"],
                                       s["k_scale"], s["v_scale"])
        return dict(o=s["o"], lse=s["lse"])
    return dict(rotary=_plain_rotary, append=_plain_append, release=_plain_release,
                turnover=_plain_turnover, compact=_plain_compact, shared=_plain_shared)[op](s)


# --------------------------------------------------------------- definition

def _spun(x, pos, freq, axis, adjacent, sign):
    """x [..., heads, H] as complex numbers times exp(i angle), pair by pair, in 64 bits."""
    out = x.double().clone()
    pairs = len(freq)
    for i in range(pairs):
        angle = sign * pos[0 if axis is None else int(axis[i])].double() * freq[i].double()
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + pairs)
        z = torch.complex(out[..., a], out[..., b]) * torch.polar(torch.ones_like(angle), angle)[..., None]
        out[..., a], out[..., b] = z.real, z.imag
    return out


def exact(case, seed):
    """The definition in 64 bits, pair by pair and request by request."""
    if case["op"] in ("release", "turnover", "compact"):
        return None                                         # whole numbers, and values only moved
    s = prepare(case, seed)
    if case["op"] in ("rotary", "append"):
        sign = -1.0 if case.get("inverse") else 1.0
        axis = None if s["axis"] is None else s["axis"].tolist()
        q, k = (_spun(s[n], s["positions"], s["freq"], axis, case["adjacent"], sign) for n in "qk")
        q = q * case["H"] ** -0.5
        if case["op"] == "rotary":
            return dict(q=q, k=k)
        n, page = case["B"] * case["T"], case["page"]
        out = dict(q=s["q_out"].double())
        B, K, G, T, H = out["q"].shape
        rows = q.reshape(B, T, K, G, H).permute(0, 2, 3, 1, 4)
        if case["pad"]:
            out["q"][:, :, :, :n] = rows[:, :, :, :n]
        else:
            out["q"] = rows
        for name, x in (("k", k), ("v", s["v"].double())):
            scale, cache = s[name + "_scale"], s[name + "_cache"].double()
            flat = cache.transpose(1, 2).reshape(-1, K, H)  # by slot
            if scale is not None:
                x = torch.clip(x / scale.double().reshape(1, -1, 1), -E4M3_MAX, E4M3_MAX)
            flat.index_copy_(0, s["slots"][:n], x[:n])
            out[name + "_cache"] = flat.unflatten(0, (-1, page)).transpose(1, 2)
        return out
    B, K, G, T, H = s["q"].shape
    page = case["page"]
    o = torch.zeros((B, K, G, T, H), dtype=torch.float64, device="cuda")
    lse = torch.full((B, K, G, T), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        ids = s["block_table"][b, :_pages(n, page)].long()

        def rows(cache, scale):                             # [K, n, H]
            x = (cache.view(torch.uint8)[ids].view(cache.dtype) if scale is not None
                 else cache[ids]).double()
            x = x.permute(1, 0, 2, 3).reshape(K, -1, H)[:, :n]
            return x if scale is None else x * scale.double().reshape(K, 1, 1)

        k, v = rows(s["k_cache"], s["k_scale"]), rows(s["v_cache"], s["v_scale"])
        for t in range(T):
            hi = n - T + t + 1
            x = torch.einsum("kgh,ksh->kgs", s["q"][b, :, :, t].double(), k[:, :hi])
            lse[b, :, :, t] = torch.logsumexp(x, -1)
            o[b, :, :, t] = torch.einsum("kgs,ksh->kgh", torch.softmax(x, -1), v[:, :hi])
    return dict(o=o, lse=lse)
