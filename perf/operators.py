"""The paged key-value cache operators, as cases to measure.

Three operators that a serving program runs in turn, once per step:
  tables   block table, slot map and positions from the requests' lengths
  append   the step's new keys and values written into the cache's pages
  decode   attention of the requests' newest tokens over their pages

``run`` computes them in a plain form (elementary torch operations in 32 bits);
with ``own`` set it calls the library.  ``exact`` is the definition in 64 bits.
Caches are [pages, kv heads, page size, head dim], read through their strides:
"head" layouts store them in that order, "token" layouts with the page's tokens
outside the heads.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
GOLDEN = 0.6180339887498949
SCRATCH = 64 << 20      # the workspace that a serving program sets aside at its start


def listed():
    return [
        # One decode step of 64 running requests: a token each, some of which open a page.
        dict(name="tables_step", op="tables", B=64, lo=1, hi=16384, new_lo=1, new_hi=1, page=16,
             pad=0),
        # A batch of prompts, with what is cached of their prefixes, into a padded token buffer.
        dict(name="tables_prompts", op="tables", B=128, lo=1, hi=2048, new_lo=16, new_hi=4096,
             page=16, pad=333),
        # The keys and values of one decode step: 64 tokens, each into a page of its own.
        dict(name="append_step", op="append", N=64, pad=0, run=1, K=8, H=128, page=16,
             dtype="bf16", layout="token", fused=False),
        # The keys and values of 16 prompts of 1000 tokens, views of a fused projection's output.
        dict(name="append_prompts", op="append", N=16000, pad=384, run=1000, K=8, H=128, page=64,
             dtype="bf16", layout="head", fused=True),
        # The same into an 8-bit cache, at head dim 256.
        dict(name="append_prompts_e4m3", op="append", N=7001, pad=7, run=777, K=2, H=256, page=32,
             dtype="e4m3", layout="head", fused=True),
        # One request, a thousand tokens in: latency.
        dict(name="decode_one", op="decode", B=1, K=2, G=8, T=1, H=256, lo=1000, hi=1000, page=16,
             dtype="bf16", layout="head", window=0),
        # One decode step against 32768 keys, the shape of the dense decode workload.
        dict(name="decode_b8_s32768", op="decode", B=8, K=8, G=8, T=1, H=128, lo=32768, hi=32768,
             page=64, dtype="bf16", layout="head", window=0),
        # Continuous batching: 64 requests from one token to 16384, pages of 16 tokens.
        dict(name="decode_ragged", op="decode", B=64, K=8, G=4, T=1, H=128, lo=1, hi=16384,
             page=16, dtype="bf16", layout="token", window=0),
        # A large batch on an 8-bit cache.
        dict(name="decode_e4m3", op="decode", B=128, K=8, G=8, T=1, H=128, lo=256, hi=8192,
             page=32, dtype="e4m3", layout="head", window=0),
        # Verification of drafted tokens: four new tokens a request, causal among themselves.
        dict(name="decode_verify", op="decode", B=16, K=4, G=8, T=4, H=128, lo=512, hi=8192,
             page=64, dtype="bf16", layout="head", window=0),
        # One request with a long context: the split over the cache's length carries it.
        dict(name="decode_long", op="decode", B=1, K=2, G=8, T=1, H=256, lo=131072, hi=131072,
             page=128, dtype="bf16", layout="head", window=0),
        # A layer with a sliding window, one query head per kv head, head dim 64.
        dict(name="decode_window", op="decode", B=32, K=16, G=1, T=1, H=64, lo=100, hi=8192,
             page=16, dtype="bf16", layout="token", window=1024),
    ]


def draw(rng):
    """A case of the same ranges: logarithmic sizes, odd ones among them."""
    def log(lo, hi):
        return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))

    op = rng.choice(["tables", "append", "decode", "decode", "decode"])
    page = 1 << rng.randrange(3, 9)
    if op == "tables":
        new_hi = rng.choice([1, log(2, 4096)])
        B = log(1, 512)
        while B * new_hi > 262144:
            B = max(1, B // 2)
        return dict(op=op, B=B, lo=1, hi=log(1, 16384), new_lo=1 if new_hi < 64 else 16,
                    new_hi=new_hi, page=page, pad=rng.randrange(0, 300))
    K, H = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([64, 128, 256])
    dtype, layout = rng.choice(["bf16", "bf16", "e4m3"]), rng.choice(["head", "token"])
    if op == "append":
        N = log(1, 16384)
        while N * K * H > 16384 * 1024:
            N //= 2
        return dict(op=op, N=N, pad=rng.randrange(0, 64), run=log(1, N), K=K, H=H, page=page,
                    dtype=dtype, layout=layout, fused=rng.random() < 0.5)
    T = rng.choice([1, 1, 1, rng.randrange(2, 9)])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    B, hi = log(1, 128), log(1, 131072)
    while B * hi * K * H > 8 * 32768 * 1024 or B * K * G * T * hi > 1 << 28:
        B, hi = (B // 2, hi) if B > 1 else (B, hi // 2)
    return dict(op=op, B=B, K=K, G=G, T=T, H=H, lo=rng.choice([1, hi]), hi=hi, page=page,
                dtype=dtype, layout=layout,
                window=rng.choice([0, 0, log(1, 4096)]))


# ------------------------------------------------------------------- sizes

def _lengths(n, lo, hi, phase=0.0):
    """n lengths spread over [lo, hi] by their logarithm: the case's, whatever the seed."""
    return [max(lo, min(hi, int(round(lo * (hi / lo) ** (((i + 0.5) * GOLDEN + phase) % 1.0)))))
            for i in range(n)]


def _pages(n, page):
    return -(-n // page)


def _seen(case):
    """(request, keys that its newest tokens attend to in all) sizes of a decode case."""
    w, T = case["window"], case["T"]
    lens = _lengths(case["B"], case["lo"], case["hi"])
    return [n if w == 0 else min(n, w + T - 1) for n in lens], lens


def work(case):
    if case["op"] == "tables":
        c = _lengths(case["B"], case["lo"], case["hi"])
        n = _lengths(case["B"], case["new_lo"], case["new_hi"], 0.37)
        N = sum(n)
        opened = sum(_pages(a + b, case["page"]) - _pages(a, case["page"]) for a, b in zip(c, n))
        # lengths and free pages read; table entries, lengths, starts, slots and positions written
        return dict(bytes=16.0 * case["B"] + 8.0 * opened + 12.0 * (N + case["pad"]), flops=0.0)
    e = 2 if case["dtype"] == "bf16" else 1
    if case["op"] == "append":
        values = 2.0 * case["N"] * case["K"] * case["H"]
        return dict(bytes=values * (2 + e) + 8.0 * (case["N"] + case["pad"]),
                    flops=0.0 if e == 2 else 2.0 * values)
    seen, lens = _seen(case)
    rows = case["B"] * case["K"] * case["G"] * case["T"]
    pairs = float(sum(seen)) * case["K"] * case["G"] * case["T"]
    cache = 2.0 * sum(seen) * case["K"] * case["H"] * e
    table = 4.0 * sum(_pages(n, case["page"]) for n in seen) + 4.0 * case["B"]
    return dict(bytes=cache + table + rows * (4.0 * case["H"] + 4.0), flops=4.0 * pairs * case["H"])


# ------------------------------------------------------------------ inputs

def _cache(case, n_pages, gen, seed):
    """One of the two caches, filled, as the view [pages, kv heads, page size, head dim]."""
    shape = (n_pages, case["K"], case["page"], case["H"])
    if case["layout"] == "token":
        shape = (shape[0], shape[2], shape[1], shape[3])
    if case["dtype"] == "bf16":
        c = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
    else:   # values over their scale: N(0, 1) over 1/64 or so
        c = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
        c = (c * 64).to(torch.float8_e4m3fn)
    return c.transpose(1, 2) if case["layout"] == "token" else c


def _scale(case, gen):
    if case["dtype"] == "bf16":
        return None
    return (torch.rand(case["K"], generator=gen, device="cuda") + 0.5) / 64


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    order = random.Random(seed)
    page = case["page"]
    s = dict(case=case)

    def ints(values, dtype=torch.int32):
        return torch.tensor(values, dtype=dtype, device="cuda")

    def empty(n, dtype=torch.int32):
        return torch.empty(n, dtype=dtype, device="cuda")

    if case["op"] == "tables":
        both = list(zip(_lengths(case["B"], case["lo"], case["hi"]),
                        _lengths(case["B"], case["new_lo"], case["new_hi"], 0.37)))
        order.shuffle(both)
        cached, new = [a for a, _ in both], [b for _, b in both]
        held = [_pages(a, page) for a in cached]
        opened = sum(_pages(a + b, page) - h for (a, b), h in zip(both, held))
        n_pages = sum(held) + opened + 100
        perm = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
        width = max(_pages(a + b, page) for a, b in both) + 3
        j = torch.arange(width, device="cuda")[None]
        first = ints([sum(held[:i]) for i in range(len(held))], torch.int64)[:, None]
        table = torch.where(j < ints(held)[:, None], perm[(first + j).clamp(max=n_pages - 1)], -1)
        tokens = sum(new) + case["pad"]
        s.update(cached_lens=ints(cached), new_lens=ints(new), n_pages=n_pages, page=page,
                 free_pages=perm[sum(held):].contiguous(), free_used=ints([order.randrange(50)]),
                 block_table=table.contiguous(), tokens=tokens, n_new=sum(new),
                 total_lens=empty(case["B"]), token_starts=empty(case["B"] + 1),
                 slots=empty(tokens, torch.int64), positions=empty(tokens),
                 free_used_out=empty(1))
        return s
    if case["op"] == "append":
        N, K, H, run = case["N"], case["K"], case["H"], case["run"]
        total = N + case["pad"]
        per = _pages(run, page)
        n_pages = (_pages(N, run)) * per + 3
        perm = torch.randperm(n_pages, generator=gen, device="cuda")
        i = torch.arange(N, device="cuda")
        at = i % run + (order.randrange(page) if run == 1 else 0)
        slots = perm[(i // run) * per + (i % run) // page] * page + at % page
        pad = torch.full((case["pad"],), -1, dtype=torch.int64, device="cuda")
        heads = 4 * K if case["fused"] else 2 * K       # queries beside them, or not
        kv = torch.randn((total, heads, H), generator=gen, device="cuda").to(torch.bfloat16)
        s.update(k=kv[:, heads - 2 * K:heads - K], v=kv[:, heads - K:],
                 slots=torch.cat([slots, pad]), k_cache=_cache(case, n_pages, gen, seed),
                 v_cache=_cache(case, n_pages, gen, seed), k_scale=_scale(case, gen),
                 v_scale=_scale(case, gen), page=page)
        return s
    B, K, G, T, H = (case[x] for x in "BKGTH")
    lens = _lengths(B, case["lo"], case["hi"])
    order.shuffle(lens)
    held = [_pages(n, page) for n in lens]
    n_pages = sum(held) + 5
    perm = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    j = torch.arange(max(held), device="cuda")[None]
    first = ints([sum(held[:i]) for i in range(B)], torch.int64)[:, None]
    table = torch.where(j < ints(held)[:, None], perm[(first + j).clamp(max=n_pages - 1)], -1)
    q = torch.randn((B, K, G, T, H), generator=gen, device="cuda") * H ** -0.5
    s.update(q=q.to(torch.bfloat16), k_cache=_cache(case, n_pages, gen, seed),
             v_cache=_cache(case, n_pages, gen, seed), k_scale=_scale(case, gen),
             v_scale=_scale(case, gen), block_table=table.contiguous(), lens=ints(lens),
             window=case["window"], page=page,
             o=torch.empty((B, K, G, T, H), dtype=torch.bfloat16, device="cuda"),
             lse=torch.empty((B, K, G, T), device="cuda"),
             workspace=torch.empty(SCRATCH, dtype=torch.uint8, device="cuda"))
    return s


# -------------------------------------------------------------- plain forms

def _plain_tables(s):
    c, n, page = s["cached_lens"].long(), s["new_lens"].long(), s["page"]
    total = c + n
    held = (c + page - 1) // page
    opened = (total + page - 1) // page - held
    starts = torch.cat([n.new_zeros(1), n.cumsum(0)])
    taken = s["free_used"].long() + opened.cumsum(0) - opened
    b = torch.repeat_interleave(torch.arange(len(n), device=n.device), n, output_size=s["n_new"])
    pos = c[b] + torch.arange(s["n_new"], device=n.device) - starts[b]
    col = pos // page
    fresh = s["free_pages"].long()[(taken[b] + col - held[b]).clamp(min=0)]
    ids = torch.where(col >= held[b], fresh, s["block_table"].long()[b, col])
    s["block_table"][b, col] = ids.int()
    pad = ids.new_full((s["tokens"] - s["n_new"],), -1)
    return dict(block_table=s["block_table"], total_lens=total.int(), token_starts=starts.int(),
                slots=torch.cat([ids * page + pos % page, pad]),
                positions=torch.cat([pos, pad]).int(),
                free_used=(s["free_used"] + opened.sum()).int())


def _plain_append(s):
    live = s["slots"] >= 0
    at = s["slots"][live]
    for x, cache, scale in ((s["k"], s["k_cache"], s["k_scale"]),
                            (s["v"], s["v_cache"], s["v_scale"])):
        x = x[live]
        if scale is not None:
            x = (x.float() / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
            x, cache = x.view(torch.uint8), cache.view(torch.uint8)
        cache[at // s["page"], :, at % s["page"]] = x
    return dict(k_cache=s["k_cache"], v_cache=s["v_cache"])


def _gathered(cache, scale, table):
    """A request's keys in order, [B, K, columns * page size, H] in 32 bits."""
    bits = cache.view(torch.uint8) if scale is not None else cache
    x = bits[table.long().clamp(min=0)]                     # [B, columns, K, page, H]
    x = x.view(torch.float8_e4m3fn).float() * scale[:, None, None] if scale is not None else x.float()
    return x.transpose(1, 2).flatten(2, 3)


def _plain_decode(s):
    B, K, G, T, H = s["q"].shape
    q = s["q"].float().flatten(2, 3)
    k = _gathered(s["k_cache"], s["k_scale"], s["block_table"])
    x = q @ k.transpose(-1, -2)                             # [B, K, G * T, keys]
    del k
    key = torch.arange(x.shape[-1], device=x.device)
    last = (s["lens"].long()[:, None] - T + torch.arange(T, device=x.device))[:, :, None]
    keep = key <= last                                      # [B, T, keys]
    if s["window"]:
        keep &= key > last - s["window"]
    keep = keep[:, None, None].expand(B, K, G, T, -1).flatten(2, 3)
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
        if op == "tables":
            binding.fa_paged_tables(
                s["cached_lens"], s["new_lens"], s["free_pages"], s["free_used"],
                s["block_table"], s["total_lens"], s["token_starts"], s["slots"], s["positions"],
                s["free_used_out"], s["n_pages"], s["page"])
            return dict(block_table=s["block_table"], total_lens=s["total_lens"],
                        token_starts=s["token_starts"], slots=s["slots"],
                        positions=s["positions"], free_used=s["free_used_out"])
        if op == "append":
            binding.fa_paged_append(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"],
                                    s["k_scale"], s["v_scale"])
            return dict(k_cache=s["k_cache"], v_cache=s["v_cache"])
        binding.fa_paged_decode(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["lens"],
                                s["o"], s["lse"], s["workspace"], s["k_scale"], s["v_scale"],
                                s["window"])
        return dict(o=s["o"], lse=s["lse"])
    return {"tables": _plain_tables, "append": _plain_append, "decode": _plain_decode}[op](s)


# --------------------------------------------------------------- definition

def exact(case, seed):
    """The definition in 64 bits, request by request and token by token group."""
    if case["op"] == "tables":
        return None                                         # whole numbers only
    s = prepare(case, seed)
    page = case["page"]
    if case["op"] == "append":
        out = {}
        for name in ("k", "v"):
            scale, cache = s[name + "_scale"], s[name + "_cache"].double()
            flat = cache.transpose(1, 2).reshape(-1, case["K"], case["H"])      # by slot
            x = s[name].double()
            if scale is not None:
                x = torch.clip(x / scale.double().reshape(1, -1, 1), -E4M3_MAX, E4M3_MAX)
            flat.index_copy_(0, s["slots"][:case["N"]], x[:case["N"]])
            out[name + "_cache"] = flat.unflatten(0, (-1, page)).transpose(1, 2)
        return out
    B, K, G, T, H = (case[x] for x in "BKGTH")
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
            lo = max(0, hi - case["window"]) if case["window"] else 0
            if hi <= 0:
                continue
            x = torch.einsum("kgh,ksh->kgs", s["q"][b, :, :, t].double(), k[:, lo:hi])
            lse[b, :, :, t] = torch.logsumexp(x, -1)
            o[b, :, :, t] = torch.einsum("kgs,ksh->kgh", torch.softmax(x, -1), v[:, lo:hi])
    return dict(o=o, lse=lse)
