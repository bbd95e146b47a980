"""Performance cases of the 4-bit cache's operators and of the page operators.

    store    pa_kv4_append, then pa_kv4_gather: the new K and V rows of a batch of
             sequences quantised into the paged 4-bit pool, and read back
    decode   pa_kv4_decode: one new token per sequence against the 4-bit pool
    prefill  pa_kv4_prefill: prompt chunks against the 4-bit pool
    fork     pa_pages_fork: sequences continued from a copy of another one's
             pages (shared, but for a part-filled last page, which is copied)
    compact  pa_pages_compact: the pages that the window has left are given up
             and the pages in use moved together at the pool's front

The 4-bit pool is uint8 [pages][kv heads][4736]: per (page, kv head) the K codes
of 16 tokens (2048 bytes: token r's 256 codes are 8 pieces of 16 bytes, dims 32 i
.. 32 i + 31 in piece i ^ (r % 8) of its 128 bytes, the lower dim in the lower
half of a byte), the V codes (2048), 16 K block scales for each token (256), V's
(256), the 16 tokens' K row scales (64) and V's (64).  A value is code (e2m1) x
block scale (e4m3, 16 dims) x row scale (fp32).

Each case is a dict of plain values.  ``run`` computes an operator in its plain
form, elementary torch operations in 32 bits, or, where ``own`` is true, by the
calls a user makes of this package.
"""
import math

import numpy as np
import torch

own = False

D, PAGE, TILE = 256, 16, 4736


def listed():
    return [
        # the step of 64 chats: one new token each, latency is all there is
        dict(name="store 64 x 1", op="store", seqs=64, new_lo=1, new_hi=1, ctx_lo=500, ctx_hi=8000, hq=16, hkv=2,
             fused=True),
        # four sequences storing 2048-token prompt chunks: bound by memory
        dict(name="store 4 x 2048", op="store", seqs=4, new_lo=2048, new_hi=2048, ctx_lo=1000, ctx_hi=30000, hq=16,
             hkv=2, fused=True),
        # short ragged prompts, as many kv heads as query heads
        dict(name="store 13 ragged", op="store", seqs=13, new_lo=3, new_hi=1501, ctx_lo=0, ctx_hi=700, hq=8, hkv=8,
             fused=False),
        # one chat at a short context: latency
        dict(name="decode 1 x 1000", op="decode", seqs=1, ctx_lo=1000, ctx_hi=1000, hq=16, hkv=2, sink=1, win=0),
        # a serving batch of long contexts behind the sliding window
        dict(name="decode 64 windowed", op="decode", seqs=64, ctx_lo=4500, ctx_hi=8192, hq=16, hkv=2, sink=1, win=256),
        # few very long contexts, one kv head, window off: the work of a row split over the whole GPU
        dict(name="decode 5 x 200000", op="decode", seqs=5, ctx_lo=120001, ctx_hi=200003, hq=8, hkv=1, sink=0, win=0),
        # a short follow-up question after a cached conversation, two sequences
        dict(name="prefill 2 x 150", op="prefill", seqs=2, new_lo=37, new_hi=150, ctx_lo=900, ctx_hi=2100, hq=16, hkv=2,
             sink=1, win=0),
        # chunks of long prompts behind the sliding window: bound by the tensor cores
        dict(name="prefill 2 x 4096 windowed", op="prefill", seqs=2, new_lo=4096, new_hi=4096, ctx_lo=8192, ctx_hi=12005,
             hq=16, hkv=2, sink=1, win=256),
        # eight answers sampled for one question, one layer's int8 pool
        dict(name="fork 8 x 1000", op="fork", pool="int8", layers=1, forks=8, ctx_lo=1000, ctx_hi=1000, hkv=2),
        # many sequences forked at once, the 4-bit pools of 24 layers
        dict(name="fork 200 ragged", op="fork", pool="kv4", layers=24, forks=200, ctx_lo=17, ctx_hi=6000, hkv=2),
        # a few sequences leave: one layer's int8 pool, window off
        dict(name="compact 5 x 2000", op="compact", pool="int8", layers=1, seqs=5, shared=0, ctx_lo=300, ctx_hi=2000,
             hkv=2, sink=1, win=0, moved=0.5),
        # long contexts behind the window: most of their pages are given up, the 4-bit pools of 8 layers
        dict(name="compact 48 windowed", op="compact", pool="kv4", layers=8, seqs=48, shared=64, ctx_lo=3000,
             ctx_hi=6000, hkv=2, sink=1, win=128, moved=0.6),
    ]


#: A drawn case's cost (bytes, or flops / 300) stays under the largest listed one's.
_MOST = 5.0e8


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(("store", "decode", "prefill", "fork", "compact"))
        hq, hkv = rng.choice(((16, 2), (8, 4), (4, 1), (8, 8), (8, 1), (8, 2), (5, 5)))
        c = dict(op=op, hkv=hkv)
        if op == "store":
            c.update(seqs=_log_int(rng, 1, 300), hq=hq, fused=rng.random() < 0.5)
            c["new_hi"] = _log_int(rng, 1, max(1, 12000 // c["seqs"]))
            c["new_lo"] = rng.randint(1, c["new_hi"])
            c["ctx_lo"] = rng.randint(0, 50)
            c["ctx_hi"] = c["ctx_lo"] + _log_int(rng, 1, 4000)
        elif op == "decode":
            c.update(seqs=_log_int(rng, 1, 200), hq=hq, sink=rng.choice((0, 1, 4)), win=rng.choice((0, 0, 0, 64, 256)))
            c["ctx_hi"] = _log_int(rng, 1, min(200000, 1000000 // (c["seqs"] * hkv)))
            c["ctx_lo"] = rng.randint(1, c["ctx_hi"])
        elif op == "prefill":
            if hq == hkv and rng.random() < 0.5:
                c["hkv"], hq = 2, 32
            if hkv == 5:
                hq = 10
            c.update(seqs=_log_int(rng, 1, 8), hq=hq, sink=rng.choice((0, 1, 4)), win=rng.choice((0, 0, 64, 256)))
            c["new_hi"] = _log_int(rng, 1, 4096)
            c["new_lo"] = rng.randint(1, c["new_hi"])
            c["ctx_lo"] = rng.randint(0, 100)
            c["ctx_hi"] = c["ctx_lo"] + _log_int(rng, 1, 16000)
        else:
            c.update(pool=rng.choice(("int8", "kv4")), layers=rng.choice((1, 1, 2, 8)))
            if c["pool"] == "kv4" and rng.random() < 0.3:
                c["layers"] = 24
            n = _log_int(rng, 1, 250)
            if op == "fork":
                c.update(forks=n)
                c["ctx_hi"] = _log_int(rng, 1, 6000)
                c["ctx_lo"] = rng.randint(1, c["ctx_hi"])
            else:
                c.update(seqs=n, sink=rng.choice((0, 1, 4)), win=rng.choice((0, 16, 64, 128)), moved=rng.random())
                c["ctx_hi"] = _log_int(rng, 1, max(1, min(20000, 200000 // n)))
                c["ctx_lo"] = rng.randint(1, c["ctx_hi"])
                c["shared"] = rng.choice((0, c["ctx_lo"] // PAGE))
        if op in ("fork", "compact") and _pool_bytes(c) > 2.5e9:
            continue
        w = work(c)
        if max(w["bytes"], w["flops"] / 300) <= _MOST:
            return c


# ---------------------------------------------------------------- sizes
def _spread(lo, hi, n, step):
    """n whole numbers over [lo, hi] in a mixed order, both ends among them where n > 1."""
    i = (np.arange(n, dtype=np.int64) * step) % n
    return (hi - i * (hi - lo) // max(1, n - 1)).astype(np.int64)


def _lengths(case):
    """Per sequence (cached tokens, new tokens)."""
    n = case.get("seqs", case.get("forks"))
    ctx = _spread(case["ctx_lo"], case["ctx_hi"], n, 104729)
    if case["op"] in ("store", "prefill"):
        return ctx, _spread(case["new_lo"], case["new_hi"], n, 7919)
    return ctx, np.zeros(n, np.int64)


def _pages(tokens):
    return (tokens + PAGE - 1) // PAGE


def _page_bytes(case):
    return PAGE * case["hkv"] * 2 * (D + 4) if case["pool"] == "int8" else case["hkv"] * TILE


def _visible(t, sink, win):
    """Of queries at positions t: visible sink blocks, the window's first block, visible keys."""
    lo = np.maximum(0, t // PAGE + 1 - win) if win > 0 else np.zeros_like(t)
    n_sink = np.minimum(sink, lo)
    return n_sink, lo, PAGE * n_sink + t + 1 - PAGE * lo


def _compact_counts(case):
    """(entries of the table, those in use, pages in use, pages that move, pages of the pool)."""
    ctx, _ = _lengths(case)
    blocks = _pages(ctx)
    lo = np.maximum(0, ctx // PAGE + 1 - case["win"]) if case["win"] > 0 else np.zeros_like(ctx)
    given_up = np.maximum(0, np.minimum(lo, blocks) - case["sink"])
    entries, used = int(blocks.sum()), int((blocks - given_up).sum())
    # of the shared first blocks, one page each, in use if a sequence still sees it
    sh = case["shared"]
    b = np.arange(sh)[:, None]
    seen = ((b < case["sink"]) | (b >= lo[None, :])) & (b < blocks[None, :])
    live = used - int(seen.sum()) + int(seen.any(1).sum())
    dead = sh - int(seen.any(1).sum()) + int(given_up.sum()) - int((~seen & (b < blocks[None, :])).sum())
    n_pool = live + dead + 7 + live // 3
    return entries, used, live, int(case["moved"] * min(live, n_pool - live)), n_pool


def _pool_bytes(case):
    if case["op"] == "fork":
        ctx, _ = _lengths(case)
        return case["layers"] * (int(_pages(ctx).sum()) + case["forks"]) * _page_bytes(case)
    return case["layers"] * _compact_counts(case)[4] * _page_bytes(case)


def work(case):
    op, hkv = case["op"], case["hkv"]
    ctx, new = _lengths(case)
    if op == "store":
        # bf16 rows in, 296 bytes of codes and scales out; those in again, bf16 rows out
        n = int(new.sum()) * hkv
        return {"bytes": n * 2 * (2 * D * 2 + 2 * (D // 2 + D // 16 + 4)), "flops": n * 2 * D * 8}
    if op == "decode":
        keys = _visible(ctx - 1, case["sink"], case["win"])[2]
        return {"bytes": int(keys.sum()) * hkv * 2 * (D // 2 + D // 16 + 4) + case["seqs"] * case["hq"] * D * 4,
                "flops": 4 * D * case["hq"] * int(keys.sum())}
    if op == "prefill":
        pairs = union = 0
        for c, n in zip(ctx, new):
            pairs += int(_visible(np.arange(c, c + n), case["sink"], case["win"])[2].sum())
            union += int(_visible(np.array([c]), case["sink"], case["win"])[2][0] + n - 1)
        return {"bytes": union * hkv * 2 * (D // 2 + D // 16 + 4) + int(new.sum()) * case["hq"] * D * 4,
                "flops": 4 * D * case["hq"] * pairs}
    if op == "fork":
        copied = int((ctx % PAGE != 0).sum())
        return {"bytes": 8 * int(_pages(ctx).sum()) + 2 * copied * case["layers"] * _page_bytes(case), "flops": 0}
    entries, used, _, moves, _ = _compact_counts(case)
    return {"bytes": 4 * used + 4 * entries + 2 * moves * case["layers"] * _page_bytes(case), "flops": 0}


# ---------------------------------------------------------------- the 4-bit format, plain
def _unmixed(device):
    """Where piece i of token r's codes lies: [16, 8]."""
    r = torch.arange(PAGE, device=device)[:, None]
    return torch.arange(8, device=device)[None] ^ (r % 8)


def _quantise(x):
    """Rows [..., 256] -> codes (uint8 of 4 bits), block scales (e4m3) [..., 16], row scales (fp32)."""
    x = x.float()
    m, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(m <= 0.65625, e - 12, e - 11).clamp_min(-100)  # the row's largest value is at most 2688 steps
    step = ((e + 127) << 23).view(torch.float32)
    y = (x / step[..., None]).unflatten(-1, (16, 16))
    block = (y.abs().amax(-1) / 6).to(torch.float8_e4m3fn)
    b = block.float()[..., None]
    a = torch.where(b > 0, y.abs() / torch.where(b > 0, b, 1.0), 0.0)
    code = torch.zeros_like(a, dtype=torch.uint8)
    for border, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (a >= border) if up else (a > border)  # ties to the even code
    code |= torch.signbit(y).to(torch.uint8) << 3
    return code.flatten(-2), block, torch.where(m > 0, step, 0.0)


def _tiles(rows_k, rows_v, out):
    """K and V rows [pages, 16, heads, 256] quantised into out [pages, heads, TILE]."""
    n, _, h, _ = rows_k.shape
    where = _unmixed(out.device)
    for kv, rows in enumerate((rows_k, rows_v)):
        code, block, step = _quantise(rows.transpose(1, 2))
        packed = (code[..., 0::2] | (code[..., 1::2] << 4)).unflatten(-1, (8, 16))
        mixed = torch.gather(packed, 3, where[None, None, :, :, None].expand(n, h, PAGE, 8, 16))  # its own inverse
        out[:, :, 2048 * kv: 2048 * (kv + 1)] = mixed.flatten(2)
        out[:, :, 4096 + 256 * kv: 4352 + 256 * kv] = block.view(torch.uint8).flatten(2)
        out[:, :, 4608 + 64 * kv: 4672 + 64 * kv] = step.contiguous().view(torch.uint8).flatten(2)


def _values(tiles, kv):
    """The values of K (kv 0) or V (1) of tiles [..., TILE], fp32 [..., 16, 256]."""
    where = _unmixed(tiles.device)
    packed = tiles[..., 2048 * kv: 2048 * (kv + 1)].unflatten(-1, (PAGE, 8, 16))
    packed = torch.gather(packed, -2, where[:, :, None].expand(packed.shape)).flatten(-2)
    code = torch.stack((packed & 15, packed >> 4), -1).flatten(-2)
    m = (code & 7).float()
    x = torch.where(m < 4, m * 0.5, torch.where(m < 6, m - 2, m * 2 - 8)) * (1 - 2 * (code >> 3).float())
    block = tiles[..., 4096 + 256 * kv: 4352 + 256 * kv].contiguous().view(torch.float8_e4m3fn).unflatten(-1, (PAGE, 16))
    step = tiles[..., 4608 + 64 * kv: 4672 + 64 * kv].contiguous().view(torch.float32)
    return (x.unflatten(-1, (16, 16)) * block.float()[..., None]).flatten(-2) * step[..., None]


def _random_pool4(g, n_pages, hkv):
    """A 4-bit pool of normal rows, 1 in 100 tokens eight times as large."""
    out = torch.empty(n_pages, hkv, TILE, dtype=torch.uint8, device="cuda")
    for a in range(0, n_pages, 8192):
        n = min(8192, n_pages - a)
        big = 1 + 7 * (torch.rand(n, PAGE, 1, 1, generator=g, device="cuda") < 0.01)
        k, v = (torch.randn(n, PAGE, hkv, D, generator=g, device="cuda").mul_(big).bfloat16() for _ in range(2))
        _tiles(k, v, out[a: a + n])
    return out


def _table(rows_of_pages, n_cols, perm):
    """int32 [rows, n_cols]: each row's pages from perm in turn, -1 behind them."""
    bt = torch.full((len(rows_of_pages), n_cols), -1, dtype=torch.int32, device="cuda")
    row = np.repeat(np.arange(len(rows_of_pages)), rows_of_pages)
    col = np.concatenate([np.arange(n) for n in rows_of_pages])
    bt[torch.from_numpy(row).cuda(), torch.from_numpy(col).cuda()] = perm[: len(row)]
    return bt


# ---------------------------------------------------------------- states
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=case)
    return {"store": _prepare_store, "decode": _prepare_attention, "prefill": _prepare_attention,
            "fork": _prepare_fork, "compact": _prepare_compact}[case["op"]](case, s, g, seed)


def _handle(s, hq, hkv, n_pool, max_pages):
    if own:
        import windowed_prefill_attention_gb300 as pa
        s["handle"] = pa.Handle(hq, hkv, n_pool, max_pages)
    return s


def _prepare_store(case, s, g, seed):
    hkv = case["hkv"]
    ctx, new = _lengths(case)
    tok = int(new.sum())
    if case["fused"]:  # views of one fused projection buffer
        x = torch.randn(tok, (case["hq"] + 2 * hkv) * D, generator=g, device="cuda").mul_(1.5).bfloat16()
        s["k"] = x[:, case["hq"] * D: (case["hq"] + hkv) * D].view(tok, hkv, D)
        s["v"] = x[:, (case["hq"] + hkv) * D:].view(tok, hkv, D)
    else:
        s["k"], s["v"] = (torch.randn(tok, hkv, D, generator=g, device="cuda").mul_(1.5).bfloat16() for _ in range(2))
    pages = _pages(ctx + new)
    n_pool, max_pages = int(pages.sum()), int(pages.max())
    s["seqs"] = np.stack([np.cumsum(new) - new, ctx, new, ctx + new], 1).astype(np.int32)
    s["block_table"] = _table(pages, max_pages, torch.randperm(n_pool, generator=g, device="cuda").to(torch.int32))
    s["pool"] = _random_pool4(g, n_pool, hkv)
    seq_of = np.repeat(np.arange(len(new)), new)
    at = np.concatenate([c + np.arange(n) for c, n in zip(ctx, new)])
    page = s["block_table"][torch.from_numpy(seq_of).cuda(), torch.from_numpy(at // PAGE).cuda()].long()
    s["slots"] = (page, torch.from_numpy(at % PAGE).cuda())
    s["k_out"], s["v_out"] = (torch.empty(tok, hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    return _handle(s, case["hq"], hkv, n_pool, max_pages)


def _prepare_attention(case, s, g, seed):
    hq, hkv = case["hq"], case["hkv"]
    ctx, new = _lengths(case)
    if case["op"] == "decode":
        end, tok = ctx, len(ctx)
        s["seqs"] = np.stack([np.arange(tok), ctx - 1, np.ones_like(ctx), ctx], 1).astype(np.int32)
    else:
        end, tok = ctx + new, int(new.sum())
        s["seqs"] = np.stack([np.cumsum(new) - new, ctx, new, end], 1).astype(np.int32)
    pages = _pages(end)
    n_pool, max_pages = int(pages.sum()), int(pages.max())
    s["block_table"] = _table(pages, max_pages, torch.randperm(n_pool, generator=g, device="cuda").to(torch.int32))
    s["pool"] = _random_pool4(g, n_pool, hkv)
    s["q"] = torch.randn(tok, hq, D, generator=g, device="cuda").bfloat16()
    s["out"] = torch.empty_like(s["q"])
    s["n_ctx"] = torch.from_numpy(end).cuda()
    s["sm_scale"] = 1.0 / 16.0
    return _handle(s, hq, hkv, n_pool, max_pages)


def _random_parts(case, g, n_pool):
    """The pools of all layers: int8 codes and fp32 scales of K and V, or 4-bit tiles."""
    parts = []
    for _ in range(case["layers"]):
        if case["pool"] == "int8":
            parts += [torch.randint(-127, 128, (n_pool, PAGE, case["hkv"], D), generator=g, device="cuda",
                                    dtype=torch.int8) for _ in range(2)]
            parts += [torch.rand(n_pool, PAGE, case["hkv"], generator=g, device="cuda") + 0.01 for _ in range(2)]
        else:
            # copied as bytes, whatever they stand for
            parts.append(torch.randint(0, 256, (n_pool, case["hkv"], TILE), generator=g, device="cuda", dtype=torch.uint8))
    return parts


def _prepare_fork(case, s, g, seed):
    """Forks of pairwise different sources, or of one source where ctx_lo is ctx_hi."""
    ctx, _ = _lengths(case)
    n = case["forks"]
    pages = _pages(ctx)
    one = case["ctx_lo"] == case["ctx_hi"]
    src_pages = pages[:1] if one else pages
    n_src, used = len(src_pages), int(src_pages.sum())
    n_pool, max_pages = used + n, int(pages.max()) + 3
    perm = torch.randperm(n_pool, generator=g, device="cuda").to(torch.int32)
    s["block_table"] = torch.cat((_table(src_pages, max_pages, perm),
                                  torch.full((n, max_pages), -1, dtype=torch.int32, device="cuda")))
    new_page = perm[used:]
    src = np.zeros(n, np.int64) if one else np.arange(n)
    s["forks"] = np.stack([src, n_src + np.arange(n), ctx, new_page.cpu().numpy()], 1).astype(np.int32)
    s["parts"] = _random_parts(case, g, n_pool)
    s["src"], s["dst"] = torch.from_numpy(src).cuda(), torch.arange(n, device="cuda") + n_src
    s["pages"], s["partial"] = torch.from_numpy(pages).cuda(), torch.from_numpy(ctx % PAGE != 0).cuda()
    s["new_page"] = new_page
    return _handle(s, 2 * case["hkv"], case["hkv"], n_pool, max_pages)


def _prepare_compact(case, s, g, seed):
    ctx, _ = _lengths(case)
    n, sh = case["seqs"], case["shared"]
    blocks = _pages(ctx)
    _, _, live, moves, n_pool = _compact_counts(case)
    max_pages = int(blocks.max()) + 2
    lo = np.maximum(0, ctx // PAGE + 1 - case["win"]) if case["win"] > 0 else np.zeros_like(ctx)
    col = np.arange(max_pages)[None]
    used = (col < blocks[:, None]) & ((col < case["sink"]) | (col >= lo[:, None]))
    # a page number for each entry: the shared blocks' own, then one for each other entry
    page = np.full((n, max_pages), -1, np.int64)
    page[:, :sh] = np.arange(sh)[None]
    rest = (col >= sh) & (col < blocks[:, None])
    page[rest] = sh + np.arange(int(rest.sum()))
    page[col >= blocks[:, None]] = -1
    total = sh + int(rest.sum())
    is_live = np.zeros(total, bool)
    is_live[page[used]] = True
    # so many pages in use behind the first `live`, the others among them
    rng = np.random.default_rng(seed)
    front, back = rng.permutation(live), live + rng.permutation(n_pool - live)
    place = np.empty(total, np.int64)
    place[is_live] = rng.permutation(np.concatenate((front[moves:], back[:moves])))
    free = rng.permutation(np.concatenate((front[:moves], back[moves:])))
    place[~is_live] = free[: total - live]
    table = np.where(page >= 0, place[np.maximum(page, 0)], -1).astype(np.int32)
    s["block_table"] = torch.from_numpy(table).cuda()
    s["new_table"] = torch.empty_like(s["block_table"])
    s["n_live"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    s["seqs"] = np.stack([np.arange(n), ctx - 1, np.ones(n, np.int64), ctx], 1).astype(np.int32)
    s["ctx"] = torch.from_numpy(ctx).cuda()
    s["parts"] = _random_parts(case, g, n_pool)
    return _handle(s, 2 * case["hkv"], case["hkv"], n_pool, max_pages)


# ---------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return {"store": _store_own, "decode": _decode_own, "prefill": _prefill_own, "fork": _fork_own,
                "compact": _compact_own}[op](s)
    return {"store": _store_plain, "decode": _decode_plain, "prefill": _prefill_plain, "fork": _fork_plain,
            "compact": _compact_plain}[op](s)


def _store_own(s):
    import windowed_prefill_attention_gb300 as pa
    h = s["handle"].h
    pa.pa_kv4_append(h, s["seqs"], s["k"], s["v"], s["block_table"], s["pool"])
    pa.pa_kv4_gather(h, s["seqs"], s["block_table"], s["pool"], s["k_out"], s["v_out"])
    return {"k": s["k_out"], "v": s["v_out"]}


def _decode_own(s):
    import windowed_prefill_attention_gb300 as pa
    c = s["case"]
    pa.pa_kv4_decode(s["handle"].h, s["seqs"], s["q"], s["pool"], s["block_table"], c["sink"], c["win"], s["sm_scale"],
                     s["out"])
    return s["out"]


def _prefill_own(s):
    import windowed_prefill_attention_gb300 as pa
    c = s["case"]
    pa.pa_kv4_prefill(s["handle"].h, s["seqs"], s["q"], s["pool"], s["block_table"], c["sink"], c["win"], s["sm_scale"],
                      s["out"])
    return s["out"]


def _fork_own(s):
    import windowed_prefill_attention_gb300 as pa
    pa.pa_pages_fork(s["handle"].h, s["forks"], s["block_table"], s["parts"])
    return {"table": s["block_table"], "parts": s["parts"]}


def _compact_own(s):
    import windowed_prefill_attention_gb300 as pa
    c = s["case"]
    pa.pa_pages_compact(s["handle"].h, s["seqs"], c["sink"], c["win"], s["block_table"], s["new_table"], s["parts"],
                        s["n_live"])
    return {"table": s["new_table"], "n_live": s["n_live"], "parts": s["parts"]}


def _store_plain(s):
    page, slot = s["slots"]
    where = _unmixed(page.device)[slot]
    pool = s["pool"]
    for kv, rows in enumerate((s["k"], s["v"])):
        code, block, step = _quantise(rows)
        packed = (code[..., 0::2] | (code[..., 1::2] << 4)).unflatten(-1, (8, 16))
        mixed = torch.gather(packed, 2, where[:, None, :, None].expand(packed.shape))
        pool[:, :, 2048 * kv: 2048 * (kv + 1)].unflatten(-1, (PAGE, 128))[page, :, slot] = mixed.flatten(2)
        pool[:, :, 4096 + 256 * kv: 4352 + 256 * kv].unflatten(-1, (PAGE, 16))[page, :, slot] = block.view(torch.uint8)
        pool[:, :, 4608 + 64 * kv: 4672 + 64 * kv].unflatten(-1, (PAGE, 4))[page, :, slot] = (
            step.contiguous().view(torch.uint8).unflatten(-1, (-1, 4)))
    # read back: the new tokens' rows
    out = []
    for kv in range(2):
        packed = pool[:, :, 2048 * kv: 2048 * (kv + 1)].unflatten(-1, (PAGE, 8, 16))[page, :, slot]
        packed = torch.gather(packed, 2, where[:, None, :, None].expand(packed.shape)).flatten(-2)
        code = torch.stack((packed & 15, packed >> 4), -1).flatten(-2)
        m = (code & 7).float()
        x = torch.where(m < 4, m * 0.5, torch.where(m < 6, m - 2, m * 2 - 8)) * (1 - 2 * (code >> 3).float())
        block = pool[:, :, 4096 + 256 * kv: 4352 + 256 * kv].unflatten(-1, (PAGE, 16))[page, :, slot]
        step = pool[:, :, 4608 + 64 * kv: 4672 + 64 * kv].unflatten(-1, (PAGE, 4))[page, :, slot]
        x = x.unflatten(-1, (16, 16)) * block.contiguous().view(torch.float8_e4m3fn).float()[..., None]
        out.append((x.flatten(-2) * step.contiguous().view(torch.float32)).bfloat16())
    return {"k": out[0], "v": out[1]}


def _decode_plain(s):
    c = s["case"]
    n, hq, hkv = c["seqs"], c["hq"], c["hkv"]
    t = s["n_ctx"] - 1
    last = t // PAGE
    lo = (last + 1 - c["win"]).clamp_min(0) if c["win"] > 0 else torch.zeros_like(t)
    n_sink = lo.clamp_max(c["sink"])
    ctx = _lengths(c)[0]
    h_sink, h_lo, _ = _visible(ctx - 1, c["sink"], c["win"])
    most = int((h_sink + (ctx - 1) // PAGE - h_lo + 1).max())  # the longest list of visible blocks
    j = torch.arange(most, device=t.device)
    block = torch.where(j < n_sink[:, None], j, lo[:, None] + j - n_sink[:, None])
    page = torch.gather(s["block_table"].long(), 1, block.clamp_max(s["block_table"].shape[1] - 1)).clamp_min(0)
    tok = (block[:, :, None] * PAGE + torch.arange(PAGE, device=t.device)).flatten(1)
    seen = tok <= t[:, None]
    out = []
    step = max(1, 500000 // (most * PAGE * hkv))
    for a in range(0, n, step):
        b = min(n, a + step)
        tiles = s["pool"][page[a:b]]
        k, v = (_values(tiles, kv).transpose(1, 2).flatten(2, 3) for kv in range(2))  # [sequences, heads, keys, 256]
        q = s["q"][a:b].float().view(b - a, hkv, hq // hkv, D)
        y = torch.matmul(q, k.transpose(2, 3)) * s["sm_scale"]
        y = y.masked_fill_(~seen[a:b, None, None], -math.inf)
        e = (y - y.amax(-1, keepdim=True)).exp_()
        out.append((torch.matmul(e, v) / e.sum(-1, keepdim=True)).view(b - a, hq, D).bfloat16())
    return torch.cat(out)


def _prefill_plain(s):
    c = s["case"]
    hq, hkv = c["hq"], c["hkv"]
    for i, (row, start, n, end) in enumerate(s["seqs"].tolist()):
        first = max(0, start // PAGE + 1 - c["win"]) if c["win"] > 0 else 0
        block = torch.cat((torch.arange(min(c["sink"], first), device="cuda"),
                           torch.arange(first, (end + PAGE - 1) // PAGE, device="cuda")))
        tiles = s["pool"][s["block_table"][i].long()[block]]
        k, v = (_values(tiles, kv).transpose(0, 1).flatten(1, 2) for kv in range(2))  # [heads, keys, 256]
        tok = (block[:, None] * PAGE + torch.arange(PAGE, device="cuda")).flatten()
        for a in range(0, n, 512):
            b = min(n, a + 512)
            t = start + torch.arange(a, b, device="cuda")
            seen = tok <= t[:, None]
            if c["win"] > 0:
                seen &= (tok // PAGE < c["sink"]) | (tok // PAGE >= (t // PAGE + 1 - c["win"])[:, None])
            q = s["q"][row + a: row + b].float().view(b - a, hkv, hq // hkv, D).permute(1, 2, 0, 3)
            y = torch.matmul(q.flatten(1, 2), k.transpose(1, 2)).view(hkv, hq // hkv, b - a, -1) * s["sm_scale"]
            y = y.masked_fill_(~seen, -math.inf)
            e = (y - y.amax(-1, keepdim=True)).exp_()
            o = torch.matmul(e.flatten(1, 2), v).view(hkv, hq // hkv, b - a, D) / e.sum(-1, keepdim=True)
            s["out"][row + a: row + b] = o.permute(2, 0, 1, 3).reshape(b - a, hq, D).bfloat16()
    return s["out"]


def _fork_plain(s):
    bt = s["block_table"]
    col = torch.arange(bt.shape[1], device=bt.device)
    rows = torch.where(col < s["pages"][:, None], bt[s["src"]], bt[s["dst"]])
    last = (s["pages"] - 1).clamp_min(0)[:, None]
    old = torch.gather(rows, 1, last).squeeze(1)
    new = torch.where(s["partial"], s["new_page"], old)
    bt[s["dst"]] = rows.scatter(1, last, new[:, None])
    for p in s["parts"]:  # a fork whose last page is full copies that page onto itself
        p[new.long()] = p[old.long()]
    return {"table": bt, "parts": s["parts"]}


def _compact_plain(s):
    c, bt = s["case"], s["block_table"]
    n_pool = s["parts"][0].shape[0]
    col = torch.arange(bt.shape[1], device=bt.device)
    valid = col < ((s["ctx"] + PAGE - 1) // PAGE)[:, None]
    used = valid
    if c["win"] > 0:
        used = valid & ((col < c["sink"]) | (col >= (s["ctx"] // PAGE + 1 - c["win"])[:, None]))
    live = torch.zeros(n_pool + 1, dtype=torch.bool, device=bt.device)
    live[torch.where(used, bt.long(), n_pool)] = True
    live = live[:n_pool]
    n_live = live.sum()
    at = torch.arange(n_pool, device=bt.device)
    hole, mover = ~live & (at < n_live), live & (at >= n_live)
    # the r-th mover goes to the r-th hole
    holes = torch.argsort(torch.where(hole, at, n_pool + at))
    movers = torch.argsort(torch.where(mover, at, n_pool + at))
    to = torch.where(mover, holes[mover.cumsum(0).sub(1).clamp_min(0)], at)
    comes_from = torch.where(hole, movers[hole.cumsum(0).sub(1).clamp_min(0)], at)
    new = torch.where(used, to[bt.long().clamp_min(0)].int(), torch.where(valid, -1, bt))
    return {"table": new, "n_live": n_live.int().view(1), "parts": [p[comes_from] for p in s["parts"]]}


# ---------------------------------------------------------------- definitions in 64 bits
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _e4m3_values():
    return [math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10) for e in range(16) for m in range(8)][:127]


def _nearest(x, values):
    """The entry of an ascending list that is nearest to x, the even index at ties, the last one beyond it."""
    v = torch.tensor(values, dtype=torch.float64, device=x.device)
    up = torch.searchsorted(v, x.contiguous()).clamp(1, len(values) - 1)
    below, above = x - v[up - 1], v[up] - x
    even = torch.where(up % 2 == 0, up, up - 1)
    return v[torch.where(below < above, up - 1, torch.where(below > above, up, even))]


def _exact_rows(x):
    x = x.double()
    most = x.abs().amax(-1, keepdim=True)
    step = torch.exp2(torch.ceil(torch.log2(most.clamp_min(1e-300) / 2688)))
    step = torch.where(most > 2688 * step, 2 * step, torch.where(most <= 1344 * step, step / 2, step))  # log2's rounding
    step = torch.where(most > 0, step.clamp_min(2.0 ** -100), 1.0)
    out = []
    for i in range(0, D, 16):
        b = x[..., i: i + 16]
        size = _nearest(b.abs().amax(-1, keepdim=True) / step / 6, _e4m3_values()) * step
        ratio = torch.where(size > 0, b.abs() / torch.where(size > 0, size, 1.0), 0.0)
        out.append(torch.sign(b) * _nearest(ratio, _E2M1) * size)
    return torch.cat(out, -1)


def _exact_tokens(tiles, r):
    """K and V values in 64 bits of token r[i] of tiles[i] ([keys, heads, TILE]), each [keys, heads, 256]."""
    dev = tiles.device
    pair = torch.tensor([[(-1.0 if c & 8 else 1.0) * _E2M1[c & 7] for c in (b & 15, b >> 4)] for b in range(256)],
                        dtype=torch.float64, device=dev)
    byte_scale = torch.tensor(_e4m3_values() + [math.nan] + [-v for v in _e4m3_values()] + [math.nan],
                              dtype=torch.float64, device=dev)
    d = torch.arange(0, D, 2, device=dev)
    out = []
    for kv in range(2):
        at = 2048 * kv + 128 * r[:, None] + 16 * ((d // 32) ^ (r[:, None] % 8)) + d % 32 // 2
        codes = torch.gather(tiles, 2, at[:, None].expand(-1, tiles.shape[1], -1))
        at = 4096 + 256 * kv + 16 * r[:, None] + d // 16
        block = torch.gather(tiles, 2, at[:, None].expand(-1, tiles.shape[1], -1))
        at = 4608 + 64 * kv + 4 * r[:, None] + torch.arange(4, device=dev)
        step = torch.gather(tiles, 2, at[:, None].expand(-1, tiles.shape[1], -1)).contiguous().view(torch.float32)
        out.append((pair[codes.int()] * byte_scale[block.int()][..., None]).flatten(-2) * step.double())
    return out


def _exact_fork(s):
    table = s["block_table"].tolist()
    return [(table[src][tok // PAGE], page) for src, _, tok, page in s["forks"].tolist() if tok % PAGE]


def _exact_moves(s):
    c, table, live = s["case"], s["block_table"].tolist(), set()
    for row, tok in zip(table, s["ctx"].tolist()):
        for b in range(-(-tok // PAGE)):
            if c["win"] <= 0 or b < c["sink"] or b > tok // PAGE - c["win"]:
                live.add(row[b])
    holes = [p for p in range(len(live)) if p not in live]
    return list(zip(sorted(p for p in live if p >= len(live)), holes))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "store":
        return {"k": _exact_rows(s["k"]), "v": _exact_rows(s["v"])}
    if case["op"] in ("fork", "compact"):  # the scales, page by page
        if case["pool"] != "int8":
            return None
        moves = _exact_fork(s) if case["op"] == "fork" else _exact_moves(s)
        parts = [None if p.dtype is torch.int8 else p.double() for p in s["parts"]]
        for p in parts:
            for source, to in moves if p is not None else ():
                p[to] = p[source]  # none writes what another reads
        return {"table": None, "parts": parts, **({} if case["op"] == "fork" else {"n_live": None})}
    # one sequence at a time over the keys that its queries see
    hq, hkv, out = case["hq"], case["hkv"], torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for i, (row, start, n, end) in enumerate(s["seqs"].tolist()):
        j = torch.arange(end, device="cuda")
        if case["win"] > 0:
            j = j[(j // PAGE < case["sink"]) | (j // PAGE > start // PAGE - case["win"])]
        page = s["block_table"][i].long()[j // PAGE]
        k, v = (torch.cat(part).transpose(0, 1) for part in zip(*(
            _exact_tokens(s["pool"][page[a: a + 8192]], j[a: a + 8192] % PAGE) for a in range(0, len(j), 8192))))
        for a in range(0, n, 256):
            t = start + torch.arange(a, min(n, a + 256), device="cuda")
            hidden = j > t[:, None]
            if case["win"] > 0:
                hidden |= (j // PAGE >= case["sink"]) & (j // PAGE <= t[:, None] // PAGE - case["win"])
            q = s["q"][row + a: row + a + len(t)].double().view(len(t), hkv, hq // hkv, D).permute(1, 2, 0, 3)
            y = torch.einsum("hgtd,hjd->hgtj", q, k) * s["sm_scale"]
            p = torch.softmax(y.masked_fill(hidden, -math.inf), -1)
            out[row + a: row + a + len(t)] = torch.einsum("hgtj,hjd->thgd", p, v).reshape(len(t), hq, D)
    return out
