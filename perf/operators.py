"""Performance cases of the layer-step operators around the paged int8 KV pool.

    rope     pa_qk_norm_rope: RMS norm of every query and key head and the
             rotary positions (one or several axes), one pass
    append   pa_qkv_append: the same pass for a batch of sequences, the new K
             and V rows quantised into the paged pool
    shared   pa_decode_shared: one new token per sequence, all sequences
             sharing a prefix whose pages the pool holds once

Each case is a dict of plain values.  ``run`` computes an operator in its
plain form, elementary torch operations in 32 bits (rotation angles in 64),
or, where ``own`` is true, by the calls a user makes of this package.
"""
import math

import numpy as np
import torch

own = False

D, PAGE = 256, 16


def listed():
    return [
        # one token of one sequence: the step of a single chat, where launch latency is all there is
        dict(name="rope 1 token", op="rope", tok=1, hq=16, hkv=2, rot=64, pairing="half", axes=1, fused=True,
             offset=0.0),
        # a mid-sized image / video prompt: three position axes, neighbouring pairs, an odd token count
        dict(name="rope 4099 three axes", op="rope", tok=4099, hq=8, hkv=4, rot=128, pairing="adjacent", axes=3,
             fused=True, offset=1.0),
        # a whole 32k prompt, every dim rotated: bound by memory
        dict(name="rope 32768", op="rope", tok=32768, hq=16, hkv=2, rot=256, pairing="half", axes=1, fused=False,
             offset=0.0),
        # a decode step of 64 sequences at long contexts
        dict(name="append 64 x 1", op="append", seqs=64, new_lo=1, new_hi=1, ctx_lo=500, ctx_hi=8000, hq=16, hkv=2,
             rot=64, pairing="half", axes=1, fused=True, offset=0.0),
        # four sequences appending 2048-token prompt chunks to caches of several lengths
        dict(name="append 4 x 2048", op="append", seqs=4, new_lo=2048, new_hi=2048, ctx_lo=1000, ctx_hi=30000, hq=16,
             hkv=2, rot=64, pairing="half", axes=1, fused=True, offset=0.0),
        # short ragged prompts with three position axes, as many kv heads as query heads
        dict(name="append 13 ragged", op="append", seqs=13, new_lo=3, new_hi=1501, ctx_lo=0, ctx_hi=700, hq=8, hkv=8,
             rot=96, pairing="adjacent", axes=3, fused=False, offset=1.0),
        # a few sequences behind a system prompt
        dict(name="shared 3 x 1024", op="shared", seqs=3, prefix=1024, suf_lo=1, suf_hi=200, hq=16, hkv=2, sink=1,
             win=0),
        # a batch behind one long document, window off
        dict(name="shared 64 x 32768", op="shared", seqs=64, prefix=32768, suf_lo=1, suf_hi=1024, hq=16, hkv=2,
             sink=1, win=0),
        # many short answers behind a medium prompt
        dict(name="shared 250 x 8192", op="shared", seqs=250, prefix=8192, suf_lo=5, suf_hi=256, hq=16, hkv=2, sink=1,
             win=0),
        # one kv head, a very long prefix and few sequences: few rows, many keys
        dict(name="shared 9 x 131072", op="shared", seqs=9, prefix=131072, suf_lo=1, suf_hi=333, hq=8, hkv=1, sink=0,
             win=0),
        # the sliding window: sequences see the sink and the part of the prefix their window still reaches
        dict(name="shared 48 windowed", op="shared", seqs=48, prefix=8192, suf_lo=1, suf_hi=2000, hq=8, hkv=4, sink=1,
             win=256),
    ]


#: A drawn case's cost (bytes, or flops / 50) stays under the largest listed one's.
_MOST = 6.0e8


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(("rope", "append", "shared"))
        if op == "shared":
            hq, hkv = rng.choice(((16, 2), (8, 4), (4, 1), (8, 8), (8, 1), (8, 2)))
            c = dict(op=op, seqs=_log_int(rng, 1, 250), prefix=16 * _log_int(rng, 1, 8192), suf_lo=rng.randint(1, 20),
                     suf_hi=_log_int(rng, 20, 2000), hq=hq, hkv=hkv, sink=rng.choice((0, 1, 4)),
                     win=rng.choice((0, 0, 0, 64, 256)))
        else:
            hq, hkv = rng.choice(((16, 2), (8, 4), (4, 1), (8, 8), (32, 2), (10, 5)))
            axes = rng.choice((1, 1, 2, 3))
            c = dict(op=op, hq=hq, hkv=hkv, rot=rng.choice((0, 32, 64, 96, 128, 256)),
                     pairing=rng.choice(("half", "adjacent")), axes=axes, fused=rng.random() < 0.5,
                     offset=rng.choice((0.0, 1.0)))
            if op == "rope":
                c["tok"] = _log_int(rng, 1, 32768)
            else:
                c["seqs"] = _log_int(rng, 1, 300)
                c["new_hi"] = _log_int(rng, 1, max(1, 12000 // c["seqs"]))
                c["new_lo"] = rng.randint(1, c["new_hi"])
                c["ctx_lo"] = rng.randint(0, 50)
                c["ctx_hi"] = c["ctx_lo"] + _log_int(rng, 1, 4000)
        w = work(c)
        if max(w["bytes"], w["flops"] / 50) <= _MOST:
            return c


def _spread(lo, hi, n, step):
    """n whole numbers over [lo, hi] in a mixed order, both ends among them where n > 1."""
    i = (np.arange(n, dtype=np.int64) * step) % n
    return (hi - i * (hi - lo) // max(1, n - 1)).astype(np.int64)


def _lengths(case):
    """Per sequence (cached tokens, new tokens) of an append case, (0, suffix tokens) of a shared one."""
    n = case["seqs"]
    if case["op"] == "shared":
        return np.zeros(n, np.int64), _spread(case["suf_lo"], max(case["suf_lo"], case["suf_hi"]), n, 7919)
    return _spread(case["ctx_lo"], case["ctx_hi"], n, 104729), _spread(case["new_lo"], case["new_hi"], n, 7919)


def _shared_visible(case):
    """Visible blocks of the prefix to any sequence, and per sequence the visible keys of prefix and suffix."""
    _, suf = _lengths(case)
    pb = case["prefix"] // PAGE
    t = case["prefix"] + suf - 1
    last = t // PAGE
    lo = np.maximum(0, last + 1 - case["win"]) if case["win"] > 0 else np.zeros_like(t)
    sink = np.minimum(case["sink"], lo) if case["win"] > 0 else np.zeros_like(t)
    pre_sink, pre_win = np.minimum(sink, pb), np.maximum(0, pb - lo)
    lo_all = int(lo.min())
    union = min(pb, int(max(0, min(case["sink"], lo_all)))) + max(0, pb - lo_all)
    suf_blocks_before = np.maximum(lo, pb) - pb  # hidden blocks of the suffix, before its window
    suf_sink = np.maximum(0, np.minimum(sink, np.maximum(lo, pb)) - pb)
    suf_keys = suf - PAGE * suf_blocks_before + PAGE * suf_sink
    return union, PAGE * (pre_sink + pre_win), suf_keys


def work(case):
    hq, hkv = case["hq"], case["hkv"]
    if case["op"] == "rope":
        return {"bytes": case["tok"] * (hq + hkv) * D * 4 + 4 * case["tok"] * case["axes"],
                "flops": case["tok"] * (hq + hkv) * D * 8}
    if case["op"] == "append":
        n = int(_lengths(case)[1].sum())
        return {"bytes": n * (hq * D * 4 + hkv * (2 * D * 2 + 2 * D + 8)) + 4 * n * case["axes"],
                "flops": n * (hq + 2 * hkv) * D * 8}
    union, pre, suf = _shared_visible(case)
    keys = union * PAGE + int(suf.sum())
    return {"bytes": keys * hkv * (2 * D + 8) + case["seqs"] * hq * D * 4,
            "flops": 4 * D * hq * int(pre.sum() + suf.sum())}


def _frequencies(case):
    """Radians per position of each rotated pair, and the position axis it follows (sections of the pairs)."""
    pairs = case["rot"] // 2
    inv = 1000000.0 ** (-np.arange(pairs, dtype=np.float64) / max(1, pairs))
    return inv, (np.arange(pairs) * case["axes"] // max(1, pairs)).astype(np.int32)


def _positions(case, starts, counts):
    """int32 [axes, tokens]: a text position, or (time, height, width) of a 32 x 32 grid of patches."""
    p = np.concatenate([s + np.arange(n) for s, n in zip(starts, counts)])
    i = np.concatenate([np.arange(n) for n in counts])
    rows = [p] if case["axes"] == 1 else [p - i + i // 1024, (i // 32) % 32, i % 32][: case["axes"]]
    return np.stack(rows).astype(np.int32)


def _projections(case, g, tok):
    """The layer's projected rows: views of one fused buffer (query and gate of a head side by side), or one tensor each."""
    hq, hkv = case["hq"], case["hkv"]
    if case["fused"]:
        x = torch.randn(tok, (2 * hq + 2 * hkv) * D, generator=g, device="cuda").mul_(1.5).bfloat16()
        q = x[:, : 2 * hq * D].view(tok, hq, 2, D)[:, :, 0]
        k = x[:, 2 * hq * D: (2 * hq + hkv) * D].view(tok, hkv, D)
        return q, k, x[:, (2 * hq + hkv) * D:].view(tok, hkv, D)
    return tuple(torch.randn(tok, h, D, generator=g, device="cuda").mul_(1.5).bfloat16() for h in (hq, hkv, hkv))


def _weights(case, g):
    return tuple((torch.randn(D, generator=g, device="cuda") * 0.1 + 1.0 - case["offset"]).bfloat16()
                 for _ in range(2))


def _pool(g, n_pages, hkv):
    """K and V pools of normal values, 1 in 100 tokens eight times as large, quantised per (token, head)."""
    x = torch.randn(2, n_pages, PAGE, hkv, D, generator=g, device="cuda")
    x *= 1 + 7 * (torch.rand(1, n_pages, PAGE, 1, 1, generator=g, device="cuda") < 0.01)
    scale = x.abs().amax(-1) / 127
    return torch.round(x / scale[..., None]).to(torch.int8), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=case)
    hq, hkv = case["hq"], case["hkv"]
    if case["op"] != "shared":
        s["eps"] = 1e-6
        s["inv_freq"], s["pair_axis"] = _frequencies(case)
        s["freq"] = torch.from_numpy(s["inv_freq"]).cuda()
        s["axis"] = torch.from_numpy(s["pair_axis"]).cuda().long()
        s["qw"], s["kw"] = _weights(case, g)
    if case["op"] == "rope":
        s["q"], s["k"], _ = _projections(case, g, case["tok"])
        start = int(torch.randint(0, 100000, (1,), generator=g, device="cuda"))
        s["positions"] = torch.from_numpy(_positions(case, [start], [case["tok"]])).cuda()
        s["q_out"] = torch.empty(case["tok"], hq, D, dtype=torch.bfloat16, device="cuda")
        s["k_out"] = torch.empty(case["tok"], hkv, D, dtype=torch.bfloat16, device="cuda")
        n_pool, max_pages = 1, 1
    elif case["op"] == "append":
        ctx, new = _lengths(case)
        tok = int(new.sum())
        s["q"], s["k"], s["v"] = _projections(case, g, tok)
        s["positions"] = torch.from_numpy(_positions(case, ctx, new)).cuda()
        s["q_out"] = torch.empty(tok, hq, D, dtype=torch.bfloat16, device="cuda")
        first = np.cumsum(new) - new
        s["seqs"] = np.stack([first, ctx, new, ctx + new], 1).astype(np.int32)
        pages = (ctx + new + PAGE - 1) // PAGE
        n_pool, max_pages = int(pages.sum()), int(pages.max())
        perm = torch.randperm(n_pool, generator=g, device="cuda").to(torch.int32)
        row = np.repeat(np.arange(len(pages)), pages)
        col = np.concatenate([np.arange(n) for n in pages])
        s["block_table"] = torch.full((len(pages), max_pages), -1, dtype=torch.int32, device="cuda")
        s["block_table"][torch.from_numpy(row).cuda(), torch.from_numpy(col).cuda()] = perm
        s["kv"], s["scale"] = _pool(g, n_pool, hkv)
        # where each new token goes, and the pages they touch
        seq_of = np.repeat(np.arange(len(new)), new)
        at = np.concatenate([c + np.arange(n) for c, n in zip(ctx, new)])
        page = s["block_table"][torch.from_numpy(seq_of).cuda(), torch.from_numpy(at // PAGE).cuda()].long()
        s["slots"] = (page, torch.from_numpy(at % PAGE).cuda())
        s["pages"] = torch.unique(page)
        s["values"] = torch.empty(2, s["pages"].numel(), PAGE, hkv, D, dtype=torch.bfloat16, device="cuda")
    else:
        _, suf = _lengths(case)
        n, pb = case["seqs"], case["prefix"] // PAGE
        own_pages = (suf + PAGE - 1) // PAGE
        n_pool, max_pages = pb + int(own_pages.sum()), pb + int(own_pages.max())
        s["kv"], s["scale"] = _pool(g, n_pool, hkv)
        perm = torch.randperm(n_pool, generator=g, device="cuda").to(torch.int32)
        bt = torch.full((n, max_pages), -1, dtype=torch.int32, device="cuda")
        bt[:, :pb] = perm[:pb]
        row = np.repeat(np.arange(n), own_pages)
        col = pb + np.concatenate([np.arange(k) for k in own_pages])
        bt[torch.from_numpy(row).cuda(), torch.from_numpy(col).cuda()] = perm[pb:]
        s["block_table"] = bt
        s["q"] = torch.randn(n, hq, D, generator=g, device="cuda").bfloat16()
        s["out"] = torch.empty_like(s["q"])
        s["n_ctx"] = torch.from_numpy(case["prefix"] + suf).cuda()
        s["seqs"] = np.stack([np.arange(n), case["prefix"] + suf - 1, np.ones_like(suf), case["prefix"] + suf],
                             1).astype(np.int32)
        s["sm_scale"] = 1.0 / 16.0
    if "kv" in s:
        s["k_pool"], s["v_pool"] = s["kv"]
        s["k_scale"], s["v_scale"] = s["scale"]
    if own:
        import windowed_prefill_attention_gb300 as pa
        s["handle"] = pa.Handle(hq, hkv, n_pool, max_pages)
        if case["op"] != "shared":
            pairing = pa.PA_ROPE_HALF if case["pairing"] == "half" else pa.PA_ROPE_ADJACENT
            s["rope"] = pa.pa_rope_init(s["inv_freq"], pairing, s["pair_axis"])
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        return {"rope": _rope_own, "append": _append_own, "shared": _shared_own}[op](s)
    return {"rope": _rope_plain, "append": _append_plain, "shared": _shared_plain}[op](s)


# ---------------------------------------------------------------- this package's calls
def _rope_own(s):
    import windowed_prefill_attention_gb300 as pa
    pa.pa_qk_norm_rope(s["handle"].h, s["q"], s["k"], s["qw"], s["kw"], s["eps"], s["rope"], s["positions"],
                       s["q_out"], s["k_out"], weight_offset=s["case"]["offset"])
    return {"q": s["q_out"], "k": s["k_out"]}


def _append_own(s):
    import windowed_prefill_attention_gb300 as pa
    pa.pa_qkv_append(s["handle"].h, s["seqs"], s["q"], s["k"], s["v"], s["qw"], s["kw"], s["eps"], s["rope"],
                     s["positions"], s["block_table"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"],
                     s["q_out"], weight_offset=s["case"]["offset"])
    return _written(s, s["q_out"])


def _shared_own(s):
    import windowed_prefill_attention_gb300 as pa
    c = s["case"]
    pa.pa_decode_shared(s["handle"].h, s["seqs"], c["prefix"], s["q"], s["k_pool"], s["v_pool"], s["k_scale"],
                        s["v_scale"], s["block_table"], c["sink"], c["win"], s["sm_scale"], s["out"])
    return s["out"]


# ---------------------------------------------------------------- plain forms
def _written(s, q):
    """The query rows, and the pages the new tokens went to: the values their codes stand for, and the scales."""
    codes, scale = s["kv"].index_select(1, s["pages"]), s["scale"].index_select(1, s["pages"])
    torch.mul(codes, scale.unsqueeze(-1), out=s["values"])
    return {"q": q, "values": s["values"], "scale": scale}


def _norm(x, w, offset, eps):
    x = x.float()
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * (offset + w.float())


def _rotate(x, s):
    """x fp32 [tokens, heads, 256], its first dims turned by the tokens' angles."""
    rot = s["case"]["rot"]
    if rot == 0:
        return x
    angle = (s["positions"].double()[s["axis"]] * s["freq"][:, None]).t()[:, None]
    c, n = angle.cos().float(), angle.sin().float()
    if s["case"]["pairing"] == "half":
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        return torch.cat((a * c - b * n, b * c + a * n, x[..., rot:]), -1)
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    return torch.cat((torch.stack((a * c - b * n, b * c + a * n), -1).flatten(-2), x[..., rot:]), -1)


def _rope_plain(s):
    off, eps = s["case"]["offset"], s["eps"]
    return {"q": _rotate(_norm(s["q"], s["qw"], off, eps), s).bfloat16(),
            "k": _rotate(_norm(s["k"], s["kw"], off, eps), s).bfloat16()}


def _quantise(x):
    scale = x.abs().amax(-1) / 127
    return torch.round(x / torch.where(scale > 0, scale, 1.0)[..., None]).to(torch.int8), scale


def _append_plain(s):
    off, eps = s["case"]["offset"], s["eps"]
    q = _rotate(_norm(s["q"], s["qw"], off, eps), s).bfloat16()
    k = _rotate(_norm(s["k"], s["kw"], off, eps), s)
    page, slot = s["slots"]
    codes, scale = _quantise(torch.stack((k, s["v"].float())))
    s["kv"][:, page, slot] = codes
    s["scale"][:, page, slot] = scale
    return _written(s, q)


def _shared_plain(s):
    c, q = s["case"], s["q"].float()
    n, hq, hkv, P = c["seqs"], c["hq"], c["hkv"], c["prefix"]
    bt, t = s["block_table"].long(), s["n_ctx"] - 1
    lo = (t // PAGE + 1 - c["win"]).clamp_min(0) if c["win"] > 0 else torch.zeros_like(t)
    # the prefix: [kv heads, keys, 256], one product for all sequences
    K, V = (s["kv"][:, bt[0, : P // PAGE]].float() * s["scale"][:, bt[0, : P // PAGE], :, :, None]).view(
        2, P, hkv, D).transpose(1, 2)
    qh = q.view(n, hkv, hq // hkv, D)
    sp = torch.matmul(qh.transpose(0, 1).reshape(hkv, -1, D), K.transpose(1, 2)).view(hkv, n, hq // hkv, P)
    blk = torch.arange(P, device=q.device) // PAGE
    seen = (blk < c["sink"]) | (blk >= lo[:, None])
    sp = (sp * s["sm_scale"]).masked_fill_(~seen[None, :, None], -math.inf)
    # the sequences' own keys, padded to the longest: [sequences, kv heads, keys, 256]
    own_pages = bt[:, P // PAGE:].clamp_min(0)
    L = own_pages.shape[1] * PAGE
    Ks, Vs = (s["kv"][:, own_pages].float() * s["scale"][:, own_pages, :, :, None]).view(
        2, n, L, hkv, D).transpose(2, 3)
    ss = torch.matmul(qh, Ks.transpose(2, 3)) * s["sm_scale"]
    tok = P + torch.arange(L, device=q.device)
    seen = (tok <= t[:, None]) & ((tok // PAGE < c["sink"]) | (tok // PAGE >= lo[:, None]))
    ss = ss.masked_fill_(~seen[:, None, None], -math.inf).transpose(0, 1)
    m = torch.maximum(sp.amax(-1), ss.amax(-1))[..., None]
    ep, es = (sp - m).exp_(), (ss - m).exp_()
    total = ep.sum(-1) + es.sum(-1)
    o = torch.matmul(ep.view(hkv, -1, P), V).view(hkv, n, hq // hkv, D)
    o = o + torch.matmul(es.transpose(0, 1), Vs).transpose(0, 1)
    return (o / total[..., None]).transpose(0, 1).reshape(n, hq, D).bfloat16()


# ---------------------------------------------------------------- definitions in 64 bits
def _exact_rows(s, x, w):
    """Normed and turned rows: every pair as one complex number times a unit one."""
    c = s["case"]
    x = x.double()
    y = x / (x.pow(2).sum(-1, keepdim=True) / D + s["eps"]).sqrt() * (w.double() + c["offset"])
    half = c["rot"] // 2
    if half == 0:
        return y
    pos = s["positions"].double()
    theta = torch.stack([pos[int(a)] * float(f) for a, f in zip(s["pair_axis"], s["inv_freq"])], -1)
    head = y[..., : c["rot"]]
    pairs = head.unflatten(-1, (2, half)).transpose(-1, -2) if c["pairing"] == "half" else head.unflatten(-1, (half, 2))
    z = torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.ones_like(theta), theta)[:, None]
    back = torch.view_as_real(z)
    back = (back.transpose(-1, -2) if c["pairing"] == "half" else back).flatten(-2)
    y = y.clone()
    y[..., : c["rot"]] = back
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return {"q": _exact_rows(s, s["q"], s["qw"]), "k": _exact_rows(s, s["k"], s["kw"])}
    if case["op"] == "append":
        values = s["kv"].double() * s["scale"].double()[..., None]
        scale = s["scale"].double()
        page, slot = s["slots"]
        for i, rows in enumerate((_exact_rows(s, s["k"], s["kw"]), s["v"].double())):
            step = rows.abs().max(-1).values / 127
            scale[i, page, slot] = step
            step = step[..., None].clamp_min(1e-300)
            values[i, page, slot] = (rows / step).round() * step
        return {"q": _exact_rows(s, s["q"], s["qw"]), "values": values[:, s["pages"]], "scale": scale[:, s["pages"]]}
    # one sequence at a time over its visible keys
    hq, hkv, out = case["hq"], case["hkv"], []
    for i in range(case["seqs"]):
        t = int(s["seqs"][i, 1])
        j = torch.arange(t + 1, device="cuda")
        if case["win"] > 0:
            b = j // PAGE
            j = j[(b < case["sink"]) | (b > t // PAGE - case["win"])]
        page = s["block_table"][i].long()[j // PAGE]
        kv = s["kv"][:, page, j % PAGE].double() * s["scale"][:, page, j % PAGE].double()[..., None]
        q = s["q"][i].double().view(hkv, hq // hkv, D) * s["sm_scale"]
        p = torch.softmax(q @ kv[0].permute(1, 2, 0), -1)
        out.append((p @ kv[1].transpose(0, 1)).reshape(hq, D))
    return torch.stack(out)
