"""GPU: norm + rotation (pa_qk_norm_rope) and the batched append of a layer's
projected rows (pa_qkv_append), against their formulas in 64 bits."""
import numpy as np
import pytest

import oracle
import qkv_testutil as ut
from pa_testutil import norm_errors

pytestmark = pytest.mark.gpu


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def dev_bf16(bits):
    import torch
    return dev(bits.view(np.int16)).view(torch.bfloat16)


def normal_bits(rng, *shape, scale=1.0):
    return ut.bf16_bits(rng.standard_normal(shape).astype(np.float32) * scale)


class Handle:
    def __init__(self, hq, hkv, n_pool=1, max_pages=1):
        import windowed_prefill_attention_gb300 as pa
        self.pa, self.h = pa, pa.pa_create(hq, hkv, n_pool, max_pages)

    def __enter__(self):
        return self.h

    def __exit__(self, *_):
        self.pa.pa_destroy(self.h)


# tokens, q heads, kv heads, rotated dims, halves, axes, fused buffer, weights, offset, first position
CASES = {
    "one_token": (1, 16, 2, 64, True, 1, True, True, 0.0, 4095),
    "two_tokens_one_head": (2, 1, 1, 256, True, 1, False, True, 1.0, 0),
    "norm_only": (37, 4, 1, 0, True, 1, False, True, 1.0, 0),
    "no_gain": (19, 4, 4, 32, False, 1, False, False, 0.0, 77),
    "halves_256": (333, 16, 2, 256, True, 1, True, True, 0.0, 131000),
    "adjacent_256": (130, 8, 4, 256, False, 1, False, True, 1.0, 65000),
    "three_axes": (1029, 8, 4, 96, False, 3, True, True, 1.0, 12345),
    "four_axes_halves": (257, 10, 5, 240, True, 4, False, True, 0.0, 3),
    "wide_group": (65, 128, 1, 16, True, 1, False, True, 0.0, 9),
    "eight_kv_heads": (2500, 8, 8, 128, True, 2, True, True, 0.0, 100),
    "far_positions": (50, 4, 2, 128, True, 1, False, True, 0.0, 2 ** 31 - 60),
    "negative_positions": (50, 4, 2, 128, False, 2, False, True, 0.0, -2 ** 31),
}


def make_case(case, seed):
    n, hq, hkv, rot, halves, axes, fused, weights, off, start = CASES[case]
    rng = np.random.default_rng(seed)
    import windowed_prefill_attention_gb300 as pa
    freq, axis = ut.frequencies(rot), (np.arange(rot // 2) * axes // max(1, rot // 2)).astype(np.int32)
    rope = pa.pa_rope_init(freq, pa.PA_ROPE_HALF if halves else pa.PA_ROPE_ADJACENT, axis)
    pos = np.stack([start + np.arange(n) // (a + 1) for a in range(axes)]).astype(np.int32)
    if fused:  # one projection's rows: query and gate side by side per head, then keys, then values
        x = normal_bits(rng, n, 2 * hq + 2 * hkv, 256, scale=1.7)
        x[n // 2, : 2 * hq: 2] = 0  # a token whose query rows are all zero
        t = dev_bf16(x)
        q, k, v = t[:, : 2 * hq].unflatten(1, (hq, 2))[:, :, 0], t[:, 2 * hq: 2 * hq + hkv], t[:, 2 * hq + hkv:]
        qb, kb, vb = x[:, : 2 * hq: 2], x[:, 2 * hq: 2 * hq + hkv], x[:, 2 * hq + hkv:]
    else:
        qb, kb, vb = (normal_bits(rng, n, h, 256, scale=s) for h, s in ((hq, 1.0), (hkv, 30.0), (hkv, 0.01)))
        q, k, v = dev_bf16(qb), dev_bf16(kb), dev_bf16(vb)
    w = [normal_bits(rng, 256, scale=0.2) if weights else None for _ in range(2)]
    return dict(n=n, hq=hq, hkv=hkv, freq=freq, axis=axis, rope=rope, pos=pos, q=q, k=k, v=v, qb=qb, kb=kb, vb=vb,
                w=w, off=off, eps=1e-6, halves=halves)


def reference(c, bits, w):
    return ut.norm_rope(ut.bf16_values(bits), None if w is None else ut.bf16_values(w), c["off"], c["eps"], c["freq"],
                        c["axis"], c["pos"], c["halves"])


def call_rope(h, c, q_out, k_out, **over):
    import windowed_prefill_attention_gb300 as pa
    a = dict(q=c["q"], k=c["k"], positions=dev(c["pos"]))
    a.update(over)
    w = [None if x is None else dev_bf16(x) for x in c["w"]]
    pa.pa_qk_norm_rope(h, a["q"], a["k"], w[0], w[1], c["eps"], c["rope"], a["positions"], q_out, k_out,
                       weight_offset=c["off"], stream=a.get("stream"))


def empty_rows(n, heads):
    import torch
    return torch.full((n, heads, 256), float("nan"), dtype=torch.bfloat16, device="cuda")


@pytest.mark.parametrize("case", sorted(CASES))
def test_norm_rope_matches_the_formula(case):
    c = make_case(case, 11)
    qo, ko = empty_rows(c["n"], c["hq"]), empty_rows(c["n"], c["hkv"])
    with Handle(c["hq"], c["hkv"]) as h:
        call_rope(h, c, qo, ko)
        ut.assert_rows(qo.float().cpu().numpy(), *reference(c, c["qb"], c["w"][0]), what="q")
        ut.assert_rows(ko.float().cpu().numpy(), *reference(c, c["kb"], c["w"][1]), what="k")


def test_norm_rope_one_kind_in_place_and_another_stream():
    """Only queries, only keys, in place and on a side stream give the bits of the whole call."""
    import torch
    c = make_case("adjacent_256", 12)
    with Handle(c["hq"], c["hkv"]) as h:
        qo, ko = empty_rows(c["n"], c["hq"]), empty_rows(c["n"], c["hkv"])
        call_rope(h, c, qo, ko)
        q2, k2 = empty_rows(c["n"], c["hq"]), empty_rows(c["n"], c["hkv"])
        call_rope(h, c, q2, None, k=None)
        call_rope(h, c, None, k2, q=None)
        assert torch.equal(qo, q2) and torch.equal(ko, k2)
        q3, k3 = c["q"].clone(), c["k"].clone()
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        call_rope(h, c, q3, k3, q=q3, k=k3, stream=side)
        side.synchronize()
        assert torch.equal(qo, q3) and torch.equal(ko, k3)


def test_norm_rope_in_place_over_many_items():
    """More tokens than warps, so that a warp's next rows are on their way while it writes others: in place gives
    the bits of the call into other rows, and each token's those of a call of its own."""
    import torch

    import windowed_prefill_attention_gb300 as pa
    g = torch.Generator("cuda").manual_seed(5)
    n, hq, hkv = 9001, 10, 5
    q, k = (torch.randn(n, h, 256, device="cuda", generator=g).bfloat16() for h in (hq, hkv))
    rope = pa.pa_rope_init(ut.frequencies(96), pa.PA_ROPE_ADJACENT)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    qo, ko = empty_rows(n, hq), empty_rows(n, hkv)
    with Handle(hq, hkv) as h:
        pa.pa_qk_norm_rope(h, q, k, None, None, 1e-6, rope, pos, qo, ko)
        for i in (0, 4000, n - 1):
            q1, k1 = empty_rows(1, hq), empty_rows(1, hkv)
            pa.pa_qk_norm_rope(h, q[i:i + 1], k[i:i + 1], None, None, 1e-6, rope, pos[i:i + 1], q1, k1)
            assert torch.equal(q1[0], qo[i]) and torch.equal(k1[0], ko[i])
        pa.pa_qk_norm_rope(h, q, k, None, None, 1e-6, rope, pos, q, k)
        assert torch.equal(q, qo) and torch.equal(k, ko)


def test_norm_rope_broadcast_rows_zero_rows_and_no_tokens():
    """Rows at stride 0 (one row for all tokens and heads), rows of zeros with eps 0, an empty call."""
    import torch

    import windowed_prefill_attention_gb300 as pa
    rng = np.random.default_rng(3)
    bits = normal_bits(rng, 1, 1, 256)
    q = dev_bf16(bits).expand(9, 4, 256)
    pos = np.arange(9, dtype=np.int32)
    freq = ut.frequencies(64)
    out = empty_rows(9, 4)
    with Handle(4, 2) as h:
        pa.pa_qk_norm_rope(h, q, None, None, None, 0.0, pa.pa_rope_init(freq), dev(pos), out, None)
        ref = ut.norm_rope(np.broadcast_to(ut.bf16_values(bits), (9, 4, 256)), None, 0, 0.0, freq, None, pos[None])
        ut.assert_rows(out.float().cpu().numpy(), *ref)
        zero = torch.zeros(9, 4, 256, dtype=torch.bfloat16, device="cuda")
        pa.pa_qk_norm_rope(h, zero, None, None, None, 0.0, pa.pa_rope_init(freq), dev(pos), out, None)
        assert torch.equal(out, zero)
        pa.pa_qk_norm_rope(h, zero[:0], None, None, None, 0.0, None, None, out[:0], None)
        with pytest.raises(ValueError):  # the handle's query heads, not the tensor's
            pa.pa_qk_norm_rope(h, zero[:, :2], None, None, None, 0.0, None, None, out[:, :2], None)
        with pytest.raises(ValueError):
            pa.pa_qk_norm_rope(h, zero, None, None, None, 0.0, pa.pa_rope_init(freq), dev(pos[:8]), out, None)


def test_norm_rope_captured_and_replayed_on_new_rows():
    import torch
    c = make_case("halves_256", 13)
    with Handle(c["hq"], c["hkv"]) as h:
        q, k, pos = c["q"].contiguous(), c["k"].contiguous(), dev(c["pos"])
        want_q, want_k = empty_rows(c["n"], c["hq"]), empty_rows(c["n"], c["hkv"])
        call_rope(h, c, want_q, want_k)
        qo, ko = empty_rows(c["n"], c["hq"]), empty_rows(c["n"], c["hkv"])
        q_in, k_in = torch.zeros_like(q), torch.zeros_like(k)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        w = [dev_bf16(x) for x in c["w"]]
        import windowed_prefill_attention_gb300 as pa
        with torch.cuda.graph(g):
            pa.pa_qk_norm_rope(h, q_in, k_in, w[0], w[1], c["eps"], c["rope"], pos, qo, ko, weight_offset=c["off"])
        q_in.copy_(q)
        k_in.copy_(k)
        for _ in range(2):
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(qo, want_q) and torch.equal(ko, want_k)


# ---------------------------------------------------------------- append
# sequences (row, first position, new tokens); kv heads etc. from the rope case of that name
APPENDS = {
    "one_token": [(0, 4095, 1)],
    "three_axes": [(0, 12, 400), (400, 0, 1), (401, 31, 17), (418, 160, 611)],
    "eight_kv_heads": [(0, 5, 1000), (1000, 0, 1500)],
    "norm_only": [(10, 3, 20), (0, 15, 2), (32, 16, 5)],     # rows out of order, some of no sequence
    "adjacent_256": [(i, (37 * i) % 300, 1) for i in range(130)],
    "wide_group": [(5 * i, 11 * i, 5) for i in range(13)],
    "no_gain": [(0, 0, 19)],
}


def append_inputs(c, seqs, seed):
    rng = np.random.default_rng(seed)
    pages = [(s + n + 15) // 16 for _, s, n in seqs]
    n_pool, max_pages = sum(pages) + 3, max(pages) + 1
    bt = np.full((len(seqs), max_pages), -1, np.int32)
    perm, at = rng.permutation(n_pool), 0
    for i, n in enumerate(pages):
        bt[i, :n] = perm[at:at + n]
        at += n
    kp, vp = (rng.integers(-127, 128, (n_pool, 16, c["hkv"], 256)).astype(np.int8) for _ in range(2))
    ks, vs = (rng.random((n_pool, 16, c["hkv"]), dtype=np.float32) for _ in range(2))
    desc = np.array([(r, s, n, s + n) for r, s, n in seqs], np.int32)
    return dict(bt=bt, kp=kp, vp=vp, ks=ks, vs=vs, desc=desc, n_pool=n_pool, max_pages=max_pages)


def call_append(h, c, a, positions, bt=None, q=True):
    import windowed_prefill_attention_gb300 as pa
    pool = [dev(a[k]) for k in ("kp", "vp", "ks", "vs")]
    qo = empty_rows(c["n"], c["hq"]) if q else None
    w = [None if x is None else dev_bf16(x) for x in c["w"]]
    pa.pa_qkv_append(h, a["desc"], c["q"] if q else None, c["k"], c["v"], w[0], w[1], c["eps"], c["rope"], positions,
                     dev(a["bt"] if bt is None else bt), *pool, qo, weight_offset=c["off"])
    rc = pa.pa_last_error(h)
    return qo, [t.cpu().numpy() for t in pool], rc


@pytest.mark.parametrize("own_positions", [False, True])
@pytest.mark.parametrize("case", sorted(APPENDS))
def test_append_matches_the_formula(case, own_positions):
    c, seqs = make_case(case, 21), APPENDS[case]
    a = append_inputs(c, seqs, 5)
    rows = np.concatenate([r + np.arange(n) for r, _, n in seqs])
    if own_positions:  # without a positions array every axis takes the token's own
        for r, s, n in seqs:
            c["pos"][:, r:r + n] = s + np.arange(n)
    with Handle(c["hq"], c["hkv"], a["n_pool"], a["max_pages"]) as h:
        qo, (kp, vp, ks, vs), rc = call_append(h, c, a, None if own_positions else dev(c["pos"]))
    assert rc == 0
    got = qo.float().cpu().numpy()
    ref, mag = reference(c, c["qb"], c["w"][0])
    ut.assert_rows(got[rows], ref[rows], mag[rows], what="q")
    others = np.setdiff1d(np.arange(c["n"]), rows)
    assert np.isnan(got[others]).all(), "rows of no sequence were written"
    ref, mag = reference(c, c["kb"], c["w"][1])
    vc, vsc = oracle.kv_quantize(c["vb"])
    want = {k: a[k].copy() for k in ("vp", "vs")}
    written = np.zeros((a["n_pool"], 16), bool)
    for i, (r, s, n) in enumerate(seqs):
        t = s + np.arange(n)
        page, slot = a["bt"][i, t // 16], t % 16
        ut.assert_codes(kp[page, slot], ks[page, slot], ref[r:r + n], mag[r:r + n], what="k")
        want["vp"][page, slot], want["vs"][page, slot] = vc[r:r + n], vsc[r:r + n]
        written[page, slot] = True
    assert np.array_equal(vp, want["vp"]) and np.array_equal(vs, want["vs"])  # as pa_kv_append, bit for bit
    assert np.array_equal(kp[~written], a["kp"][~written]) and np.array_equal(ks[~written], a["ks"][~written])


def test_append_more_sequences_than_one_launch_takes():
    """1100 sequences of one to three tokens: three launches, ragged."""
    rng = np.random.default_rng(4)
    lens = rng.integers(1, 4, 1100)
    first = np.cumsum(lens) - lens
    seqs = [(int(f), int(s), int(n)) for f, s, n in zip(first, rng.integers(0, 40, 1100), lens)]
    n = int(lens.sum())
    CASES["many"] = (n, 2, 1, 32, True, 1, False, True, 0.0, 0)
    try:
        c = make_case("many", 6)
    finally:
        del CASES["many"]
    a = append_inputs(c, seqs, 7)
    for r, s, k in seqs:
        c["pos"][:, r:r + k] = s + np.arange(k)
    with Handle(2, 1, a["n_pool"], a["max_pages"]) as h:
        qo, (kp, vp, ks, vs), rc = call_append(h, c, a, None)
    assert rc == 0
    ut.assert_rows(qo.float().cpu().numpy(), *reference(c, c["qb"], c["w"][0]))
    ref, mag = reference(c, c["kb"], c["w"][1])
    vc, vsc = oracle.kv_quantize(c["vb"])
    seq = np.repeat(np.arange(1100), lens)
    t = np.concatenate([s + np.arange(k) for _, s, k in seqs])
    page, slot = a["bt"][seq, t // 16], t % 16
    ut.assert_codes(kp[page, slot], ks[page, slot], ref, mag)
    assert np.array_equal(vp[page, slot], vc) and np.array_equal(vs[page, slot], vsc)


def test_append_keys_only_and_bad_pages():
    """Without queries the pool is the same; a page entry outside the pool skips its tokens' keys and values,
    is reported, and leaves queries and other tokens as they are."""
    import windowed_prefill_attention_gb300 as pa
    c, seqs = make_case("three_axes", 22), APPENDS["three_axes"]
    a = append_inputs(c, seqs, 8)
    with Handle(c["hq"], c["hkv"], a["n_pool"], a["max_pages"]) as h:
        qo, pool, rc = call_append(h, c, a, dev(c["pos"]))
        assert rc == 0
        _, pool2, rc = call_append(h, c, a, dev(c["pos"]), q=False)
        assert rc == 0 and all(np.array_equal(x, y) for x, y in zip(pool, pool2))
        bad = a["bt"].copy()
        bad[0, 3], bad[3, 12] = a["n_pool"], -7
        q3, pool3, rc = call_append(h, c, a, dev(c["pos"]), bt=bad)
        assert rc == pa.PA_EBADPAGE and pa.pa_last_error(h) == 0
    import torch
    assert torch.equal(q3.nan_to_num(), qo.nan_to_num())
    keep = np.ones(a["n_pool"], bool)
    keep[[a["bt"][0, 3], a["bt"][3, 12]]] = False
    for x, y, was in zip(pool3, pool, (a["kp"], a["vp"], a["ks"], a["vs"])):
        assert np.array_equal(x[keep], y[keep]) and np.array_equal(x[~keep], was[~keep])


def test_append_then_prefill_and_decode():
    """The step as a user runs it: rows of a fused projection appended, the returned queries attended with, in two
    chunks, then one token decoded, against the definition on the pool the calls wrote."""
    import torch

    import windowed_prefill_attention_gb300 as pa
    n, hq, hkv, S, W = 301, 8, 2, 1, 6
    CASES["step"] = (n, hq, hkv, 64, True, 1, True, True, 1.0, 0)
    try:
        c = make_case("step", 31)
    finally:
        del CASES["step"]
    n_pool = max_pages = (n + 15) // 16
    rng = np.random.default_rng(9)
    bt = rng.permutation(n_pool).astype(np.int32)[None]
    w = [dev_bf16(x) for x in c["w"]]
    kp, vp = (torch.zeros(n_pool, 16, hkv, 256, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(n_pool, 16, hkv, device="cuda") for _ in range(2))
    btd, qo = dev(bt), empty_rows(n, hq)
    out = empty_rows(n, hq)
    with Handle(hq, hkv, n_pool, max_pages) as h:
        for a, b in ((0, 200), (200, n - 1), (n - 1, n)):
            seqs = np.array([(a, a, b - a, b)], np.int32)
            pa.pa_qkv_append(h, seqs, c["q"], c["k"], c["v"], w[0], w[1], c["eps"], c["rope"], None, btd, kp, vp, ks,
                             vs, qo, weight_offset=c["off"])
            step = pa.pa_decode if b - a == 1 else pa.pa_prefill_batch
            step(h, seqs, qo, kp, vp, ks, vs, btd, S, W, 1 / 16, out)
        assert pa.pa_last_error(h) == 0
    from synth.workloads import Inputs, Workload
    wl = Workload("step", hq, hkv, ((0, n),), S, W, seed=0)
    inp = Inputs(wl, qo.view(torch.int16).cpu().numpy().view(np.uint16), kp.cpu().numpy(), vp.cpu().numpy(),
                 ks.cpu().numpy(), vs.cpu().numpy(), bt, np.array([(0, 0, n, n)], np.int32))
    rows = oracle.all_rows(inp)
    ref = oracle.exact(oracle.Problem.from_inputs(inp), rows).reshape(n, hq, 256)
    mx, mean = norm_errors(out.float().cpu().numpy().astype(np.float64), ref)
    assert mx <= 3e-2 and mean <= 1e-2
