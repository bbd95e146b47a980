"""GPU: decode of a batch that shares a prefix (pa_decode_shared), against the
definition in 64 bits."""
import numpy as np
import pytest

from shared_testutil import Batch

pytestmark = pytest.mark.gpu


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def to_device(b):
    import torch
    return dict(q=dev(b.q.view(np.int16)).view(torch.bfloat16), kp=dev(b.k_pool), vp=dev(b.v_pool),
                ks=dev(b.k_scale), vs=dev(b.v_scale), bt=dev(b.block_table))


class Handle:
    """A handle whose calls compute the prefix once (most batches here are so small that by size they would not)."""

    def __init__(self, b, prefix_pass=1, **opts):
        import windowed_prefill_attention_gb300 as pa
        self.pa, self.h = pa, pa.pa_create(b.hq, b.hkv, b.n_pool, b.max_pages, **opts)
        pa.pa_debug_decode_shared_pass(self.h, prefix_pass)

    def __enter__(self):
        return self.h

    def __exit__(self, *_):
        self.pa.pa_destroy(self.h)


def call(h, b, d, out=None, seqs=None, stream=None, **over):
    import torch

    import windowed_prefill_attention_gb300 as pa
    out = torch.full_like(d["q"], float("nan")) if out is None else out
    a = {**d, **over}
    pa.pa_decode_shared(h, b.seqs if seqs is None else seqs, b.prefix, a["q"], a["kp"], a["vp"], a["ks"], a["vs"],
                        a["bt"], b.S, b.W, b.sm_scale, out, stream=stream)
    return out


def check(b, out, skip_pages=(), only=None):
    got = out.float().cpu().numpy().astype(np.float64)
    ref, bound = b.reference(skip_pages, only)
    err = np.abs(got[b.rows if only is None else b.rows[list(only)]] - ref)
    assert np.all(err <= bound), float((err / bound).max())
    others = np.setdiff1d(np.arange(got.shape[0]), b.rows)
    assert np.isnan(got[others]).all(), "a row of no sequence was written"


# Up to 128 query rows a kv head (sequences x q heads a kv head) are one CTA's, more a pair's in groups of 256.
CASES = {
    "two_blocks": Batch(8, 1, 16, (1, 1), 1, 0, 1),
    "one_tile": Batch(8, 2, 128, (5, 17, 40), 1, 0, 2),
    "ragged_tile": Batch(16, 2, 144, (1, 300, 16, 31), 1, 0, 3),
    "full_group": Batch(8, 1, 2048, tuple(range(1, 17)), 0, 0, 4),
    "one_row_too_many": Batch(8, 1, 2048, tuple(range(1, 18)), 0, 0, 23),
    "two_ctas": Batch(16, 2, 1040, tuple(1 + 7 * i for i in range(17)), 1, 0, 5),
    "many_rows": Batch(8, 2, 4096, tuple(1 + (37 * i) % 90 for i in range(130)), 1, 0, 6),
    "long_prefix": Batch(8, 1, 20000, (1, 100, 2000), 1, 0, 7),
    "long_prefix_pair": Batch(8, 1, 20000, tuple(1 + 19 * i for i in range(33)), 1, 0, 24),
    "ragged_pair": Batch(2, 2, 1232, tuple(1 + i % 37 for i in range(129)), 1, 0, 25),
    "gqa1": Batch(4, 4, 1600, (3, 33, 64), 1, 0, 8),
    "gqa2": Batch(4, 2, 800, tuple(2 + i for i in range(70)), 1, 0, 9),
    "gqa4_windowed": Batch(8, 2, 3200, tuple(1 + 53 * i for i in range(40)), 1, 64, 10),
    "kv_heads_8": Batch(8, 8, 2000, (10, 1, 500), 2, 0, 11),
    "window_hides_prefix": Batch(8, 1, 640, (700, 900, 2000), 0, 16, 12),
    "window_hides_some": Batch(8, 2, 640, (1, 900, 30, 300, 641), 0, 24, 13),
    "sink_past_prefix": Batch(8, 1, 32, (1, 700, 90, 1500), 5, 8, 14),
    "sink_only": Batch(16, 2, 1600, tuple(2000 + 31 * i for i in range(20)), 2, 32, 15),
    "one_sequence": Batch(8, 2, 3200, (77,), 1, 0, 16),
    "one_sequence_windowed": Batch(8, 2, 3200, (77,), 1, 20, 17),
    "no_prefix": Batch(8, 2, 0, (77, 1, 2500, 16), 1, 0, 18),
    "long_own": Batch(8, 2, 256, (9000, 1, 3000), 1, 0, 19),
    "over_512": Batch(2, 1, 320, tuple(1 + (13 * i) % 40 for i in range(1030)), 1, 0, 20),
    "one_chunk_a_row": Batch(8, 2, 16, tuple(1 + i % 40 for i in range(200)), 1, 0, 27),
    "many_ctas": Batch(8, 8, 16, tuple(1 + i % 50 for i in range(200)), 1, 0, 28),
    "cold_softmax": Batch(8, 1, 1024, (9, 90, 3), 1, 0, 21, outliers=0.0, sm_scale=0.0),
    "steep_softmax": Batch(8, 1, 1024, (9, 90, 3), 1, 0, 22, outliers=0.05, sm_scale=2.0),
    "steep_softmax_pair": Batch(8, 1, 2560, tuple(1 + i for i in range(40)), 1, 0, 26, outliers=0.05, sm_scale=2.0),
}


@pytest.mark.parametrize("prefix_pass", (1, 0))
@pytest.mark.parametrize("case", sorted(CASES))
def test_matches_the_definition(case, prefix_pass):
    import windowed_prefill_attention_gb300 as pa
    b = CASES[case].make()
    with Handle(b, prefix_pass) as h:
        out = call(h, b, to_device(b))
        assert pa.pa_last_error(h) == 0
    check(b, out)


def test_passes_by_size_agree():
    """Batches on both sides of the rule, each call's bits those of the pass that the rule names."""
    import torch

    import windowed_prefill_attention_gb300 as pa
    for b, by_size in ((Batch(16, 2, 1024, (5, 40, 17), 1, 0, 31), 0),
                       (Batch(8, 4, 4096, tuple(1 + 3 * i for i in range(40)), 1, 0, 32), 1),
                       (Batch(8, 4, 2048, tuple(1 + 3 * i for i in range(80)), 1, 0, 33), 1)):
        b.make()
        d = to_device(b)
        runs, _ = pa.pa_decode_shared_plan(b.hq, b.hkv, b.max_pages, 152, b.seqs, b.prefix, b.S, b.W)
        assert (len(runs) > 0) == by_size
        outs = []
        for prefix_pass in (-1, by_size):
            with Handle(b, prefix_pass) as h:
                outs.append(call(h, b, d))
                assert pa.pa_last_error(h) == 0
        check(b, outs[0])
        assert torch.equal(*(o.view(torch.int16) for o in outs))


@pytest.mark.parametrize("prefix_pass", (1, 0))
def test_scales_of_every_magnitude(prefix_pass):
    """K and V scales over many powers of two (falling and rising along the keys, zero among them)."""
    import windowed_prefill_attention_gb300 as pa
    b = Batch(8, 2, 1536, (40, 5, 333), 1, 0, 30).make()
    rng = np.random.default_rng(1)
    for s in (b.k_scale, b.v_scale):
        with np.errstate(invalid="ignore"):
            s *= (2.0 ** rng.integers(-9, 3, s.shape)).astype(np.float32)
    b.v_scale[b.block_table[0, 5]] = 0
    b.v_scale[b.block_table[0, :4]] *= np.float32(2.0 ** -40)
    with Handle(b, prefix_pass) as h:
        out = call(h, b, to_device(b))
        assert pa.pa_last_error(h) == 0
    check(b, out)


def test_equals_decode_and_repeats_bit_for_bit():
    """pa_decode on the same batch, its table with the prefix's pages in every row, agrees to the roundings; calls
    of other sizes in between do not change a call's bits."""
    import torch

    import windowed_prefill_attention_gb300 as pa
    b = CASES["two_ctas"].make()
    d = to_device(b)
    with Handle(b) as h:
        first = call(h, b, d)
        few = call(h, b, d, seqs=b.seqs[:3])
        again = call(h, b, d)
        few2 = call(h, b, d, seqs=b.seqs[:3])
        assert pa.pa_last_error(h) == 0
        full = b.block_table.copy()
        full[:, : b.prefix // 16] = full[0, : b.prefix // 16]
        ref = torch.full_like(first, float("nan"))
        pa.pa_decode(h, b.seqs, d["q"], d["kp"], d["vp"], d["ks"], d["vs"], dev(full), b.S, b.W, b.sm_scale, ref)
        assert pa.pa_last_error(h) == 0
    bits = lambda t: t.view(torch.int16)  # noqa: E731
    assert torch.equal(bits(first), bits(again)) and torch.equal(bits(few), bits(few2))
    _, bound = b.reference()
    diff = (first - ref).float()[torch.from_numpy(b.rows).cuda()].abs().cpu().numpy()
    assert np.all(diff <= 2 * bound)


@pytest.mark.parametrize("prefix_pass", (1, 0))
def test_bad_pages_are_skipped_and_reported(prefix_pass):
    """A prefix entry outside the pool: its keys leave every sequence's softmax; an own entry: that sequence's."""
    import windowed_prefill_attention_gb300 as pa
    b = CASES["ragged_tile"].make()
    d = to_device(b)
    gone = [int(b.block_table[0, 3]), int(b.block_table[1, b.prefix // 16 + 2])]
    b.block_table[0, 3], b.block_table[1, b.prefix // 16 + 2] = b.n_pool, -1
    with Handle(b, prefix_pass) as h:
        out = call(h, b, d, bt=dev(b.block_table))
        assert pa.pa_last_error(h) == pa.PA_EBADPAGE
        assert pa.pa_last_error(h) == 0
    b.block_table[0, 3], b.block_table[1, b.prefix // 16 + 2] = gone
    check(b, out, skip_pages=gone)


def test_captured_graphs_outlive_a_growing_workspace():
    """A graph of a small batch replays correctly after a larger call has outgrown the handle's buffers; a call
    that would have to grow them inside a capture is refused."""
    import torch

    import windowed_prefill_attention_gb300 as pa
    b = CASES["many_rows"].make()
    d = to_device(b)
    small = b.seqs[:4]
    side = torch.cuda.Stream()
    with Handle(b) as h:
        want = call(h, b, d, seqs=small)
        torch.cuda.synchronize()
        out = torch.zeros_like(d["q"])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            call(h, b, d, out=out, seqs=small)
            with pytest.raises(pa.PAError) as e:
                call(h, b, d, out=out)
            assert e.value.code == pa.PA_ENOMEM
        big = call(h, b, d)
        check(b, big)
        for _ in range(2):
            g.replay()
        torch.cuda.synchronize()
        assert pa.pa_last_error(h) == 0
        rows = torch.from_numpy(b.rows[:4]).cuda()
        assert torch.equal(out[rows], want[rows])


def test_on_a_side_stream_and_shapes_are_checked():
    import torch
    b = CASES["gqa2"].make()
    d = to_device(b)
    side = torch.cuda.Stream()
    with Handle(b) as h:
        out = torch.full_like(d["q"], float("nan"))
        torch.cuda.synchronize()
        call(h, b, d, out=out, stream=side)
        side.synchronize()
        check(b, out)
        for bad in (dict(q=d["q"][:, :2].contiguous()), dict(kp=d["kp"][:-1]), dict(bt=d["bt"][:, :-1].contiguous()),
                    dict(bt=d["bt"][:5]), dict(vs=d["vs"][..., :1].contiguous()), dict(q=d["q"][:3])):
            with pytest.raises(ValueError):
                call(h, b, d, out=out, **bad)


@pytest.mark.parametrize("prefix_pass", (1, 0))
def test_in_place_and_overlapping_outputs(prefix_pass):
    import torch

    import windowed_prefill_attention_gb300 as pa
    b = CASES["two_ctas"].make()
    d = to_device(b)
    rows = torch.from_numpy(b.rows).cuda()
    with Handle(b, prefix_pass) as h:
        want = call(h, b, d)[rows]
        q = d["q"].clone()
        call(h, b, d, q=q, out=q)
        assert torch.equal(q[rows].view(torch.int16), want.view(torch.int16))
        both = torch.empty(2 * d["q"].shape[0] - 1, *d["q"].shape[1:], dtype=torch.bfloat16, device="cuda")
        n = d["q"].shape[0]
        with pytest.raises(pa.PAError) as e:
            call(h, b, d, q=both[:n], out=both[n - 1:])
        assert e.value.code == pa.PA_EINVAL and pa.pa_last_error(h) == 0


def test_two_handles_on_two_streams_at_once():
    """Batches of all forms, each handle's calls on its own stream, beside one another."""
    import torch

    import windowed_prefill_attention_gb300 as pa
    work = []
    for case, prefix_pass in (("long_prefix", 1), ("many_rows", 1), ("gqa4_windowed", 0), ("long_own", 1)):
        b = CASES[case].make()
        d = to_device(b)
        h = pa.pa_create(b.hq, b.hkv, b.n_pool, b.max_pages)
        pa.pa_debug_decode_shared_pass(h, prefix_pass)
        work.append((h, b, d, call(h, b, d), torch.cuda.Stream(), []))
    torch.cuda.synchronize()
    for _ in range(40):
        for h, b, d, _, stream, outs in work:
            outs.append(torch.empty_like(d["q"]))
            call(h, b, d, out=outs[-1], stream=stream)
    torch.cuda.synchronize()
    for h, b, _, want, _, outs in work:
        assert pa.pa_last_error(h) == 0
        pa.pa_destroy(h)
        rows = torch.from_numpy(b.rows).cuda()
        assert all(torch.equal(o[rows].view(torch.int16), want[rows].view(torch.int16)) for o in outs)


def test_calls_back_to_back_of_changing_sizes():
    """Calls back to back on one stream, of changing sizes, without a synchronisation between them."""
    import windowed_prefill_attention_gb300 as pa
    b = CASES["many_rows"].make()
    d = to_device(b)
    with Handle(b) as h:
        sizes = (130, 3, 17, 64, 130, 1, 33)
        outs = [call(h, b, d, seqs=b.seqs[:n]) for n in sizes]
        assert pa.pa_last_error(h) == 0
        for n, o in zip(sizes, outs):
            alone = call(h, b, d, seqs=b.seqs[:n])
            assert pa.pa_last_error(h) == 0
            import torch
            assert torch.equal(o.view(torch.int16), alone.view(torch.int16))


def short_first_segment(hq, n, from_prefix):
    """The first prefix from this one on whose split has a unit with two groups or more, the first of them short."""
    import windowed_prefill_attention_gb300 as pa
    for prefix in range(from_prefix, from_prefix + 8192, 64):
        b = Batch(hq, 8, prefix, (1,) * n if n > 100 else tuple(1 + i for i in range(n)), 1, 0, 50)
        seqs = [(i, prefix + s - 1, 1, prefix + s) for i, s in enumerate(b.suffix)]
        runs, _ = pa.pa_decode_shared_plan(hq, 8, 4096, 152, seqs, prefix, b.S, b.W, 1)
        segs = {}  # tiles of eight blocks
        for r in runs.tolist():
            segs.setdefault(r[0], []).append((r[7] - r[6] + 7) // 8)
        if any(len(s) > 1 and s[0] <= 2 for s in segs.values()):
            return b.make()
    raise AssertionError("no such split")


@pytest.mark.parametrize("hq, n, from_prefix", ((8, 3, 8192), (8, 3, 14384), (8, 3, 19712), (8, 101, 9216), (64, 17, 6144),
                                                (64, 17, 9600)))
def test_units_that_begin_with_a_short_segment(hq, n, from_prefix):
    """Units whose first group ends after a tile or two: the next one's queries, K and V come in while the first
    one's are on their way (with 101 sequences of one row a head, 101 copies a group)."""
    import torch

    import windowed_prefill_attention_gb300 as pa
    b = short_first_segment(hq, n, from_prefix)
    first = None
    for _ in range(20):
        d = to_device(b)
        with Handle(b) as h:
            out = call(h, b, d)
            assert pa.pa_last_error(h) == 0
        if first is None:
            first = out
            check(b, out, only=range(0, n, max(1, n // 5)))
        assert torch.equal(out.view(torch.int16), first.view(torch.int16))


@pytest.mark.parametrize("case", ("long_prefix", "long_prefix_pair"))
def test_first_calls_on_cold_memory_repeat_bit_for_bit(case):
    """Fresh handles, fresh copies of the inputs, other data in the freed memory in between: codes that arrive
    late must not let any part of the kernel run ahead of another."""
    import torch

    import windowed_prefill_attention_gb300 as pa
    b = CASES[case].make()
    first = None
    for i in range(100):
        d = to_device(b)
        with Handle(b) as h:
            out = call(h, b, d)
            assert pa.pa_last_error(h) == 0
        if first is None:
            first = out
            check(b, out)
        assert torch.equal(out.view(torch.int16), first.view(torch.int16)), i
        if i % 7 == 6:
            del d
            junk = torch.empty(1 << 27, dtype=torch.uint8, device="cuda").random_()
            del junk
            torch.cuda.empty_cache()


@pytest.mark.parametrize("prefix_pass", (1, 0))
def test_append_then_shared_decode(prefix_pass):
    """A layer's step as a serving loop runs it: the prefix appended once, each sequence's own tokens in one batched
    append, a decode step of the batch, against the definition on the pool the calls wrote."""
    import torch

    import windowed_prefill_attention_gb300 as pa
    b = Batch(16, 2, 208, (1, 20, 16, 37, 5), 1, 0, 40).make()
    ctx = b.seqs[:, 3]
    own = np.array(b.suffix)
    first = b.prefix + np.cumsum(own) - own
    tok = b.prefix + int(own.sum())
    x = torch.randn(tok, 20 * 256, device="cuda", generator=torch.Generator("cuda").manual_seed(3)).bfloat16()
    q, k, v = x[:, :4096].view(tok, 16, 256), x[:, 4096:4608].view(tok, 2, 256), x[:, 4608:].view(tok, 2, 256)
    w = torch.ones(256, device="cuda", dtype=torch.bfloat16)
    rope = pa.pa_rope_init(10000.0 ** (-np.arange(32) / 32.0))
    kp, vp = (torch.zeros(b.n_pool, 16, 2, 256, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((b.n_pool, 16, 2), float("nan"), device="cuda") for _ in range(2))
    bt, qo = dev(b.block_table), torch.empty(tok, 16, 256, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(qo, float("nan"))
    with Handle(b, prefix_pass) as h:
        for seqs in ([(0, 0, b.prefix, b.prefix)], [(f, b.prefix, m, c) for f, m, c in zip(first, own, ctx)]):
            pa.pa_qkv_append(h, seqs, q, k, v, w, w, 1e-6, rope, None, bt, kp, vp, ks, vs, qo)
        last = first + own - 1
        pa.pa_decode_shared(h, [(r, c - 1, 1, c) for r, c in zip(last, ctx)], b.prefix, qo, kp, vp, ks, vs, bt, b.S,
                            b.W, b.sm_scale, out)
        assert pa.pa_last_error(h) == 0
    b.k_pool, b.v_pool, b.k_scale, b.v_scale = (t.cpu().numpy() for t in (kp, vp, ks, vs))
    b.q = qo.view(torch.int16).cpu().numpy().view(np.uint16)
    b.rows = last
    check(b, out)
