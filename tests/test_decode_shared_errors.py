"""GPU: what a bad page entry, an error that was not read, and a short wait limit do
to a shared-prefix decode whose units work on one group for a millisecond and more."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

N, HQ, HKV, PREFIX = 512, 64, 8, 131072


class Long:
    """512 sequences of 64 query heads on 131072 shared keys: 128 groups of 1024 tiles on 76 pairs, so that most units
    go on to a second group after hundreds of tiles."""

    def __init__(self):
        import torch

        import windowed_prefill_attention_gb300 as pa
        self.pa, self.torch = pa, torch
        g = torch.Generator("cuda").manual_seed(3)
        pb = PREFIX // 16
        self.n_pool, self.max_pages = pb + N, pb + 1
        shape = (self.n_pool, 16, HKV, 256)
        self.pool = [torch.randint(-127, 128, shape, dtype=torch.int8, device="cuda", generator=g) for _ in range(2)]
        # small keys: every one of them has a say in every row
        self.scale = [torch.rand(shape[:3], device="cuda", generator=g) * s for s in (2e-3, 2e-2)]
        self.bt = torch.full((N, self.max_pages), -1, dtype=torch.int32, device="cuda")
        self.bt[0, :pb] = torch.randperm(pb, device="cuda", generator=g).int()
        self.bt[:, pb] = pb + torch.arange(N, device="cuda").int()
        self.q = torch.randn(N, HQ, 256, device="cuda", generator=g).bfloat16()
        self.own = 1 + np.arange(N) % 16
        ctx = PREFIX + self.own
        self.seqs = np.stack([np.arange(N), ctx - 1, np.ones_like(ctx), ctx], 1).astype(np.int32)

    def call(self, h, bt=None):
        out = self.torch.full_like(self.q, float("nan"))
        self.pa.pa_decode_shared(h, self.seqs, PREFIX, self.q, *self.pool, *self.scale, self.bt if bt is None else bt, 1,
                                 0, 1 / 16, out)
        return out

    def check(self, s, h, out):
        """A sequence's query head against the definition, within 2^-8 |out| (the bf16 result), 2^-11 sum p |v| (P' in
        fp16), where P' is subnormal half its fixed step, and the scores' fp32 errors e (256 additions of 2^-23 of sum
        |q k|, and 2^-21 of the score for the scale products and the exponent), which move p by 1 + e."""
        torch, g = self.torch, h // (HQ // HKV)
        page = torch.cat((self.bt[0, :-1], self.bt[s, -1:])).long()
        n = PREFIX + int(self.own[s])
        k, v = ((p[page, :, g].double() * c[page, :, g, None].double()).view(-1, 256)[:n]
                for p, c in zip(self.pool, self.scale))
        vs = self.scale[1][page, :, g].double().view(-1)[:n]
        q = self.q[s, h].double() / 16
        score, size = k @ q, k.abs() @ q.abs()
        p = torch.exp(score - score.max())
        tiny = (p * vs / vs.max() < 2.0 ** -13).sum() * 2.0 ** -25 * 2 * vs.max() * 127
        p /= p.sum()
        e = 256 * 2.0 ** -23 * size + 2.0 ** -21 * (score.abs() + score.abs().max() + 2)
        ref, av = p @ v, v.abs()
        bound = 2.0 ** -8 * ref.abs() + (1 + 2.0 ** -8) * (2.0 ** -11 * (p @ av) + tiny + (p * e) @ av + ref.abs() * (p * e).sum())
        err = (out[s, h].double() - ref).abs()
        assert bool((err <= bound).all()), (s, h, float((err / bound).max()))


@pytest.fixture(scope="module")
def long():
    b = Long()
    runs, _ = b.pa.pa_decode_shared_plan(HQ, HKV, b.max_pages, 152, b.seqs, PREFIX, 1, 0, 1)
    tiles = (runs[:, 7] - runs[:, 6] + 7) // 8
    goes_on = runs[:-1, 0] == runs[1:, 0]
    assert tiles[:-1][goes_on].max() >= 1000 and np.count_nonzero(tiles[:-1][goes_on] >= 500) >= 30
    return b


def handle(b, **opts):
    import contextlib

    @contextlib.contextmanager
    def live():
        h = b.pa.pa_create(HQ, HKV, b.n_pool, b.max_pages, **opts)
        try:
            yield h
        finally:
            b.pa.pa_destroy(h)
    return live()


def test_long_segments_bad_pages_and_unread_errors(long):
    """A bad own entry concerns its sequence alone, however long the other groups take; and the calls after it, its
    error not yet read, are what they are without it."""
    import torch
    bits = lambda t: t.view(torch.int16)  # noqa: E731
    with handle(long) as h:
        want = long.call(h)
        assert long.pa.pa_last_error(h) == 0
        for s, head in ((0, 0), (511, 63), (300, 17), (37, 40)):
            long.check(s, head, want)
        gone = 200
        bt = long.bt.clone()
        bt[gone, -1] = long.n_pool
        got = long.call(h, bt)
        after = long.call(h)
        assert long.pa.pa_last_error(h) == long.pa.PA_EBADPAGE
        assert long.pa.pa_last_error(h) == 0
    others = np.arange(N) != gone
    assert torch.equal(bits(got)[others], bits(want)[others])
    assert torch.isfinite(got).all()
    assert torch.equal(bits(after), bits(want))


def test_long_segments_outlast_a_short_wait_limit(long):
    """The limit bounds a wait for one step of the work, not for a whole group's (1.7 ms here)."""
    import torch
    with handle(long) as h:
        want = long.call(h)
        assert long.pa.pa_last_error(h) == 0
    with handle(long, wait_timeout_ms=1) as h:
        got = long.call(h)
        assert long.pa.pa_last_error(h) == 0
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
