"""GPU: a bad page entry of one sequence while the work units of others take over a
millisecond, in the prefill and the decode: the others' outputs, and those of the
calls after it, are what they are without it."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

HQ, HKV, CTX, N_Q = 16, 2, 131072, 512


@pytest.mark.parametrize("form", ("prefill", "decode"))
def test_bad_page_concerns_its_sequence_alone(form):
    """Two sequences of 131072 tokens without a window: a prefill unit is 256 rows against 1008 tiles of keys and more,
    about 1.3 ms, for all of which its epilogue waits."""
    import torch

    import windowed_prefill_attention_gb300 as pa
    g = torch.Generator("cuda").manual_seed(4)
    pages = CTX // 16
    shape = (2 * pages, 16, HKV, 256)
    kp, vp = (torch.randint(-127, 128, shape, dtype=torch.int8, device="cuda", generator=g) for _ in range(2))
    ks, vs = (torch.rand(shape[:3], device="cuda", generator=g) * s for s in (2e-3, 2e-2))
    bt = torch.randperm(2 * pages, device="cuda", generator=g).int().view(2, pages)
    n = N_Q if form == "prefill" else 1
    q = torch.randn(2 * n, HQ, 256, device="cuda", generator=g).bfloat16()
    seqs = np.array([(i * n, CTX - n, n, CTX) for i in range(2)], np.int32)
    call = pa.pa_prefill_batch if form == "prefill" else pa.pa_decode

    def run(h, table):
        out = torch.full_like(q, float("nan"))
        call(h, seqs, q, kp, vp, ks, vs, table, 1, 0, 1 / 16, out)
        return out.view(torch.int16)
    bad = bt.clone()
    bad[1, 17] = 2 * pages
    h = pa.pa_create(HQ, HKV, 2 * pages, pages)
    try:
        want = run(h, bt)
        assert pa.pa_last_error(h) == 0
        got = run(h, bad)
        after = run(h, bt)
        assert pa.pa_last_error(h) == pa.PA_EBADPAGE
        assert pa.pa_last_error(h) == 0
    finally:
        pa.pa_destroy(h)
    assert torch.isfinite(want.view(torch.bfloat16)).all() and torch.isfinite(got.view(torch.bfloat16)).all()
    assert torch.equal(got[:n], want[:n])
    assert torch.equal(after, want)
