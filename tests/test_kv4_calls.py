"""Calls on the 4-bit pool beside each other: plans that change from call to call, recorded times, captured calls whose
work buffers grow, calls that fail."""
import numpy as np
import pytest

from kv4_testutil import D, random_rows
from test_kv4 import PREFILL_FLOOR, Cache, check, decode, dev_bf16, host

pytestmark = pytest.mark.gpu


def test_prefills_whose_plans_change_from_call_to_call():
    """Each call uploads a plan of another size (one unit, many, split ones) while the kernels of the one before it still
    run: no pair may take its units from the plan before."""
    import torch

    import windowed_prefill_attention_gb300 as pa
    c = Cache(60, [900, 1500, 40], 8, 2)
    q = random_rows(np.random.default_rng(9), (700, 8, D))
    dq = dev_bf16(q)
    plans = [[(0, 1)], [(0, 600), (1, 30), (2, 40)], [(1, 33)], [(0, 64), (2, 7)], [(2, 40)], [(1, 500), (0, 100), (2, 1)]]

    def seqs_of(plan):
        rows, at = [], 0
        for s, n in plan:
            rows.append((at, c.lengths[s] - n, n, c.lengths[s]))
            at += n
        return np.array(rows, np.int32), torch.from_numpy(c.bt[[s for s, _ in plan]]).cuda()

    calls = [seqs_of(p) for p in plans]
    outs = [torch.zeros_like(dq) for _ in range(4 * len(calls))]
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        seqs, bt = calls[i % len(calls)]
        pa.pa_kv4_prefill(c.h, seqs, dq, c.d_tiles, bt, 1, 0, 1 / 16, out)
    assert pa.pa_last_error(c.h) == 0
    for i, (seqs, _) in enumerate(calls):
        assert all(torch.equal(outs[i], o) for o in outs[i::len(calls)])
        rows = [(int(r[0]) + j, s, int(r[1]) + j) for r, (s, n) in zip(seqs, plans[i]) for j in {0, n // 2, n - 1}]
        check(host(outs[i]), q.astype(np.float64), c, rows, 1, 0, 1 / 16, PREFILL_FLOOR)


def test_prefill_after_one_whose_workspace_does_not_fit():
    """A call on 2^29 keys, whose widened copy would take 550 GB, fails; the call before it, whose plan the handle still
    knows, is right again, on both pools."""
    import torch

    import windowed_prefill_attention_gb300 as pa
    c = Cache(61, [200], 8, 2)
    width = 1 << 25
    bt = torch.zeros(1, width, dtype=torch.int32, device="cuda")
    bt[0, : c.max_pages] = c.d_bt[0]
    h = pa.Handle(8, 2, c.n_pool, width)
    q = random_rows(np.random.default_rng(10), (16, 8, D))
    dq = dev_bf16(q)
    small, large = np.array([(0, 184, 16, 200)], np.int32), np.array([(0, (1 << 29) - 16, 16, 1 << 29)], np.int32)
    codes = [torch.randint(-127, 128, (c.n_pool, 16, 2, D), device="cuda").to(torch.int8) for _ in range(2)]
    scales = [torch.full((c.n_pool, 16, 2), 0.01, device="cuda") for _ in range(2)]

    def kv4(seqs, out):
        pa.pa_kv4_prefill(h.h, seqs, dq, c.d_tiles, bt, 1, 0, 1 / 16, out)

    def int8(seqs, out):
        pa.pa_prefill_batch(h.h, seqs, dq, *codes, *scales, bt, 1, 0, 1 / 16, out)

    for call in (kv4, int8):
        outs = [torch.zeros_like(dq) for _ in range(3)]
        call(small, outs[0])
        for out in outs[1:]:
            with pytest.raises(pa.PAError) as e:
                call(large, torch.zeros_like(dq))
            assert e.value.code == pa.PA_ENOMEM
            call(small, out)
        assert pa.pa_last_error(h.h) == 0
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
        if call is kv4:
            check(host(outs[0]), q.astype(np.float64), c, [(i, 0, 184 + i) for i in range(16)], 1, 0, 1 / 16, PREFILL_FLOOR)
