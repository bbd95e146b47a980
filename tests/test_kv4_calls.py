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
