"""Calls on the 4-bit pool beside each other: plans that change from call to call, recorded times, captured calls whose
work buffers grow, calls that fail."""
import numpy as np
import pytest

from kv4_testutil import D, PAGE, quantise, random_rows, unpack, values
from test_kv4 import DECODE_FLOOR, PREFILL_FLOOR, Cache, check, dev_bf16, host

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


def test_recorded_times_of_whole_and_split_prefills():
    """Each call adds one widening and one attention time, split units or not, and they are of the call's own work."""
    import torch

    import windowed_prefill_attention_gb300 as pa
    c = Cache(62, [30000], 8, 2)
    h = pa.Handle(8, 2, c.n_pool, c.max_pages, record_timing=True)
    dq = dev_bf16(random_rows(np.random.default_rng(11), (3000, 8, D)))
    out = torch.zeros_like(dq)

    def times(seqs, calls):
        for _ in range(calls):
            pa.pa_kv4_prefill(h.h, np.array(seqs, np.int32), dq, c.d_tiles, c.d_bt, 1, 0, 1 / 16, out)
        assert pa.pa_last_error(h.h) == 0
        got = pa.pa_timing(h.h, reset=True)
        assert got[2] == calls
        return got[0] / calls, got[1] / calls

    times([(0, 29970, 30, 30000)], 2)
    split = times([(0, 29970, 30, 30000)], 3)     # 235 tiles over many pairs
    whole = times([(0, 27000, 3000, 30000)], 3)   # as many tiles for each of 188 units
    short = times([(0, 0, 30, 30)], 3)            # one tile
    assert min(split + whole + short) > 0
    assert whole[1] > 5 * split[1] > 5 * short[1]
    assert whole[0] > 2 * short[0] and split[0] > 2 * short[0]  # 1875 blocks widened, and 2


def test_captured_decodes_keep_their_buffers_when_a_larger_call_moves_them():
    import torch

    import windowed_prefill_attention_gb300 as pa
    c = Cache(63, [40000, 900, 300], 8, 2)
    short, long = [(1, 1, 900), (2, 2, 300)], [(0, 0, 40000)]

    def seqs_of(rows):
        return np.array([(r, n - 1, 1, n) for r, _, n in rows], np.int32), c.d_bt[[s for _, s, _ in rows]].contiguous()

    q = random_rows(np.random.default_rng(12), (3, 8, D))
    dq = dev_bf16(q)
    (seqs, bt), (l_seqs, l_bt) = seqs_of(short), seqs_of(long)
    want = torch.zeros_like(dq)
    pa.pa_kv4_decode(c.h, seqs, dq, c.d_tiles, bt, 1, 0, 1 / 16, want)
    outs = [torch.zeros_like(dq) for _ in range(2)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g, o in zip(graphs, outs):
        with torch.cuda.graph(g):
            pa.pa_kv4_decode(c.h, seqs, dq, c.d_tiles, bt, 1, 0, 1 / 16, o)
    with pytest.raises(pa.PAError) as e:  # the longer call's partials do not fit yet, and may not be made room for here
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            pa.pa_kv4_decode(c.h, l_seqs, dq, c.d_tiles, l_bt, 1, 0, 1 / 16, outs[0])
    assert e.value.code == pa.PA_ENOMEM
    torch.cuda.synchronize()
    big = torch.zeros_like(dq)
    pa.pa_kv4_decode(c.h, l_seqs, dq, c.d_tiles, l_bt, 1, 0, 1 / 16, big)
    first = big.clone()
    for i in range(3):  # replays between calls on the new buffers
        for g, o in zip(graphs, outs):
            o.zero_()
            g.replay()
            big.zero_()
            pa.pa_kv4_decode(c.h, l_seqs, dq, c.d_tiles, l_bt, 1, 0, 1 / 16, big)
            assert torch.equal(o, want) and torch.equal(big, first), i
    assert pa.pa_last_error(c.h) == 0
    check(host(want), q.astype(np.float64), c, [(1, 1, 899), (2, 2, 299)], 1, 0, 1 / 16, DECODE_FLOOR)
    check(host(first), q.astype(np.float64), c, [(0, 0, 39999)], 1, 0, 1 / 16, DECODE_FLOOR)


@pytest.mark.parametrize("n_seq,hq,hkv", [(700, 4, 2), (520, 14, 7)])
def test_every_call_of_more_sequences_than_a_launch_takes(n_seq, hq, hkv):
    import torch

    import windowed_prefill_attention_gb300 as pa
    lengths = [1 + (37 * s) % 90 for s in range(n_seq)]
    new = [min(n, 1 + s % 3) for s, n in enumerate(lengths)]
    off = np.cumsum([0] + new)
    c = Cache(n_seq, lengths, hq, hkv)
    rng = np.random.default_rng(n_seq)
    k, v = (random_rows(rng, (off[-1], hkv, D)) for _ in range(2))
    q = random_rows(rng, (off[-1], hq, D))
    seqs = np.array([(off[s], lengths[s] - new[s], new[s], lengths[s]) for s in range(n_seq)], np.int32)
    pa.pa_kv4_append(c.h, seqs, dev_bf16(k), dev_bf16(v), c.d_bt, c.d_tiles)
    ko, vo = (torch.zeros(off[-1], hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pa.pa_kv4_gather(c.h, seqs, c.d_bt, c.d_tiles, ko, vo)
    assert pa.pa_last_error(c.h) == 0
    assert np.array_equal(host(ko), values(*quantise(k))) and np.array_equal(host(vo), values(*quantise(v)))
    c.k, c.v = ([x[c.bt[s, : -(-n // PAGE)]].reshape(-1, hkv, D)[:n] for s, n in enumerate(lengths)] for x in unpack(c.d_tiles.cpu().numpy()))
    dq = dev_bf16(q)
    out = torch.zeros_like(dq)
    pa.pa_kv4_prefill(c.h, seqs, dq, c.d_tiles, c.d_bt, 1, 3, 1 / 16, out)
    assert pa.pa_last_error(c.h) == 0
    check(host(out), q.astype(np.float64), c, [(off[s] + i, s, lengths[s] - new[s] + i) for s in range(0, n_seq, 7) for i in range(new[s])],
          1, 3, 1 / 16, PREFILL_FLOOR)
    one = np.array([(s, n - 1, 1, n) for s, n in enumerate(lengths)], np.int32)
    pa.pa_kv4_decode(c.h, one, dq, c.d_tiles, c.d_bt, 1, 3, 1 / 16, out)
    assert pa.pa_last_error(c.h) == 0
    check(host(out), q.astype(np.float64), c, [(s, s, n - 1) for s, n in enumerate(lengths)][::5], 1, 3, 1 / 16, DECODE_FLOOR)
