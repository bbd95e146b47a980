"""CPU: pa_decode_shared's work split (pa_decode_shared_plan) against the mask's
definition, and its refusals."""
import ctypes as C
import os
import subprocess
import sys

import numpy as np
import pytest

import oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def pa():
    subprocess.run([sys.executable, os.path.join(ROOT, "windowed_prefill_attention_gb300", "build.py")], check=True,
                   capture_output=True)
    import windowed_prefill_attention_gb300 as mod
    return mod


def listed(base, sink, lo, first, last):
    return [base + b if b < sink else lo + (b - sink) for b in range(first, last)]


CASES = [
    # q heads, kv heads, SMs, prefix, own tokens, sink, window
    (16, 2, 152, 32768, [1, 17, 500, 1024] * 16, 1, 0),
    (16, 2, 152, 8192, list(range(1, 251)), 1, 0),
    (8, 1, 152, 131072, [5, 77, 300], 0, 0),
    (8, 4, 152, 8192, [1 + 41 * i for i in range(48)], 1, 256),
    (4, 1, 7, 160, [1, 2, 3], 2, 4),
    (4, 4, 152, 64, [1, 900, 40, 8000], 9, 20),     # sinks past the prefix; windows that hide all of it
    (8, 8, 152, 16, [16] * 130, 0, 1),              # one-block windows: no prefix visible
    (8, 1, 3, 4096, [100] * 512, 1, 64),
    (8, 1, 3, 4096, [100] * 600, 1, 64),            # the first 512
    (16, 2, 152, 4096, [70000], 1, 0),              # one sequence: no prefix pass
    (16, 2, 152, 0, [300, 20], 1, 0),               # no prefix
    (2, 2, 152, 48, [1, 1], 0, 0),
]


@pytest.mark.parametrize("prefix_pass", (1, 0, -1))
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in (c[0], c[1], c[2], c[3], len(c[4]), c[6])))
def test_every_visible_block_is_computed_once(pa, case, prefix_pass):
    hq, hkv, n_sm, prefix, suffix, S, W = case
    seqs = np.array([(i, prefix + x - 1, 1, prefix + x) for i, x in enumerate(suffix)], np.int32)
    pre, own = pa.pa_decode_shared_plan(hq, hkv, 1 << 20, n_sm, seqs, prefix, S, W, prefix_pass)
    assert prefix_pass or not len(pre)
    n, pb = min(512, len(suffix)), prefix // 16
    n_cta = 1 if n * (hq // hkv) <= 128 else 2  # CTAs of a unit of the prefix pass
    tile, rows = 8, 128 * n_cta                 # blocks of a tile; rows of a group
    done = {}  # (sequence, head) -> blocks of its own passes
    for s, g, base, sink, lo, first, last in own.tolist():
        assert 0 < last - first <= 128
        done.setdefault((s, g), []).extend(listed(base, sink, lo, first, last))
    groups = {}
    for _, g, s0, ns, sink, lo, first, last in pre.tolist():
        assert 0 <= first < last and first % tile == 0 and ns * (hq // hkv) <= rows
        groups.setdefault((g, s0, ns), []).extend(listed(0, sink, lo, first, last))
    seen_by = {}
    for (g, s0, ns), blocks in groups.items():
        assert len(blocks) == len(set(blocks)) and (not blocks or max(blocks) < pb)
        for s in range(s0, s0 + ns):
            assert (s, g) not in seen_by
            seen_by[s, g] = set(blocks)
    union = {}
    for s in range(n):
        t = prefix + suffix[s] - 1
        want = [b for b in range(t // 16 + 1) if oracle.key_visible(t, 16 * b, S, W)] if t < 20000 else None
        for g in range(hkv):
            mine = done.pop((s, g))
            assert len(mine) == len(set(mine))
            if want is None:
                assert W == 0
                want = list(range(t // 16 + 1))
            shared = seen_by.get((s, g), set())
            # a group's list may hold blocks its mask hides from this row; never one of its own pass
            assert not shared & set(mine)
            assert set(mine) | {b for b in shared if b in set(want)} == set(want)
            for b in want:
                if b in shared:
                    union.setdefault((g, s // (rows // (hq // hkv))), set()).add(b)
    assert not done
    for (g, s0, ns), blocks in groups.items():  # a block is listed only if some sequence of the group sees it
        assert set(blocks) == union[g, s0 // (rows // (hq // hkv))]
    if len(pre):  # one unit's tiles are consecutive, and the costliest unit (4 for every group after its first) is
        # within one group's charge of the mean
        units, most = pre[:, 0], max(1, n_sm // n_cta)
        assert np.all(np.diff(units) >= 0) and units[0] == 0 and units[-1] < most
        cost = np.full(units[-1] + 1, -4)
        np.add.at(cost, units, (pre[:, 7] - pre[:, 6] + tile - 1) // tile + 4)
        assert cost.min() >= 1
        assert cost.max() <= -(-cost.sum() // most) + 5 or len(cost) < most
        assert len(cost) == most or cost.max() <= cost.sum() // len(cost) + 5


def test_prefix_pass_by_size(pa):
    """Few sequences or a short prefix: every sequence reads it; many on a long one: once for all."""
    def runs(n, prefix, **kw):
        seqs = [(i, prefix + 9, 1, prefix + 10) for i in range(n)]
        return len(pa.pa_decode_shared_plan(16, 2, 1 << 20, 152, seqs, prefix, 1, 0, **kw)[0])
    assert runs(3, 1024) == 0 < runs(3, 1024, prefix_pass=1)
    assert runs(250, 16) == 0
    assert runs(64, 32768) > 0 == runs(64, 32768, prefix_pass=0)
    assert runs(1, 32768, prefix_pass=1) == 0


def test_plan_refusals(pa):
    ok = [(0, 99, 1, 100), (1, 119, 1, 120)]

    def plan(hq=8, hkv=2, pages=100, n_sm=152, seqs=ok, prefix=64, S=1, W=0, prefix_pass=-1):
        return pa.pa_decode_shared_plan(hq, hkv, pages, n_sm, seqs, prefix, S, W, prefix_pass)
    plan()
    plan(prefix=96)
    plan(W=-1)
    for bad in (dict(hq=32), dict(hq=7), dict(hkv=0), dict(hq=9, hkv=9), dict(pages=7), dict(pages=0), dict(n_sm=0),
                dict(prefix=-16), dict(prefix=60), dict(prefix=112), dict(prefix=1 << 20), dict(S=-1), dict(seqs=[]),
                dict(seqs=[(0, 99, 2, 101)]), dict(seqs=[(0, 98, 1, 100)]), dict(seqs=[(-1, 99, 1, 100)]),
                dict(seqs=[(0, 99, 1, 100), (0, 119, 1, 120)]), dict(seqs=[(0, 2 ** 31 - 2, 1, 2 ** 31 - 1)]),
                dict(seqs=[(2 ** 30, 99, 1, 100)]), dict(prefix_pass=2), dict(prefix_pass=-2)):
        with pytest.raises(pa.PAError):
            plan(**bad)
    n = C.c_int()
    assert pa._lib.pa_decode_shared_plan(8, 2, 100, 152, 2, pa._seqs(ok), 64, 1, 0, 1, None, 0, None, None,
                                         0, C.byref(n)) == pa.PA_EINVAL
    buf = np.zeros(8, np.int32)
    for prefix_pass, pre, own in ((1, buf.ctypes.data, None), (1, None, buf.ctypes.data), (0, None, buf.ctypes.data)):
        assert pa._lib.pa_decode_shared_plan(8, 2, 100, 152, 2, pa._seqs(ok), 64, 1, 0, prefix_pass, pre, 1, C.byref(n),
                                             own, 1, C.byref(n)) == pa.PA_EINVAL
    assert pa._lib.pa_debug_decode_shared_pass(None, 1) == pa.PA_EINVAL


def test_null_handle_is_refused(pa):
    assert pa._lib.pa_decode_shared(None, 1, pa._seqs([(0, 99, 1, 100)]), 64, 1, *[None] * 6, 1, 0, 0.1, None,
                                    None) == pa.PA_EINVAL
