"""CPU: overlaps of what pa_qk_norm_rope and pa_qkv_append write with what they
read beside the rows (weights, positions, the block table) and with each other."""
import ctypes as C

import numpy as np
import pytest

from test_qkv_host import A, B, O1, O2, pa, rope_args, rows  # noqa: F401

P = 5 << 32  # positions


@pytest.mark.parametrize("out, size", (("qo", 10 * 16 * 512), ("ko", 10 * 2 * 512)))
def test_norm_rope_outputs_keep_off_weights_and_positions(pa, out, size):  # noqa: F811
    at = {"qo": O1, "ko": O2}[out]
    ok = lambda **k: rope_args(pa, **k) == pa.PA_OK          # noqa: E731
    no = lambda **k: rope_args(pa, **k) == pa.PA_EINVAL      # noqa: E731
    for w in ("qw", "kw"):
        assert no(**{w: at}) and no(**{w: at + size - 16}) and no(**{w: at - 496})
        assert ok(**{w: at + size}) and ok(**{w: at - 512})
    # gains of rows that the call leaves out are not read
    assert ok(qw=O2, q=None, qo=None) and ok(kw=O1, k=None, ko=None)
    assert no(pos=at) and no(pos=at + size - 4) and no(pos=at - 36) and ok(pos=at + size) and ok(pos=at - 40)
    assert ok(pos=at, rope=None) and ok(pos=at, rope=pa.pa_rope_init([]))  # nothing to turn: not read
    two = pa.pa_rope_init(np.ones(32), pair_axis=np.arange(32) % 2)
    assert ok(rope=two, pos=P, ps=1000)
    assert no(rope=two, pos=at - 4000, ps=1000) and no(rope=two, pos=at - 4036, ps=1000)  # the second axis
    assert ok(rope=two, pos=at - 4040, ps=1000)
    assert no(rope=two, pos=P, ps=(1 << 46) + 1)


POOL, SCALES = 4 * 16 * 2 * 256, 4 * 16 * 2 * 4  # bytes of a pool of four pages, of its scales
AT = dict(kp=11 << 32, vp=12 << 32, ks=13 << 32, vs=14 << 32, qo=O1)  # what the append writes
SIZE = dict(kp=POOL, vp=POOL, ks=SCALES, vs=SCALES, qo=10 * 16 * 512)
V, TABLE = 6 << 32, 7 << 32
ROWS = ((A, 10 * 16 * 512), (B, 10 * 2 * 512), (V, 10 * 2 * 512))  # q, k and v


def append_args(pa, n_pool=4, qw=None, kw=None, pos=None, ps=10, bt=TABLE, **at):  # noqa: F811
    """pa_debug_qkv_append_pool_check for 16 q / 2 kv heads, two sequences, ten tokens; `at` moves what is written."""
    to = {**AT, **at}
    rope = pa.pa_rope_init(np.ones(32))
    return pa._lib.pa_debug_qkv_append_pool_check(
        16, 2, n_pool, 4, 2, pa._seqs([(0, 5, 3, 8), (3, 0, 7, 7)]), rows(pa, A, 4096, 256), rows(pa, B, 512, 256),
        rows(pa, V, 512, 256), qw, kw, 0.0, 1e-6, C.byref(rope), pos, ps, bt, to["kp"], to["vp"], to["ks"], to["vs"],
        to["qo"])


def test_append_outputs_keep_off_each_other_and_the_inputs(pa):  # noqa: F811
    ok = lambda **k: append_args(pa, **k) == pa.PA_OK          # noqa: E731
    no = lambda **k: append_args(pa, **k) == pa.PA_EINVAL      # noqa: E731
    assert ok() and no(n_pool=-1)
    for i, a in enumerate(AT):
        at, end = AT[a], AT[a] + SIZE[a]
        for b in list(AT)[i + 1:]:
            assert no(**{b: at}) and no(**{b: end - 16}) and ok(**{b: end}), (a, b)
            assert no(**{b: at - SIZE[b] + 16}) and ok(**{b: at - SIZE[b]}), (a, b)
        assert no(bt=at) and no(bt=end - 4) and no(bt=at - 28) and ok(bt=end) and ok(bt=at - 32), a
        assert no(pos=at) and no(pos=end - 4) and no(pos=at - 36) and ok(pos=end) and ok(pos=at - 40), a
        for w in ("qw", "kw"):
            assert no(**{w: at}) and no(**{w: end - 16}) and no(**{w: at - 496}) and ok(**{w: end}) and ok(**{w: at - 512}), a
        for data, size in ROWS:
            if (a, data) != ("qo", A):  # the query rows in place
                assert no(**{a: data}), (a, data)
            assert no(**{a: data + size - 16}) and ok(**{a: data + size}), (a, data)
            assert no(**{a: data - SIZE[a] + 16}) and ok(**{a: data - SIZE[a]}), (a, data)
    assert ok(qo=A)
    # a form that knows no pool leaves overlaps with it out
    assert ok(n_pool=0, kp=B) and no(n_pool=0, qo=B)
