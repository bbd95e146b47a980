"""CPU: the host side of pa_rope_init, pa_qk_norm_rope and pa_qkv_append (no
GPU): the rotation's turns, and every refusal of bad arguments."""
import ctypes as C
import os
import subprocess
import sys
from fractions import Fraction

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def pa():
    subprocess.run([sys.executable, os.path.join(ROOT, "windowed_prefill_attention_gb300", "build.py")], check=True,
                   capture_output=True)
    import windowed_prefill_attention_gb300 as mod
    return mod


PI = Fraction(314159265358979323846264338327950288419716939937510, 10 ** 50)


@pytest.mark.parametrize("pos", [1, -1, 4096, 131072, 2 ** 31 - 1, -2 ** 31])
def test_rope_turns_hold_the_fraction_of_a_turn(pa, pos):
    """pos * turn mod 2^64 is the fraction of a turn of pos * inv_freq.  Two roundings of 2^-53 (2 pi as a double,
    the quotient) times the turns taken, and 2^-64 a position from the fraction's last bit."""
    freq = 10000.0 ** (-np.arange(128) / 128.0)
    freq[5] = 7.25  # more than one turn a position
    freq[6] = -0.3
    r = pa.pa_rope_init(freq)
    assert (r.rot_dim, r.pairing, r.n_axes) == (256, pa.PA_ROPE_HALF, 1)
    for i in range(128):
        turns = pos * Fraction(float(freq[i])) / (2 * PI)
        want = turns - turns.__floor__()
        got = Fraction((r.turn[i] * pos) % 2 ** 64, 2 ** 64)
        off = abs(got - want)
        off = min(off, 1 - off)
        assert off <= abs(turns) * Fraction(2, 2 ** 53) + abs(pos) * Fraction(1, 2 ** 53), (i, float(off))


def test_rope_init_refuses(pa):
    ok = lambda **k: pa.pa_rope_init(**{**dict(inv_freq=np.ones(32)), **k})  # noqa: E731
    assert ok(pair_axis=np.arange(32) // 8).n_axes == 4
    assert pa.pa_rope_init([]).rot_dim == 0
    for bad in (dict(inv_freq=np.ones(4)),             # 8 dims: not a multiple of 16
                dict(inv_freq=np.ones(136)),           # more than a head
                dict(inv_freq=[np.nan] * 8), dict(inv_freq=[np.inf] * 8),
                dict(pairing=2), dict(pair_axis=np.full(32, 4)), dict(pair_axis=np.full(32, -1))):
        with pytest.raises(pa.PAError):
            ok(**bad)
    with pytest.raises(ValueError):
        ok(pair_axis=np.zeros(31, int))
    assert pa._lib.pa_rope_init(None, 0, 0, 1, None, None) == pa.PA_EINVAL


def rows(pa, data, ts, hs, n_tok=10):
    return C.byref(pa.pa_rows(data, n_tok, ts, hs))


# addresses only: the checks read no memory behind them
A, B, O1, O2 = 1 << 32, 2 << 32, 3 << 32, 4 << 32


def rope_args(pa, **over):
    """pa_debug_qk_norm_rope_check for 16 q / 2 kv heads, 10 tokens, contiguous rows; `over` replaces arguments."""
    a = dict(hq=16, hkv=2, n=10, q=(A, 16 * 256, 256), k=(B, 2 * 256, 256), qw=None, kw=None, off=0.0, eps=1e-6,
             rope=pa.pa_rope_init(np.ones(32)), pos=1 << 20, ps=10, qo=O1, ko=O2)
    a.update(over)
    r = lambda x: None if x is None else rows(pa, *x)  # noqa: E731
    return pa._lib.pa_debug_qk_norm_rope_check(a["hq"], a["hkv"], a["n"], r(a["q"]), r(a["k"]), a["qw"], a["kw"],
                                               a["off"], a["eps"], None if a["rope"] is None else C.byref(a["rope"]),
                                               a["pos"], a["ps"], a["qo"], a["ko"])


def test_norm_rope_argument_checks(pa):
    ok = lambda **k: rope_args(pa, **k) == pa.PA_OK          # noqa: E731
    no = lambda **k: rope_args(pa, **k) == pa.PA_EINVAL      # noqa: E731
    assert ok()
    assert ok(n=0, q=None)                                    # nothing to do
    assert no(n=11, ps=11) and ok(n=9)                        # past the rows there are
    assert ok(q=None, qo=None) and ok(k=None, ko=None)
    assert no(q=None) and no(k=None) and no(q=None, qo=None, k=None, ko=None) and no(qo=None) and no(ko=None)
    assert no(n=-1) and no(n=2 ** 30 + 1)
    assert no(q=(A + 8, 4096, 256)) and no(k=(B + 2, 512, 256)) and no(qo=O1 + 8) and no(ko=O2 + 4)
    assert no(qw=24) and no(kw=24) and ok(qw=32, kw=64)
    assert no(q=(A, 4100, 256)) and no(q=(A, 4096, 250)) and no(q=(A, -4096, 256)) and no(k=(B, 512, -256))
    assert no(q=(A, 2 ** 62, 256)) and no(q=(A, 4096, 2 ** 62)) and no(q=(0, 4096, 256))
    assert ok(q=(A, 0, 0), k=(B, 0, 256))                     # broadcast rows
    assert no(eps=-1e-9) and no(eps=float("nan")) and no(eps=float("inf")) and no(off=float("nan")) and ok(eps=0.0)
    assert no(pos=None) and ok(pos=None, rope=None) and no(pos=(1 << 20) + 2) and no(ps=-1)
    two = pa.pa_rope_init(np.ones(32), pair_axis=np.arange(32) % 2)
    assert ok(rope=two) and no(rope=two, ps=9)
    # in place, and everything that overlaps without being that
    assert ok(qo=A) and ok(ko=B) and ok(qo=A, ko=B)
    assert no(qo=A, q=(A, 8192, 256)) and no(qo=A, q=(A, 4096, 512)) and no(qo=A + 4096)
    assert no(ko=A) and no(qo=B) and no(ko=O1) and no(ko=O1 + 16 * 256 * 2 * 10 - 16) and ok(ko=O1 + 16 * 256 * 2 * 10)
    assert ok(qo=A, n=1, q=(A, 0, 256)) and ok(ko=B, hkv=1, hq=16, k=(B, 256, 0))
    broken = pa.pa_rope_init(np.ones(32))
    for field, value in (("rot_dim", 24), ("rot_dim", 272), ("rot_dim", -16), ("pairing", 7), ("n_axes", 0),
                         ("n_axes", 5)):
        r = type(broken).from_buffer_copy(broken)
        setattr(r, field, value)
        assert no(rope=r), field
    broken.axis[31] = 1
    assert no(rope=broken)
    assert no(hq=15) and no(hkv=0) and no(hkv=9, hq=9)


def append_args(pa, **over):
    a = dict(seqs=[(0, 5, 3, 8), (3, 0, 7, 7)], max_pages=4, q=(A, 16 * 256, 256), k=(B, 512, 256),
             v=(B + (1 << 20), 512, 256), off=0.0, eps=1e-6, rope=pa.pa_rope_init(np.ones(32)), pos=None, ps=0,
             bt=64, kp=1 << 33, vp=2 << 33, ks=3 << 33, vs=4 << 33, qo=O1)
    a.update(over)
    r = lambda x: None if x is None else rows(pa, *x)  # noqa: E731
    s = None if a["seqs"] is None else pa._seqs(a["seqs"])
    return pa._lib.pa_debug_qkv_append_check(16, 2, a["max_pages"], 0 if s is None else len(s), s, r(a["q"]),
                                             r(a["k"]), r(a["v"]), None, None, a["off"], a["eps"],
                                             None if a["rope"] is None else C.byref(a["rope"]), a["pos"], a["ps"],
                                             a["bt"], a["kp"], a["vp"], a["ks"], a["vs"], a["qo"])


def test_append_argument_checks(pa):
    ok = lambda **k: append_args(pa, **k) == pa.PA_OK          # noqa: E731
    no = lambda **k: append_args(pa, **k) == pa.PA_EINVAL      # noqa: E731
    assert ok() and ok(seqs=None) and ok(rope=None) and ok(q=None, qo=None)
    assert no(k=None) and no(v=None) and no(q=None) and no(qo=None)
    for name in ("bt", "kp", "vp", "ks", "vs"):
        assert no(**{name: None}), name
    assert no(kp=(1 << 33) + 8) and no(vs=(4 << 33) + 2) and no(bt=66) and no(v=(B + 8, 512, 256))
    assert no(seqs=[(0, 5, 0, 8)]) and no(seqs=[(-1, 5, 3, 8)]) and no(seqs=[(0, -1, 3, 8)])
    assert no(seqs=[(0, 5, 4, 8)])                                     # past its own context
    assert ok(seqs=[(0, 60, 4, 64)]) and no(seqs=[(0, 60, 5, 65)])     # past max_pages_per_seq pages
    assert no(seqs=[(2 ** 30 - 1, 0, 3, 3)])
    assert no(seqs=[(0, 5, 3, 8), (4, 0, 7, 7)]) and no(v=(B + (1 << 20), 512, 256, 9))  # past the rows there are
    assert no(seqs=[(0, 5, 3, 8), (2, 0, 7, 7)])                       # a row of two sequences
    assert no(seqs=[(4, 0, 6, 6), (0, 5, 5, 10)]) and ok(seqs=[(5, 0, 5, 5), (0, 5, 5, 10)])
    assert no(qo=B) and no(qo=B + (1 << 20)) and ok(qo=A) and no(qo=A, q=(A, 9216, 256))
    two = pa.pa_rope_init(np.ones(32), pair_axis=np.arange(32) % 2)
    assert ok(rope=two, pos=1 << 20, ps=10) and no(rope=two, pos=1 << 20, ps=9)


def test_null_handles_are_refused(pa):
    n = C.c_void_p()
    assert pa._lib.pa_qk_norm_rope(n, 1, None, None, None, None, 0.0, 0.0, None, None, 0, None, None,
                                   None) == pa.PA_EINVAL
    assert pa._lib.pa_qkv_append(n, 1, None, None, None, None, None, None, 0.0, 0.0, None, None, 0, None, None, None,
                                 None, None, None, None) == pa.PA_EINVAL
    with pytest.raises(ValueError):
        pa._geometry_of(n)
