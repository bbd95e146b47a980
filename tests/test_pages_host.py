"""Refusals of the page operators, without a GPU."""
import numpy as np

import windowed_prefill_attention_gb300 as pa

N_POOL, MAX_PAGES = 8, 4
TABLE, NEW, LIVE, A, B = (1 << 40, 2 << 40, 3 << 40, 4 << 40, 5 << 40)  # addresses that nothing reads


def _parts(*parts):
    return len(parts), (pa.pa_part * max(1, len(parts)))(*[pa.pa_part(*p) for p in parts])


def _fork(forks=((0, 1, 20, 3),), n_rows=4, bt=TABLE, parts=((A, 64), (B, 4736)), n_fork=None):
    f = np.array(forks, np.int32).reshape(-1, 4)
    return pa._lib.pa_debug_pages_fork_check(N_POOL, MAX_PAGES, len(f) if n_fork is None else n_fork, f.ctypes.data, n_rows,
                                             bt, *_parts(*parts))


def test_fork_refusals():
    assert _fork() == pa.PA_OK
    assert _fork(parts=()) == pa.PA_OK  # the table alone
    assert _fork(forks=((0, 1, 0, -5), (0, 2, 32, -1), (0, 3, 64, 99))) == pa.PA_OK  # no part-filled page
    assert _fork(n_fork=0, n_rows=0, bt=None) == pa.PA_OK
    for b in (dict(n_fork=-1), dict(bt=None), dict(bt=TABLE + 2), dict(n_rows=0), dict(n_rows=1), dict(forks=((0, 1, 65, 3),)),
              dict(forks=((0, 1, -1, 3),)), dict(forks=((4, 1, 5, 3),)), dict(forks=((0, 4, 5, 3),)), dict(forks=((-1, 1, 5, 3),)),
              dict(forks=((0, 1, 5, 8),)), dict(forks=((0, 1, 5, -1),)), dict(forks=((0, 0, 5, 3),)),
              dict(forks=((0, 1, 5, 3), (0, 1, 5, 4))), dict(forks=((0, 1, 5, 3), (1, 2, 5, 4))),
              dict(forks=((0, 1, 5, 3), (0, 2, 5, 3))), dict(parts=((0, 64),)), dict(parts=((A + 2, 64),)),
              dict(parts=((A, 0),)), dict(parts=((A, 6),)), dict(parts=((A, 2 << 30),)), dict(parts=((A, 64), (A + 508, 64))),
              dict(parts=((TABLE + 4, 64),)), dict(parts=((TABLE - 508, 64),)), dict(parts=((A, 4),) * (pa.PA_MAX_PARTS + 1))):
        assert _fork(**b) == pa.PA_EINVAL, b
    assert _fork(parts=((A, 64), (A + 512, 64))) == pa.PA_OK
    long = np.array([(0, 1, (1 << 30) + 1, 3)], np.int32)  # tokens and pages beyond 2^30 are refused, not wrapped round
    for n, want in ((1 << 30, pa.PA_OK), ((1 << 30) + 1, pa.PA_EINVAL), (2 ** 31 - 1, pa.PA_EINVAL)):
        long[0, 2] = n
        assert pa._lib.pa_debug_pages_fork_check(N_POOL, 2 ** 27, 1, long.ctypes.data, 2, TABLE, *_parts()) == want


def _compact(n_ctx=(20, 0, 64), S=1, bt=TABLE, nt=NEW, parts=((A, 64),), live=LIVE, n_seq=None):
    s = np.array([(0, 0, 0, n) for n in n_ctx], np.int32).reshape(-1, 4)
    return pa._lib.pa_debug_pages_compact_check(N_POOL, MAX_PAGES, len(s) if n_seq is None else n_seq, s.ctypes.data, S, bt,
                                                nt, *_parts(*parts), live)


def test_compact_refusals():
    assert _compact() == pa.PA_OK
    assert _compact(nt=TABLE) == pa.PA_OK and _compact(parts=()) == pa.PA_OK
    assert _compact(n_ctx=(), bt=None, nt=None) == pa.PA_OK
    for b in (dict(n_ctx=(65,)), dict(n_ctx=(-1,)), dict(S=-1), dict(bt=None), dict(nt=None), dict(nt=NEW + 2),
              dict(nt=TABLE + 16), dict(live=None), dict(live=LIVE + 1), dict(live=TABLE), dict(live=NEW + 4), dict(live=A + 8),
              dict(parts=((NEW + 16, 64),)), dict(parts=((A, 64), (A, 64))), dict(n_seq=-1)):
        assert _compact(**b) == pa.PA_EINVAL, b


def test_compact_of_more_pages_than_its_kernels_count():
    """Page numbers past 2^31 - 32, rounded up to whole words of marks, would leave int32."""
    s = np.array([(0, 0, 1, 20)], np.int32)
    for n_pool, want in ((1 << 30, pa.PA_OK), ((1 << 30) + 1, pa.PA_EINVAL), (2 ** 31 - 1, pa.PA_EINVAL)):
        assert pa._lib.pa_debug_pages_compact_check(n_pool, MAX_PAGES, 1, s.ctypes.data, 1, TABLE, NEW, *_parts(), LIVE) == want
