"""Calls on pages beside each other."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def test_compactions_of_large_pools_from_threads():
    """Handles whose marks take more shared memory than a kernel has without asking, each its own amount."""
    import threading

    import torch

    import windowed_prefill_attention_gb300 as pa
    steps, errors, tables, lives = 300, [], {}, {}

    def run(n_pool):
        try:
            torch.cuda.set_device(0)
            st = torch.cuda.Stream()
            h = pa.Handle(4, 2, n_pool, 4)
            bt = torch.tensor([[n_pool - 1, n_pool // 2, -1, -1]], dtype=torch.int32, device="cuda")
            nt = torch.empty_like(bt)
            live = torch.zeros(1, dtype=torch.int32, device="cuda")
            part = torch.zeros(n_pool, 1, dtype=torch.int32, device="cuda")
            seqs = np.array([(0, 0, 1, 32)], np.int32)
            torch.cuda.synchronize()
            gate.wait()
            for _ in range(steps):
                pa.pa_pages_compact(h.h, seqs, 1, 0, bt, nt, [part], live, stream=st)
            st.synchronize()
            assert pa.pa_last_error(h.h) == 0
            tables[n_pool], lives[n_pool] = nt.cpu().tolist(), int(live)
        except Exception as e:  # raised again by the test's own thread
            errors.append(e)
            gate.abort()

    sizes = (1000000, 500000, 700000)
    gate = threading.Barrier(len(sizes))
    threads = [threading.Thread(target=run, args=(n,)) for n in sizes]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert lives == {n: 2 for n in sizes} and tables == {n: [[1, 0, -1, -1]] for n in sizes}


def test_a_bad_page_is_reported_of_a_fork_without_pools():
    import torch

    import windowed_prefill_attention_gb300 as pa
    h = pa.Handle(4, 2, 8, 3)
    bt = torch.tensor([[1, 8, -1], [-1, -1, -1], [2, 3, -1], [-1, -1, -1]], dtype=torch.int32, device="cuda")
    part = torch.zeros(8, 4, dtype=torch.int32, device="cuda")
    for parts in ([part], []):
        for src, want in ((0, pa.PA_EBADPAGE), (2, 0)):
            t = bt.clone()
            pa.pa_pages_fork(h.h, [(src, 1, 20, 5)], t, parts)
            assert pa.pa_last_error(h.h) == want, (src, len(parts))
            assert t[1].tolist() == [1 + src // 2, 5, -1]
        pa.pa_pages_fork(h.h, [(0, 1, 32, 5)], bt.clone(), parts)  # whole pages are taken over unread
        assert pa.pa_last_error(h.h) == 0


@pytest.mark.parametrize("n_seq,n_pool,max_pages,S,W", [(600, 20000, 20, 1, 4), (1300, 30000, 20, 0, 0), (20, 1500000, 400, 2, 30),
                                                        (40, 60000, 1200, 1, 64)])
def test_compactions_in_place_and_captured_of_many_rows_and_pages(n_seq, n_pool, max_pages, S, W):
    """More rows than a launch takes, more pages than one CTA marks: each launch's rows of the table, in place."""
    import torch

    import windowed_prefill_attention_gb300 as pa
    from test_pages import plain_compact
    rng = np.random.default_rng(n_seq)
    n_ctx = rng.integers(0, max_pages * 16 + 1, n_seq)
    perm, at = rng.permutation(n_pool), 0
    table = rng.integers(-5, 5, (n_seq, max_pages)).astype(np.int32)
    for s, n in enumerate(n_ctx):
        k = -(-n // 16)
        table[s, :k] = perm[at: at + k]
        at += k
    table[2], n_ctx[2] = table[1], n_ctx[1]
    first = [torch.from_numpy(rng.integers(0, 256, (n_pool, w), dtype=np.uint8)).cuda() for w in (16, 4)]
    parts = [p.clone() for p in first]
    want, n_live, pools = plain_compact(table, n_ctx, S, W, n_pool, [p.cpu().numpy() for p in first])
    h = pa.Handle(4, 2, n_pool, max_pages)
    seqs = np.array([(0, 0, 1, n) for n in n_ctx], np.int32)
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    start = torch.from_numpy(table).cuda()
    bt = start.clone()

    def check():
        assert pa.pa_last_error(h.h) == 0 and int(live) == n_live
        assert np.array_equal(bt.cpu().numpy(), want)
        for p, w in zip(parts, pools):
            assert np.array_equal(p.cpu().numpy()[:n_live], w[:n_live])

    pa.pa_pages_compact(h.h, seqs, S, W, bt, bt, parts, live)
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_pages_compact(h.h, seqs, S, W, bt, bt, parts, live)
    for _ in range(2):
        bt.copy_(start)
        live.fill_(-1)
        for p, f in zip(parts, first):
            p.copy_(f)
        graph.replay()
        check()
