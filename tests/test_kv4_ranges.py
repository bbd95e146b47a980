"""The 4-bit pool's attention over the whole range of row scales: V rows at the top of bf16's range, rows far
larger than those beside them, queries at the bottom of bf16's range."""
import numpy as np
import pytest

from kv4_testutil import D, PAGE, attention, bf16_round, pack, random_rows, unpack
from test_kv4 import PREFILL_FLOOR, Cache, dev_bf16, host

pytestmark = pytest.mark.gpu


def cache_of(seed, lengths, hq, hkv, change):
    """A Cache whose K and V rows [pages, 16, hkv, 256] went through change(k, v, slots): slots[s] gives the pages and rows
    of sequence s's tokens."""
    import torch
    c = Cache(seed, lengths, hq, hkv)
    rng = np.random.default_rng(seed + 1000)
    k, v = (random_rows(rng, (c.n_pool, PAGE, hkv, D)).astype(np.float64) for _ in range(2))
    slots = [(c.bt[s, np.arange(n) // PAGE], np.arange(n) % PAGE) for s, n in enumerate(lengths)]
    change(k, v, slots)
    with np.errstate(over="ignore"):
        c.tiles = pack(*(bf16_round(x.astype(np.float32)) for x in (k, v)))
    c.d_tiles = torch.from_numpy(c.tiles).cuda()
    k, v = unpack(c.tiles)
    c.k, c.v = ([x[pages, rows] for pages, rows in slots] for x in (k, v))
    return c


def largest_share(q, c, s, t, S, W, sm):
    """[HQ]: of a query token the largest weight x V row scale, over the sum of the weights."""
    hq, hkv = q.shape[0], c.hkv
    n = len(c.k[s])
    scale = c.tiles[c.bt[s, np.arange(n) // PAGE], :, 4672:].copy().view(np.float32).reshape(n, hkv, PAGE)
    scale = scale[np.arange(n), :, np.arange(n) % PAGE].astype(np.float64)
    j = np.arange(min(n, t + 1))
    if W > 0:
        j = j[(j // PAGE < S) | (j // PAGE >= max(0, t // PAGE + 1 - W))]
    out = np.zeros(hq)
    for h in range(hq):
        y = sm * (c.k[s][j, h // (hq // hkv)] @ q[h])
        p = np.exp(y - y.max())
        out[h] = (p * scale[j, h // (hq // hkv)]).max() / p.sum()
    return out


def check_rows(got, q, c, rows, S, W, sm, half_step):
    """Against the 64-bit definition.  A weight x row scale is held in fp16 under a power of two of the row's own:
    2^-11 of it, or, where it leaves fp16's normal range, half_step of the row's largest; V's codes under their block
    scales are at most 2688."""
    worst = 0.0
    for row, s, t in rows:
        qq = q[row].astype(np.float64)
        ref, bound = attention(qq, c.k[s], c.v[s], t, S, W, sm, 0.0)
        bound = bound + half_step * 2688 * (t + 1) * largest_share(qq, c, s, t, S, W, sm)[:, None]
        assert np.isfinite(got[row]).all(), (row, s, t)
        worst = max(worst, float((np.abs(got[row] - ref) / bound).max()))
    assert worst <= 1.0, worst


# decode: the largest product is at least 2^6 in its units (a reference up to 2^8 behind, a significand of 1/2 or more)
DECODE_STEP = 2.0 ** (-25 - 6)
# prefill: at least 2^-6 (the first reference lies 2^6 above the first tile's largest)
PREFILL_STEP = 2.0 ** (-25 + 6)


@pytest.mark.parametrize("lengths", [[1, 40, 700], [5, 9000]])  # one run a pair and several; over many CTAs
@pytest.mark.parametrize("exponent", [100, 112, 120, 126])
def test_decode_of_values_at_the_top_of_the_range(lengths, exponent):
    """Finite V rows of up to 3e38, equal weights among them: finite outputs, whose sums before the division are not."""
    import windowed_prefill_attention_gb300 as pa

    def change(k, v, slots):
        for pages, rows in slots:
            # quantised, 2.8e38 is 6 x 288 x 2^117 = 2.87e38, which bf16 holds (3.38e38 would become 3.51e38)
            v[pages, rows] = np.clip(np.ldexp(v[pages, rows], exponent), -2.8e38, 2.8e38)
            k[pages[len(pages) // 2:], rows[len(pages) // 2:]] *= 2.0 ** -6  # many weights alike
            v[pages[0], rows[0]] = np.sign(v[pages[0], rows[0]]) * 2.8e38

    c = cache_of(61, lengths, 8, 2, change)
    q = random_rows(np.random.default_rng(10), (len(lengths), 8, D))
    for sm in (1 / 16, 0.0):
        seqs = np.array([(s, n - 1, 1, n) for s, n in enumerate(lengths)], np.int32)
        dq = dev_bf16(q)
        pa.pa_kv4_decode(c.h, seqs, dq, c.d_tiles, c.d_bt, 1, 0, sm, dq)
        assert pa.pa_last_error(c.h) == 0
        check_rows(host(dq), q, c, [(s, s, n - 1) for s, n in enumerate(lengths)], 1, 0, sm, DECODE_STEP)


@pytest.mark.parametrize("n_ctx", [30, 700, 9000])
@pytest.mark.parametrize("ratio", [20, 40, 100])
def test_decode_beside_a_row_that_is_far_larger(n_ctx, ratio):
    """A V row 2^ratio larger than the others, whose weight is next to nothing: the outputs are the others'."""
    import windowed_prefill_attention_gb300 as pa
    sm = 1 / 128  # weights much alike
    q = np.tile(bf16_round(np.random.default_rng(11).standard_normal((1, 1, D)).astype(np.float32)), (1, 4, 1))

    def change(k, v, slots):
        for pages, rows in slots:
            for at in (0, len(pages) // 2):  # scores far under the others'
                g = q[0, 0].astype(np.float64)
                k[pages[at], rows[at]] = -g * (1.6 * ratio * np.log(2) / (g @ g) / sm)
                v[pages[at], rows[at]] *= 2.0 ** ratio

    c = cache_of(62, [n_ctx], 4, 1, change)
    dq = dev_bf16(q)
    pa.pa_kv4_decode(c.h, np.array([(0, n_ctx - 1, 1, n_ctx)], np.int32), dq, c.d_tiles, c.d_bt, 1, 0, sm, dq)
    assert pa.pa_last_error(c.h) == 0
    check_rows(host(dq), q, c, [(0, 0, n_ctx - 1)], 1, 0, sm, DECODE_STEP)


@pytest.mark.parametrize("exponent", [-119, -122, -124, -126, -130])
def test_decode_of_tiny_queries_on_great_keys(exponent):
    """Queries down to bf16's subnormal values, keys of up to 2^122: scores of a few units all the same."""
    import windowed_prefill_attention_gb300 as pa
    rng = np.random.default_rng(12)
    q = bf16_round(np.ldexp(rng.uniform(1, 2, (1, 4, D)) * rng.choice([-1, 1], (1, 4, D)), exponent).astype(np.float32))

    def change(k, v, slots):
        k[:] = np.ldexp(bf16_round(rng.standard_normal(k.shape).astype(np.float32)), 120)

    c = cache_of(63, [200], 4, 2, change)
    sm = float(np.ldexp(1.0, -exponent - 120 - 3))
    dq = dev_bf16(q)
    pa.pa_kv4_decode(c.h, np.array([(0, 199, 1, 200)], np.int32), dq, c.d_tiles, c.d_bt, 1, 0, sm, dq)
    assert pa.pa_last_error(c.h) == 0
    check_rows(host(dq), q, c, [(0, 0, 199)], 1, 0, sm, DECODE_STEP)
