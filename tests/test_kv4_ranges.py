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


def largest_share(q, c, s, t, S, W, sm, least):
    """[HQ]: of a query token the largest weight x V row scale, over the sum of the weights; no scale counts less than
    least(the sequence's largest)."""
    hq, hkv = q.shape[0], c.hkv
    n = len(c.k[s])
    scale = c.tiles[c.bt[s, np.arange(n) // PAGE], :, 4672:].copy().view(np.float32).reshape(n, hkv, PAGE)
    scale = scale[np.arange(n), :, np.arange(n) % PAGE].astype(np.float64)
    scale = np.maximum(scale, least(scale.max()))
    j = np.arange(min(n, t + 1))
    if W > 0:
        j = j[(j // PAGE < S) | (j // PAGE >= max(0, t // PAGE + 1 - W))]
    out = np.zeros(hq)
    for h in range(hq):
        y = sm * (c.k[s][j, h // (hq // hkv)] @ q[h])
        p = np.exp(y - y.max())
        out[h] = (p * scale[j, h // (hq // hkv)]).max() / p.sum()
    return out


def check_rows(got, q, c, rows, S, W, sm, half_step, least):
    """Against the 64-bit definition.  A weight x row scale is held in fp16 under a power of two of the row's own:
    2^-11 of it, or, where it leaves fp16's normal range, half_step of the row's largest; V's codes under their block
    scales are at most 2688.  For the choice of that power of two a scale counts as `least` at least, a row of zeros too."""
    worst = 0.0
    for row, s, t in rows:
        qq = q[row].astype(np.float64)
        ref, bound = attention(qq, c.k[s], c.v[s], t, S, W, sm, 0.0)
        bound = bound + half_step * 2688 * (t + 1) * largest_share(qq, c, s, t, S, W, sm, least)[:, None]
        assert np.isfinite(got[row]).all(), (row, s, t)
        worst = max(worst, float((np.abs(got[row] - ref) / bound).max()))
    assert worst <= 1.0, worst


# decode: the largest product is at least 2^6 in its units (a reference up to 2^8 behind, a significand of 1/2 or more)
# with scales of 2^-100 and less at 2^-99.  A weight under 2^-126 of the largest, which fp32 does not hold, is 0: with any
# scale a product of at most 2^-126 x the largest scale, half_step of 2^-95 of that scale.
DECODE_STEP = 2.0 ** (-25 - 6), lambda most: max(2.0 ** -99, most * 2.0 ** -95)
# prefill: at least 2^-13 (the first reference lies 2^6 above the first tile's largest, the normaliser 2^6 above the least
# scale, a significand of 1/2 or more), scales of 2^-100 and less at 2^-99 again.  Weights are 0 under 2^-120 of the largest,
# half_step of 2^-106 of the largest scale, or where a product is 2^-17 of the row's largest, under half_step of that.
PREFILL_STEP = 2.0 ** (-25 + 13), lambda most: max(2.0 ** -99, most * 2.0 ** -106)


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
        check_rows(host(dq), q, c, [(s, s, n - 1) for s, n in enumerate(lengths)], 1, 0, sm, *DECODE_STEP)


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
    check_rows(host(dq), q, c, [(0, 0, n_ctx - 1)], 1, 0, sm, *DECODE_STEP)


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
    check_rows(host(dq), q, c, [(0, 0, 199)], 1, 0, sm, *DECODE_STEP)


# whole units (few keys; many pieces of them), split ones
PREFILLS = [[(0, 90), (100, 33)], [(1500, 40)], [(700, 5), (40, 20)]]


def prefill(c, pieces, q, S, W, sm, gate=None, options={}):
    """pa_kv4_prefill of each piece (cached, new), rows end to end -> out, [(row, sequence, position)]."""
    import torch

    import windowed_prefill_attention_gb300 as pa
    off = np.cumsum([0] + [n for _, n in pieces])
    seqs = np.array([(off[s], a, n, a + n) for s, (a, n) in enumerate(pieces)], np.int32)
    dq = dev_bf16(q)
    out = torch.full_like(dq, 7.0)
    h = pa.Handle(c.hq, c.hkv, c.n_pool, c.max_pages, **options)
    pa.pa_kv4_prefill(h.h, seqs, dq, c.d_tiles, c.d_bt, S, W, sm, out, q_gate=gate)
    assert pa.pa_last_error(h.h) == 0
    return host(out), [(off[s] + i, s, a + i) for s, (a, n) in enumerate(pieces) for i in range(n)]


@pytest.mark.parametrize("pieces", PREFILLS)
@pytest.mark.parametrize("ratio", [12, 20, 60])
def test_prefill_behind_which_a_far_larger_row_lies(pieces, ratio):
    """The last token's V row 2^ratio larger than all others: the rows of the tokens before it do not see it, those beside it
    in its block of 16 neither, and keep all their bits."""
    lengths = [a + n for a, n in pieces]

    def change(k, v, slots):
        for pages, rows in slots:
            v[pages[-1], rows[-1]] *= 2.0 ** ratio

    c = cache_of(64, lengths, 8, 2, change)
    q = random_rows(np.random.default_rng(13), (sum(n for _, n in pieces), 8, D))
    got, rows = prefill(c, pieces, q, 1, 0, 1 / 128)
    check_rows(got, q, c, rows, 1, 0, 1 / 128, *PREFILL_STEP)


@pytest.mark.parametrize("pieces", PREFILLS)
@pytest.mark.parametrize("ratio", [20, 40, 100])
def test_prefill_beside_a_row_that_is_far_larger(pieces, ratio):
    """A first and a middle V row 2^ratio larger than the others, in every row's sight but of next to no weight."""
    lengths = [a + n for a, n in pieces]
    sm = 1 / 128
    base = bf16_round(np.random.default_rng(14).standard_normal(D).astype(np.float32)).astype(np.float64)

    def change(k, v, slots):
        for pages, rows in slots:
            for at in (0, len(pages) // 2):
                k[pages[at], rows[at]] = -base * (1.6 * ratio * np.log(2) / (base @ base) / sm)
                v[pages[at], rows[at]] *= 2.0 ** ratio

    c = cache_of(65, lengths, 4, 1, change)
    q = np.tile(base.astype(np.float32), (sum(n for _, n in pieces), 4, 1))
    got, rows = prefill(c, pieces, q, 1, 0, sm)
    rows = [r for r in rows if r[2] > 0]  # a first token sees nothing else
    check_rows(got, q, c, rows, 1, 0, sm, *PREFILL_STEP)


@pytest.mark.parametrize("pieces", PREFILLS)
@pytest.mark.parametrize("exponent", [-80, 60, 100, 112, 126])
def test_prefill_of_values_at_the_ends_of_the_range(pieces, exponent):
    """V rows of up to 2.8e38 beside ordinary ones and rows of zeros, scores that grow behind the first tile."""
    lengths = [a + n for a, n in pieces]

    def change(k, v, slots):
        for pages, rows in slots:
            x = np.clip(np.ldexp(v[pages, rows], exponent), -2.8e38, 2.8e38)
            x[::5] = v[pages[::5], rows[::5]]
            x[1::7] = 0
            v[pages, rows] = x
            v[pages[0], rows[0]] = np.sign(v[pages[0], rows[0]]) * (2.8e38 if exponent > 0 else 2.0 ** exponent)
            k[pages[: len(pages) // 2], rows[: len(pages) // 2]] *= 2.0 ** -6

    c = cache_of(66, lengths, 8, 2, change)
    q = random_rows(np.random.default_rng(15), (sum(n for _, n in pieces), 8, D))
    for sm in (1 / 16, 0.0):
        got, rows = prefill(c, pieces, q, 1, 0, sm)
        check_rows(got, q, c, rows, 1, 0, sm, *PREFILL_STEP)


@pytest.mark.parametrize("q_mode,p_mode", [(1, 0), (0, 1), (1, 1)])
def test_prefill_on_the_integer_grids_behind_which_a_far_larger_row_lies(q_mode, p_mode):
    """The grids round relative to a row's own largest weight x scale; a later row's scale has no say in it.  Against the
    same call without the large row, whose scores are the same: what each side's weights are off by, fp16's 2^-11 of each
    and half a step of the largest (PREFILL_STEP), or half of the u8 grid's step, 1/255 of the largest; and bf16's 2^-8."""
    pieces = [(0, 60), (400, 30)]
    lengths = [a + n for a, n in pieces]
    q = bf16_round(np.random.default_rng(16).standard_normal((90, 8, D)).astype(np.float32))
    sm = 1 / 128
    outs, caches = [], []
    for ratio in (0, 30):
        def change(k, v, slots):
            for pages, rows in slots:
                v[pages[-1], rows[-1]] *= 2.0 ** ratio
        caches.append(cache_of(67, lengths, 8, 2, change))
        outs.append(prefill(caches[-1], pieces, q, 1, 0, sm, options=dict(q_mode=q_mode, p_mode=p_mode)))
    half_step, least = PREFILL_STEP
    for row, s, t in outs[0][1]:
        if t == lengths[s] - 1:
            continue
        c, qq = caches[0], q[row].astype(np.float64)
        a, b = outs[0][0][row], outs[1][0][row]
        share = largest_share(qq, c, s, t, 1, 0, sm, least)
        for h in range(8):
            kk, vv = c.k[s][: t + 1, h // 4], c.v[s][: t + 1, h // 4]
            y = sm * (kk @ qq[h])
            p = np.exp(y - y.max())
            # the int8 grid moves a score by at most half a code, 1/254 of the query's largest, in each dim
            p *= np.exp(2 * sm * (np.abs(kk).sum(-1) * np.abs(qq[h]).max() / 254).max()) if q_mode else 1.0
            weighed = (p / np.exp(y - y.max()).sum()) @ np.abs(vv)
            bound = 2 * 2.0 ** -8 * np.maximum(np.abs(a[h]), np.abs(b[h])) + 2 * 2.0 ** -133
            steps = 2 * half_step if p_mode == 0 else 1.02 / 255
            bound = bound + 2 * 2.0 ** -11 * weighed + steps * 2688 * (t + 1) * share[h]
            assert np.all(np.abs(a[h] - b[h]) <= bound), (row, h)


@pytest.mark.parametrize("drop", [60, 90, 108, 114, 117, 119, 121, 123, 125, 130])
def test_prefill_on_the_u8_grid_of_tiles_of_next_to_no_weight(drop):
    """Keys behind the first tile whose weights are 2^-drop of those in it: the u8 grid's step for their tile would be
    under fp32's range, or O in units of it over that.  The outputs are the first tile's."""
    base = bf16_round(np.random.default_rng(17).standard_normal(D).astype(np.float32)).astype(np.float64)
    sm = 1 / 16

    def change(k, v, slots):
        for pages, rows in slots:
            for at in range(len(pages)):
                k[pages[at], rows[at]] = -base * (drop * np.log(2) / (base @ base) / sm) if at >= 128 else 0.0

    lengths = [420, 300]
    c = cache_of(68, lengths, 8, 2, change)
    q = np.tile(base.astype(np.float32), (60, 8, 1))
    got, rows = prefill(c, [(380, 40), (280, 20)], q, 1, 0, sm, options=dict(p_mode=1))
    for row, s, t in rows:
        for h in range(8):
            vv = c.v[s][:128, h // 4]
            # half a step of the grid, 1/255 of the tile's largest weight x scale, for each key; codes are at most 2688
            scale = np.abs(vv).max()
            bound = 2.0 ** -8 * np.abs(vv.mean(0)) + 0.51 / 255 * scale + 2.0 ** -10 * np.abs(vv).mean(0) + 2.0 ** (7 - drop) * scale
            assert np.all(np.abs(got[row, h] - vv.mean(0)) <= bound), (row, h)


@pytest.mark.parametrize("drop", [90, 108, 117, 123])
def test_int8_prefill_on_the_u8_grid_of_tiles_of_next_to_no_weight(drop):
    """The same of the int8 pool: V codes of the first 128 keys, K codes of 0 there, a large negative score behind."""
    import torch

    import windowed_prefill_attention_gb300 as pa
    rng = np.random.default_rng(18)
    n, new, sm = 420, 40, 1 / 16
    pages = -(-n // PAGE)
    codes = rng.integers(-127, 128, D)
    kc = np.zeros((pages, PAGE, 2, D), np.int8)
    kc.reshape(-1, 2, D)[128:] = -codes
    vc = rng.integers(-127, 128, (pages, PAGE, 2, D)).astype(np.int8)
    q = bf16_round(np.tile(codes.astype(np.float32) / 64, (new, 8, 1)))
    ks = np.full((pages, PAGE, 2), drop * np.log(2) / sm / (q[0, 0].astype(np.float64) @ codes), np.float32)
    vs = np.full((pages, PAGE, 2), 0.01, np.float32)
    kc, vc, ks, vs = (torch.from_numpy(x).cuda() for x in (kc, vc, ks, vs))
    dq, bt = dev_bf16(q), torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    out = torch.zeros_like(dq)
    h = pa.Handle(8, 2, pages, pages, p_mode=1)
    pa.pa_prefill_batch(h.h, np.array([(0, n - new, new, n)], np.int32), dq, kc, vc, ks, vs, bt, 1, 0, sm, out)
    assert pa.pa_last_error(h.h) == 0
    for g in range(2):
        v = vc.cpu().numpy().astype(np.float64).reshape(-1, 2, D)[:128, g] * np.float64(np.float32(0.01))
        bound = 2.0 ** -8 * np.abs(v.mean(0)) + 0.51 / 255 * 1.27 + 2.0 ** -10 * np.abs(v).mean(0) + 2.0 ** (7 - drop)
        assert np.all(np.abs(host(out)[:, 4 * g: 4 * g + 4] - v.mean(0)) <= bound)


@pytest.mark.parametrize("pieces", PREFILLS)
@pytest.mark.parametrize("ratio", [8, 16, 30])
def test_prefill_beside_rows_of_zeros(pieces, ratio):
    """Every third V row of zeros, with 2^ratio times the others' weight: the outputs are small, and as right as others."""
    lengths = [a + n for a, n in pieces]
    sm = 1 / 128
    base = bf16_round(np.random.default_rng(19).standard_normal(D).astype(np.float32)).astype(np.float64)

    def change(k, v, slots):
        for pages, rows in slots:
            v[pages[::3], rows[::3]] = 0
            k[pages[::3], rows[::3]] = base * (ratio * np.log(2) / (base @ base) / sm)

    c = cache_of(69, lengths, 8, 2, change)
    q = np.tile(base.astype(np.float32), (sum(n for _, n in pieces), 8, 1))
    got, rows = prefill(c, pieces, q, 1, 0, sm)
    check_rows(got, q, c, rows, 1, 0, sm, *PREFILL_STEP)


@pytest.mark.parametrize("exponent", [-30, -60, -80])
@pytest.mark.parametrize("drop", [30, 60])
def test_prefill_on_the_u8_grid_of_small_values(exponent, drop):
    """Small V rows, and behind the first tile one of little weight, so that the grid's step is small too."""
    base = bf16_round(np.random.default_rng(20).standard_normal(D).astype(np.float32)).astype(np.float64)
    sm = 1 / 16

    def change(k, v, slots):
        for pages, rows in slots:
            k[pages, rows] = 0
            k[pages[128:], rows[128:]] = -base * (drop * np.log(2) / (base @ base) / sm)
            v[pages, rows] = np.ldexp(v[pages, rows], exponent)
            v[pages[5], rows[5]] = 0  # by products, not under one normaliser

    c = cache_of(70, [180], 8, 2, change)
    q = np.tile(base.astype(np.float32), (40, 8, 1))
    got, rows = prefill(c, [(140, 40)], q, 1, 0, sm, options=dict(p_mode=1))
    half_step, least = PREFILL_STEP
    check_rows(got, q, c, rows, 1, 0, sm, half_step + 0.51 / 255, least)
