"""GPU: rows at the edges of fp32 for the norm and the quantiser of pa_qk_norm_rope
and pa_qkv_append, against their formulas."""
import numpy as np
import pytest

import qkv_testutil as ut
from test_qkv import Handle, dev, dev_bf16, empty_rows, normal_bits

pytestmark = pytest.mark.gpu


def append_rows(k, kw, offset, eps, rope=None):
    """Codes and scales of key rows [tokens, heads, 256] (bf16 bits) appended to one sequence."""
    import torch

    import windowed_prefill_attention_gb300 as pa
    n, hkv = k.shape[:2]
    pages = (n + 15) // 16
    kp, vp = (torch.full((pages, 16, hkv, 256), 99, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((pages, 16, hkv), -1.0, device="cuda") for _ in range(2))
    bt = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    kd = dev_bf16(k)
    with Handle(hkv, hkv, pages, pages) as h:
        pa.pa_qkv_append(h, [(0, 0, n, n)], None, kd, kd, None, None if kw is None else dev_bf16(kw), eps, rope, None, bt,
                         kp, vp, ks, vs, None, weight_offset=offset)
        assert pa.pa_last_error(h) == 0
    return kp.view(-1, hkv, 256)[:n].cpu().numpy(), ks.view(-1, hkv)[:n].cpu().numpy()


@pytest.mark.parametrize("half", (45, 46, 50, 60))
def test_codes_of_a_scale_whose_significand_is_all_ones(half):
    """Rows whose values are exact in fp32: the gains offset + w are, and r = 2^-half, since eps = 2^(2 half) swallows a
    mean square under 2^46 (squares of at most (60 2^17)^2 < 2^46).  The largest, 127 - 2^-17 (times r), has the scale
    1 - 2^-24, and a value of 1/2 is then a little more than half a step: code 1, both signs."""
    offset = -2.0 ** -17
    w = np.zeros(256, np.float32)
    w[0], w[1:9] = 127.0, 2.0 ** -16
    x = np.zeros((7, 3, 256), np.float32)
    x[..., 0] = 1.0
    # halves of a step and a little more, and whole steps, of either sign; then values of the other gain
    x[..., 1:9] = 2.0 ** 16 * np.array([1, -1, 3, -3, 2, 5, -127, 253], np.float32)
    x[..., 9:30] = np.random.default_rng(2).integers(-60, 61, (7, 3, 21)) * 2.0 ** 17
    x = ut.bf16_values(ut.bf16_bits(x)).astype(np.float32)
    y = (x * (np.float32(offset) + w)) * np.float32(2.0 ** -half)
    y = y.astype(np.float32)
    codes, scale = append_rows(ut.bf16_bits(x), ut.bf16_bits(w), offset, 2.0 ** (2 * half))
    want_scale = (np.abs(y).max(-1) / np.float32(127)).astype(np.float32)
    assert np.all(want_scale == np.float32((1 - 2.0 ** -24) * 2.0 ** -half))
    want = np.rint((y / want_scale[..., None]).astype(np.float32))
    assert np.all(want[..., 1] == 1) and np.all(want[..., 2] == -1)
    assert np.array_equal(scale, want_scale)
    assert np.array_equal(codes, want.astype(np.int8))


# rows' magnitudes, as powers of two: a normal row, rows whose squares leave fp32's normal range, and its whole range,
# down to bf16's smallest subnormals; zeros
TINY = (0, -19, -21, -60, -62, -63, -64, -66, -70, -74, -75, -80, -100, -120, -126, -130, -133, None)


def tiny_rows(rng, tokens, heads):
    """bf16 bits [tokens, heads, 256], the magnitudes of TINY in turn over tokens and heads; the last token's rows with
    one value that is not zero."""
    x = rng.standard_normal((tokens, heads, 256))
    e = [TINY[i % len(TINY)] for i in range(tokens * heads)]
    x *= np.array([0.0 if k is None else 2.0 ** k for k in e]).reshape(tokens, heads, 1)
    x[-1, :, 1:] = 0
    return ut.bf16_bits(x.astype(np.float32))


@pytest.mark.parametrize("halves, rot", ((True, 128), (False, 256), (True, 0)))
@pytest.mark.parametrize("eps", (0.0, 2.0 ** -149, 2.0 ** -131, 2.0 ** -90, 2.0 ** -41, 1e-6))
def test_norm_of_tiny_rows(eps, halves, rot):
    """With a small eps a row of tiny values has a root mean square of 1 like any other.  Numbers of rows that a warp
    takes four, two and one at a time, tiny ones beside normal ones in a batch."""
    import windowed_prefill_attention_gb300 as pa
    rng = np.random.default_rng(8)
    n, hq, hkv = 33, 14, 7
    q, k = tiny_rows(rng, n, hq), tiny_rows(rng, n, hkv)
    w = normal_bits(rng, 256)
    freq, pos = ut.frequencies(rot), rng.integers(0, 5000, n).astype(np.int32)
    rope = pa.pa_rope_init(freq, pa.PA_ROPE_HALF if halves else pa.PA_ROPE_ADJACENT)
    qo, ko = empty_rows(n, hq), empty_rows(n, hkv)
    with Handle(hq, hkv) as h:
        pa.pa_qk_norm_rope(h, dev_bf16(q), dev_bf16(k), dev_bf16(w), None, eps, rope, dev(pos), qo, ko)
        assert pa.pa_last_error(h) == 0
    eps = float(np.float32(eps))
    for out, bits, gain in ((qo, q, w), (ko, k, None)):
        ref, mag = ut.norm_rope(ut.bf16_values(bits), None if gain is None else ut.bf16_values(gain), 0.0, eps, freq, None,
                                pos[None], halves)
        ut.assert_rows(out.float().cpu().numpy(), ref, mag)


@pytest.mark.parametrize("eps", (0.0, 2.0 ** -140))
def test_append_of_tiny_rows(eps):
    rng = np.random.default_rng(9)
    n, hkv = 40, 7
    k, w = tiny_rows(rng, n, hkv), normal_bits(rng, 256)
    import windowed_prefill_attention_gb300 as pa
    freq = ut.frequencies(64)
    codes, scale = append_rows(k, w, 1.0, eps, pa.pa_rope_init(freq))
    ref, mag = ut.norm_rope(ut.bf16_values(k), ut.bf16_values(w), 1.0, eps, freq, None, np.arange(n)[None])
    ut.assert_codes(codes, scale, ref, mag)
