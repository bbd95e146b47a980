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
