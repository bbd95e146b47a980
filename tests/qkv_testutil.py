"""Plain numpy forms, in 64 bits, of the norm / rotation / append calls, and the
bounds their results are held to."""
import numpy as np

D = 256
# Roundings, each at most half a step: bf16 2^-8 and fp32 2^-24 of the value.
BF16 = 2.0 ** -8
# fp32 work before the last rounding: the sum of 256 squares (8 + 5 additions deep), the reciprocal square root
# (2 ulp), gain, cosine / sine (2 ulp, and 2^-24 of the turned pair from the angle's own rounding), three products
# and a sum: under 40 roundings of 2^-24, relative to the row's scale times the pair's magnitudes.
FP32 = 40 * 2.0 ** -24


def bf16_bits(x):
    b = np.asarray(x, dtype=np.float32).view(np.uint32)
    return ((b + np.uint32(0x7FFF) + ((b >> np.uint32(16)) & np.uint32(1))) >> np.uint32(16)).astype(np.uint16)


def bf16_values(bits):
    return (bits.astype(np.uint32) << np.uint32(16)).view(np.float32).astype(np.float64)


def frequencies(rot, base=10000.0):
    return base ** (-np.arange(rot // 2, dtype=np.float64) / max(1, rot // 2))


def norm_rope(x, w, offset, eps, inv_freq=(), axis=None, positions=None, halves=True):
    """x float64 [tokens, heads, 256], w float64 [256] or None, positions int [axes, tokens].  Returns the rows
    and, per value, the magnitudes its rounding errors are relative to."""
    x = np.asarray(x, np.float64)
    ms = (x * x).mean(-1, keepdims=True) + eps
    r = np.where(ms > 0, 1.0 / np.sqrt(np.where(ms > 0, ms, 1.0)), 0.0)
    y = x * r * (1.0 if w is None else offset + w)
    size = np.abs(x * r) * (1.0 if w is None else np.abs(offset) + np.abs(w))
    half = len(inv_freq)
    if half == 0:
        return y, size
    inv_freq = np.asarray(inv_freq, np.float64)
    axis = np.zeros(half, int) if axis is None else np.asarray(axis)
    angle = np.asarray(positions, np.float64)[axis].T * inv_freq  # [tokens, pairs]
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    first = np.arange(half) if halves else 2 * np.arange(half)
    second = first + (half if halves else 1)
    out, mag = y.copy(), size.copy()
    out[..., first] = y[..., first] * c - y[..., second] * s
    out[..., second] = y[..., second] * c + y[..., first] * s
    # the reference's own angle is rounded to 53 bits twice
    far = 1.0 + (2 * 2.0 ** -53 * np.abs(angle) / FP32)[:, None]
    mag[..., first] = mag[..., second] = (size[..., first] + size[..., second]) * far
    return out, mag


def assert_rows(got, ref, mag, what=""):
    """bf16 rows against the 64-bit ones: half a bf16 step of the value, plus the fp32 work."""
    bound = BF16 * np.abs(ref) + (1 + BF16) * FP32 * mag + 2.0 ** -133  # half the smallest bf16 subnormal's step
    err = np.abs(np.asarray(got, np.float64) - ref)
    assert np.all(err <= bound), (what, float((err / np.maximum(bound, 1e-300)).max()))


def assert_codes(codes, scale, ref, mag, what=""):
    """int8 codes and fp32 scales of rows against the 64-bit rows: scale = absmax / 127 to fp32 work, and every
    value within half a step, plus the fp32 work (the scale's part times up to 127 steps)."""
    absmax = np.abs(ref).max(-1)
    slack = FP32 * mag.max(-1)
    assert np.all(np.abs(scale * 127.0 - absmax) <= slack + 2.0 ** -23 * absmax), what
    err = np.abs(codes * scale[..., None].astype(np.float64) - ref)
    bound = 0.5 * absmax[..., None] / 127.0 + FP32 * mag + 2 * slack[..., None] + 2.0 ** -22 * absmax[..., None]
    assert np.all(err <= bound), (what, float((err / np.maximum(bound, 1e-300)).max()))
    assert np.all(np.abs(codes.astype(int)) <= 127)
