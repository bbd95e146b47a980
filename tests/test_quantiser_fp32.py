"""CPU proofs, in exact arithmetic, of the quantiser of fp32 rows (keys that
come normed and turned): its scale and its codes are those of correctly rounded
quotients, without a division.

* Scale: q0 = RN(a r), r = RN(1/127), q1 = RN(q0 + (a - 127 q0) r) is RN(a / 127)
  for every binary32 significand of a, and where the result is subnormal.
* Codes: r0 approximates 1/b within a unit in its last place (what the hardware
  reciprocal is documented to give), r = RN(r0 + r0 RN(1 - r0 b)), q0 = RN(a r),
  q1 = RN(q0 + (a - q0 b) r).
  r is within (1/2 + 2^-22) units of 1/b, so |1 - b r| < 1.01 2^-25 b (b in
  [1, 2)) and |a/b - q0| < 1.5 units of q0, and q0 + (a - q0 b) r is off by
  (a/b - q0)(1 - b r), under 2^-23 units.  q1 and RN(a / b) therefore differ only
  where a/b is that near to the middle between two binary32 values, and round to
  different codes only where one of the two is a tie n + 1/2.  The quotients next
  to those middles are a/b = mid + k / (2^j b), k a small integer: with mid =
  M / 2^s the pairs solve A 2^t - M b = k, so b is -k / M modulo 2^t.  All of them
  with |k| <= 6 (the bound above leaves |k| <= 2) are run through the steps.  One
  of them hangs on the approximation: 2^23 / (2^24 - 1), which test_qkv_rows.py
  holds on the GPU."""
import math
from fractions import Fraction

import numpy as np

from test_quantiser_math import _rn32


def test_scale_is_the_rounded_quotient_for_every_significand():
    r = np.float64(np.float32(1.0) / np.float32(127.0))
    a = (np.arange(1 << 23, 1 << 24, dtype=np.uint32).astype(np.float32) * np.float32(2.0 ** -23)).astype(np.float64)
    q0 = (a * r).astype(np.float32).astype(np.float64)  # 48 bits: one rounding
    rem = a - 127.0 * q0                                # exact in 53 bits
    assert np.array_equal(rem.astype(np.float32).astype(np.float64), rem)
    # a / 127 is at least 2^-8 of a unit from the middle between two binary32 values, so that the roundings to 53 bits
    # on the way to 24 change nothing
    got = (q0 + rem * r).astype(np.float32)
    assert np.array_equal(got, (a / 127.0).astype(np.float32))


def test_scale_is_the_rounded_quotient_where_it_is_subnormal():
    r = np.float64(np.float32(1.0) / np.float32(127.0))
    a = np.arange(1 << 24, dtype=np.float64)  # in units of 2^-149
    q0 = np.rint(a * r)
    got = np.rint(q0 + (a - 127.0 * q0) * r)
    assert np.array_equal(got, np.rint(a / 127.0))


def reciprocals(b):
    """What the Newton step makes of every approximation within a unit of 1/b, b an integer in [2^23, 2^24)."""
    exact = _rn32(Fraction(1, b))
    unit = Fraction(1, 2 ** 47) if b > 1 << 23 else Fraction(1, 2 ** 46)  # of [2^-24, 2^-23)
    out = set()
    for d in (-1, 0, 1):
        r0 = exact + d * unit
        out.add(_rn32(r0 + r0 * _rn32(1 - r0 * b)))
    return out


def quotient(a, b, r):
    q0 = _rn32(a * r)
    rem = a - q0 * b
    assert _rn32(rem) == rem  # one FMA gives it exactly
    return _rn32(q0 + rem * r)


def near_pairs(n, k_most=6):
    """(a, b), significands of 24 bits and a's exponent such that a/b is within k_most / (2^j b) of the middle between
    n + 1/2 and its neighbours."""
    tie = Fraction(2 * n + 1, 2)
    e = math.floor(math.log2(tie))
    up, down = Fraction(2) ** (e - 23), Fraction(2) ** (e - 23) / (2 if tie == Fraction(2) ** e else 1)
    for mid in (tie + up / 2, tie - down / 2):
        M, s = mid.numerator, mid.denominator.bit_length() - 1
        assert M % 2 == 1 and mid == Fraction(M, 2 ** s)
        for ea in (e + 22, e + 23, e + 24):  # a = A 2^(ea - 23), near mid b
            t = ea - 23 + s
            if t <= 0:
                continue
            inverse = pow(M, -1, 1 << t)
            for k in range(-k_most, k_most + 1):
                first = (-k * inverse) % (1 << t)
                first += -(-max(0, (1 << 23) - first) // (1 << t)) * (1 << t)
                for b in range(first, 1 << 24, 1 << t):
                    A, rest = divmod(M * b + k, 1 << t)
                    assert rest == 0
                    if 1 << 23 <= A < 1 << 24:
                        yield A * Fraction(2) ** (ea - 23), b


def test_codes_are_those_of_the_rounded_quotient():
    n_pairs, hang = 0, set()
    for n in range(128):
        for a, b in near_pairs(n):
            want = _rn32(a / b)
            for r in reciprocals(b):
                n_pairs += 1
                if quotient(a, b, r) != want:
                    hang.add((a, b, r < Fraction(1, b)))
    assert n_pairs > 1000
    # just above 1/2 + 2^-25: 1, but 0 with the reciprocal's lower neighbour, on which the step ends from itself
    assert hang == {(Fraction(1 << 23), (1 << 24) - 1, True)}
    ones = (1 << 24) - 1
    assert reciprocals(ones) == {Fraction(1, 1 << 24), _rn32(Fraction(1, ones))}
