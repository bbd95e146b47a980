"""CPU: the turns that pa_rope_init makes of frequencies, against exact arithmetic."""
from fractions import Fraction

import numpy as np
import pytest

from test_qkv_host import pa  # noqa: F401

# pi to 110 decimals: 1e-110 of it times the largest frequency here is 2^-298
PI = Fraction(int("3" + "14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706"
                  "798214808651"), 10 ** 110)


def off(turn, pos, freq):
    """Distance, in turns, of pos * turn / 2^64 from pos * freq / (2 pi), whole turns aside."""
    want = pos * Fraction(freq) / (2 * PI)
    d = Fraction(turn * pos, 2 ** 64) - want
    return abs(d - round(d))


def check(pa, freqs):  # noqa: F811
    for i in range(0, len(freqs), 128):
        part = np.zeros(128)
        part[: len(freqs[i:i + 128])] = freqs[i:i + 128]
        r = pa.pa_rope_init(part)
        for j, f in enumerate(part):
            for pos in (1, -1, 131072, 2 ** 31 - 1, -2 ** 31):
                # half of the fraction's last bit a position, and the 256-bit constant's own end (2^-256 of 2^53 at most)
                assert off(r.turn[j], pos, float(f)) <= abs(pos) * (Fraction(1, 2 ** 65) + Fraction(1, 2 ** 130)), (f, pos)


def test_turns_are_rounded_once(pa):  # noqa: F811
    """Usual tables; frequencies of many turns a position (an angle of 2e13 rad at the last position); tiny ones."""
    check(pa, list(10000.0 ** (-np.arange(128) / 128.0)) + list(1e6 ** (-np.arange(32) / 32.0)))
    check(pa, [1e4, -1e4, 7.25, -0.3, 2 * np.pi, -2 * np.pi, np.pi, 6.283185307179587 * 1000, 1e15, 2.0 ** 53, 3.7e18,
               np.nextafter(2.0 ** 64, 0), -np.nextafter(2.0 ** 64, 0), 1e-9, 2.0 ** -61, 2.0 ** -62, -2.0 ** -63, 1e-30,
               2.0 ** -200, 5e-324, -5e-324, 0.0, -0.0])
    rng = np.random.default_rng(0)
    check(pa, list(rng.choice((-1, 1), 512) * 2.0 ** rng.uniform(-70, 64, 512)))


@pytest.mark.parametrize("freq", (2.0 ** 64, -2.0 ** 64, 1e300, np.inf, -np.inf, np.nan))
def test_frequencies_past_the_fraction_are_refused(pa, freq):  # noqa: F811
    with pytest.raises(pa.PAError):
        pa.pa_rope_init([1.0] * 7 + [freq])
