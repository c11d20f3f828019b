"""The rotation's frequencies as whole numbers, against rational arithmetic (no GPU needed)."""
import random
from fractions import Fraction

import pytest


@pytest.fixture(scope="module")
def s():
    import substitute_speculative_decoding_gb300 as s
    return s


def _arctan_of_inverse(n, bits):
    total, term, k, sign = 0, (1 << bits) // n, 1, 1
    while term:
        total += sign * (term // k)
        term //= n * n
        k, sign = k + 2, -sign
    return total


# 2 pi to some 380 bits (Machin: pi / 4 = 4 arctan(1/5) - arctan(1/239))
TWO_PI = Fraction(8 * (4 * _arctan_of_inverse(5, 400) - _arctan_of_inverse(239, 400)), 1 << 400)


def exact_step(freq: float) -> Fraction:
    """freq / (2 pi) without its whole turns, in units of 2^-64."""
    return Fraction(freq) / TWO_PI % 1 * 2 ** 64


FREQS = [0.0, 1.0, 2.0, 0.1, 3.0, 1e-3, 6.283185307179586, 6.283185307179587, 3.141592653589793, 1e6, 999999.7,
         999999.9999999999, 65536.0, 2.0 ** -33, 2.0 ** -52, 2.0 ** -63, 2.0 ** -64, 1e-18, 1e-19, 1e-20, 1e-30,
         2.0 ** -1022, 5e-324]


@pytest.mark.parametrize("d", [64, 128])
def test_every_bit_of_a_step_is_right(s, d):
    rng = random.Random(d)
    todo = FREQS + [10.0 ** rng.uniform(-20, 6) for _ in range(500)] + [rng.uniform(0, 1e6) for _ in range(500)]
    while todo:
        freqs, todo = todo[:d // 2], todo[d // 2:]
        r = s.rope(d, freqs=freqs + [0.0] * (d // 2 - len(freqs)))
        for f, step in zip(freqs, r.step):
            off = (step - exact_step(f)) % 2 ** 64
            # to the nearest, as far as 190 bits of 1 / (2 pi) times 53 of the frequency tell
            assert min(off, 2 ** 64 - off) <= Fraction(1, 2) + Fraction(1, 2 ** 60), f
        assert list(r.step[d // 2:]) == [0] * (64 - d // 2)


@pytest.mark.parametrize("d,theta", [(64, 1e4), (128, 5e5), (128, 1e6), (64, 1.0), (128, 1e12)])
def test_steps_of_a_base(s, d, theta):
    r = s.rope(d, theta)
    for i in range(d // 2):
        # the power is a double that is less than a unit in its last place off
        f, step = theta ** (-2.0 * i / d), exact_step(theta ** (-2.0 * i / d))
        off = abs(r.step[i] - step)
        assert min(off, 2 ** 64 - off) <= 2 * Fraction(f) * 2 ** 64 / 2 ** 52 / TWO_PI + 1
