"""The quotient of the 8-bit codes, v / s by the rounded inverse and one correction, evaluated
in exact arithmetic: it can round apart from the division only where the quotient lies within
2^-22 of a step of the middle between two floats.  Beside the borders between codes (an odd
number of at most 8 bits times a power of two) every such pair is tried (no GPU needed)."""
from fractions import Fraction as F


def rounded(x):
    """x > 0 or x < 0 to 24 bits, to nearest even."""
    if x == 0:
        return x
    sign, x = (-1, -x) if x < 0 else (1, x)
    e = x.numerator.bit_length() - x.denominator.bit_length()
    while F(2) ** e > x:
        e -= 1
    while F(2) ** (e + 1) <= x:
        e += 1
    return sign * round(x / F(2) ** (e - 23)) * F(2) ** (e - 23)  # (round: half to even)


def corrected(v, s):
    inv = rounded(1 / s)
    q = rounded(v * inv)
    return rounded(q + rounded(v - q * s) * inv)


def test_the_corrected_quotient_beside_every_border():
    tried = 0
    for T in range(1, 255, 2):
        bits = T.bit_length()
        for side in (1, -1):
            middle = (T << (25 - bits)) + side  # 25 bits: half a step beside the border
            # v 2^k = s * middle + D with |D| <= 6 needs the scale's 24 bits within 6 of a multiple of 2^(25 - bits)
            for j in range(1 << bits):
                for eps in range(-6, 7):
                    S = (j << (25 - bits)) + eps
                    if not 1 << 23 <= S < 1 << 24:
                        continue
                    P = S * middle
                    k = P.bit_length() - 24
                    V = (P + (1 << (k - 1))) >> k
                    if abs((V << k) - P) > 6 or V >> 24:
                        continue
                    v, s = F(V << k, 1 << 48), F(S, 1 << 23)
                    assert corrected(v, s) == rounded(v / s), (T, side, S, V)
                    tried += 1
    assert tried > 100
