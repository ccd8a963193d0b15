"""Inputs and error bounds that show how exactly the 4-bit attention computes.

Every query row has one channel that is not zero.  A score is then one product of a value of six significant bits and
one of eight, exact in float32, and what is left is the precision of the weights, of the second product and
of the sums.  Bounds are relative to the largest |v|, in units of u = 2^-24; scores lie within +-2 in log2 units.

A weight:
  12  its score's factor (the softmax scale, log2 e, their product and the product with the score: 4 u of at
      most 2) and the subtraction of the maximum, a whole number (a difference below 8: half a step is 4 u),
      times ln 2: 8.4; the exponential, within 2^-22: 4
A result, from weights off by e each (2 e at most, as numerator and denominator are off), and
   4  the weights' second fp16 part, rounded at 2^-22 of the weight
  68  the second product's sums in the matrix instructions: at most four of them add up a unit of 32 tokens, each cuts
      off its 16 products and its accumulator at 24 bits of the largest
   7  the denominator: four additions per lane and three over the lanes
   2  the quotient and its product
   6  the addition of two partials in numerator and denominator, and their factors, which are powers of two
"""
import numpy as np

from oracle import zf_step_oracle as S

U24 = 2.0 ** -24
WEIGHT = 12.4
ONE_UNIT = (2 * WEIGHT + 4 + 68 + 7 + 2 + 6) * U24
# log-sum-exp of one unit: weights and their sum; the logarithm (a step of 2^-20 at up to 12, half a step of
# the addition), the product with ln 2 (two roundings of at most 5)
ONE_UNIT_LSE = (WEIGHT + 7 + 0.7 * (16 + 4) + 10) * U24


def chain(units, merged=168):
    """A range of `units` units whose weights differ, and a merge of `merged` additions in a row: besides one unit's
    errors, each addition to the result rounds to nearest, an error of at most u times the running sum, either
    way alike: over n additions a standard deviation of u sqrt(n) / 3.  Six of them: the result's n, the
    denominator's (4 n additions in each of 8 lanes), the merge's in both.  (Sums cut off instead lose 0.36 of
    a step of 2 u per addition and instruction, at half the final sum on the average: 0.36 u of the result per
    unit and instruction, of which a unit has two up to 4 columns, else four.)"""
    return ONE_UNIT + 6 * (np.sqrt(units) + np.sqrt(units / 2) + 2 * np.sqrt(merged)) / 3 * U24


def repeated(additions, shares):
    """Error of a sum of many additions of few different numbers (shares: how often each occurs, adding up to 1).
    While a sum stays between two powers of two its step is fixed, and adding the same number to any multiple
    of the step is off by the same: equal numbers err alike, in every lane and range.  Each different number's
    error has a standard deviation of 0.29 steps; a sum of n additions meets steps of 2 u of its final value in
    its last half, of half that in the quarter before, and so on, 4/3 u n in all: six times 0.29 times 4/3 u n
    sqrt(sum of shares^2)."""
    return 6 * 0.29 * 4 / 3 * additions * np.sqrt((np.asarray(shares) ** 2).sum()) * U24


def queries(rng, k, rows, scale, channels=1):
    """BF16 bits [rows][128]: `channels` channels each (one: exact scores), which add up to scores within +-2 log2 units
    over the keys k [n][128] (float64)."""
    q = np.zeros((rows, 128))
    for r in range(rows):
        for c in rng.permutation(128)[:channels] if channels > 1 else [int(rng.integers(0, 128))]:
            top = max(np.abs(k[:, c]).max(), 1e-6)
            q[r, c] = rng.choice([-1, 1]) * rng.uniform(0.5, 0.99) * 2 * np.log(2) / scale / top / channels
    return S.f64_to_bf16(q)


def attend(k, v, q_bits, scale, rounded=lambda p: p):
    """float64 attention of query rows over k, v [n][128]: (out, lse).  rounded: what happens to the numerator's
    weights (1 at the maximum)."""
    s = (S.bf16_to_f64(q_bits) @ k.T) * scale
    top = s.max(-1, keepdims=True)
    p = np.exp(s - top)
    return rounded(p) @ v / p.sum(-1, keepdims=True), top[:, 0] + np.log(p.sum(-1))
