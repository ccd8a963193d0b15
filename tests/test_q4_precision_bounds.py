"""The bounds of the 4-bit attention's precision tests see the mistakes they are there for: planted in the
oracle's arithmetic, on the CPU."""
import numpy as np

from oracle import zf_step_oracle as S
from tests import q4_precision as P


def keys_and_values(n, seed):
    rng = np.random.default_rng(seed)
    k = S.bf16_to_f64(S.f64_to_bf16(rng.standard_normal((n, 128))))
    v = S.bf16_to_f64(S.f64_to_bf16(np.abs(rng.standard_normal((n, 128))) + 0.5))
    return rng, k, v


def cut(x, bits):
    m, e = np.frexp(x)
    return np.ldexp(np.trunc(m * 2.0 ** bits) / 2.0 ** bits, e)


def test_weights_without_their_second_part_are_seen():
    for n in (1, 2, 5, 32):
        rng, k, v = keys_and_values(n, n)
        q = P.queries(rng, k, 8, 128 ** -0.5)
        out, lse = P.attend(k, v, q, 128 ** -0.5)
        # weights are taken below the largest score's next whole number in log2 units
        top = (S.bf16_to_f64(q) @ k.T).max(-1, keepdims=True) * 128 ** -0.5 / np.log(2)
        f = 2.0 ** (top - np.ceil(top))
        bad, _ = P.attend(k, v, q, 128 ** -0.5, lambda p: cut(p * f, 11) / f)
        two, _ = P.attend(k, v, q, 128 ** -0.5, lambda p: (cut(p * f, 11) + cut(p * f - cut(p * f, 11), 11)) / f)
        assert (np.abs(bad - out).max(-1) > 4 * P.ONE_UNIT * v.max()).any()
        assert (np.abs(two - out).max(-1) <= P.ONE_UNIT * v.max()).all()


def test_sums_that_are_cut_off_are_seen():
    """A range of 4000 units with two instructions per unit on one chain, against additions that round."""
    units = 4000
    rng = np.random.default_rng(1)
    x = rng.uniform(1, 4, (2 * units, 64)).astype(np.float32)
    exact = x.astype(np.float64).sum(0)
    cuts, rounds = np.zeros(64, np.float32), np.zeros(64, np.float32)
    for row in x:
        cuts = cut(cuts.astype(np.float64) + row, 24).astype(np.float32)
        rounds = rounds + row
    assert (np.abs(cuts - exact) / exact > 3 * P.chain(units)).all()
    assert (np.abs(rounds - exact) / exact < P.chain(units) / 3).all()


def test_few_different_numbers_err_alike():
    """The same number added again and again is off the same way each time: more than independent errors allow,
    within the bound for repeated numbers."""
    n = 16000
    rng = np.random.default_rng(2)
    for different in (20, 100):
        values = rng.uniform(8, 128, (different, 64)).astype(np.float32)
        total, exact = np.zeros(64, np.float32), np.zeros(64)
        for i in rng.integers(0, different, n):
            total = total + values[i]
            exact += values[i]
        off = np.abs(total - exact) / exact
        assert (off <= P.repeated(n, [1 / different] * different)).all()
        assert (off > 6 * np.sqrt(n) / 3 * P.U24).any()
