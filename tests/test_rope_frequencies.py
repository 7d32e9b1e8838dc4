"""What a Rope is made of: frequencies that are none are refused (on the host)."""
import math

import pytest

torch = pytest.importorskip("torch")

import serving_mog_decode_gb300 as mog

YARN = dict(type="yarn", factor=4, original_len=4096)
BANDS = dict(type="bands", factor=4, original_len=4096)


@pytest.mark.parametrize("at", [0, 17, 31])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_frequencies_that_are_not_finite_are_refused(bad, at):
    f = [0.5 ** i for i in range(32)]
    f[at] = bad
    for given in (f, torch.tensor(f), torch.tensor(f, dtype=torch.float64)):
        with pytest.raises(ValueError, match="finite"):
            mog.Rope(64, inv_freq=given, device="cpu")
    assert mog.Rope(64, inv_freq=[0.0] * 32, device="cpu").turns.eq(0).all()


@pytest.mark.parametrize("base", [0.0, -10000.0, math.nan, math.inf])
def test_bases_that_have_no_frequencies_are_refused(base):
    for scaling in (None, dict(type="linear", factor=2), dict(type="ntk", factor=2), YARN, BANDS):
        with pytest.raises(ValueError, match="base"):
            mog.rope_frequencies(64, base, scaling)
    with pytest.raises(ValueError, match="base"):
        mog.Rope(64, base=base, device="cpu")


@pytest.mark.parametrize("scaling", [dict(type="linear", factor=math.inf), dict(type="ntk", factor=math.nan), dict(YARN, factor=-1),
                                     dict(YARN, original_len=0), dict(BANDS, original_len=-5), dict(BANDS, original_len=math.nan),
                                     dict(YARN, attention_factor=math.inf)])
def test_scalings_that_are_none_are_refused(scaling):
    with pytest.raises(ValueError):
        mog.Rope(64, scaling=scaling, device="cpu")
    with pytest.raises(ValueError, match="base"):
        mog.rope_frequencies(64, 1.0, YARN)


def two_pi(bits):
    """2 pi * 2^bits, to a few units: Machin's formula in whole numbers."""
    def arctan_of_inverse(x, one):
        total, term, k = 0, one // x, 1
        while term:
            total += term // k if k % 4 == 1 else -(term // k)
            term, k = term // (x * x), k + 2
        return total

    one = 1 << bits + 16
    return 8 * (4 * arctan_of_inverse(5, one) - arctan_of_inverse(239, one)) >> 16


def test_turns_are_rounded_once():
    """A frequency's 64-bit fraction of a turn is the nearest one, so that an angle is off by at most 2^-34 of a turn at
    any 32-bit position (2^-65 * 2^31)."""
    tau = two_pi(256)
    f = mog.rope_frequencies(128, 500000.0)[0] + mog.rope_frequencies(128, 10000.0, YARN)[0]
    f += [-x for x in f[1:30]] + [7.0, 2 * math.pi, 1e6 / 3, -1e6 / 7, 0.0, 2.0 ** -40]
    f += [0.0] * (-len(f) % 64)
    for i in range(0, len(f), 64):
        part = f[i:i + 64]
        for x, t in zip(part, mog.Rope(128, inv_freq=part, device="cpu").turns.tolist()):
            num, den = x.as_integer_ratio()
            off = (t * den * tau - (num << 320)) % (den * tau << 64)  # (t - 2^64 x / 2 pi) * den * tau
            off = min(off, (den * tau << 64) - off)
            assert 2 * off <= den * tau * (1 + 2.0 ** -30), (x, off / (den * tau))
