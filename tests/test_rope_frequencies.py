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
