"""Rotary positions at the ends of 32 bits: as exact as near ones, against angles reduced in whole numbers."""
import math

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import serving_mog_decode_gb300 as mog
from serving_mog_decode_gb300 import buildlib
from test_rope_frequencies import two_pi

pytestmark = pytest.mark.gpu
DEV, D = "cuda", 128


@pytest.fixture(scope="module", autouse=True)
def built():
    buildlib.build()


def angles(freq, positions):
    """Radians within half a turn of zero, [positions][freq], to fp64."""
    tau, rows = two_pi(256), []
    for p in positions:
        row = []
        for x in freq:
            num, den = x.as_integer_ratio()
            turn = (p * num << 376) // (den * tau) % (1 << 120)  # p x / 2 pi, the fraction
            row.append((turn - (1 << 120) if turn >> 119 else turn) * 2 * math.pi / 2.0 ** 120)
        rows.append(row)
    return torch.tensor(rows, dtype=torch.float64, device=DEV)


@pytest.mark.parametrize("start", [(1 << 31) - 33, -(1 << 31), 1 << 30, 0])
@pytest.mark.parametrize("pairs", [False, True])
def test_far_positions_round_once(start, pairs):
    """Before the rounding to bf16 an element is off by at most 3 * 2^-24 of its pair at any position: the fraction's 2^-34 of
    a turn is 2^-31.3 radians; the rest as near position 0 (turn to 2^-32, sine and cosine to a unit, three roundings)."""
    freq = mog.rope_frequencies(128, 500000.0)[0]
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn((1, 33, 200, D), generator=g, device=DEV).bfloat16()
    out = mog.rope(x, torch.tensor([start], dtype=torch.int32, device=DEV), mog.Rope(128, inv_freq=freq, interleaved=pairs))
    z = angles(freq, range(start, start + 33))[:, None]
    c, s, y = torch.cos(z), torch.sin(z), x[0].double()
    ia = torch.arange(0, D, 2, device=DEV) if pairs else torch.arange(D // 2, device=DEV)
    ib = ia + (1 if pairs else D // 2)
    a, b = y[..., ia], y[..., ib]
    for at, want in ((ia, a * c - b * s), (ib, b * c + a * s)):
        half = torch.exp2(torch.frexp(want).exponent.double() - 9)  # half a step of bf16
        off = (out[0][..., at].double() - want).abs() - half
        assert (off <= 3 * 2.0 ** -24 * (a.abs() + b.abs())).all(), (off / (a.abs() + b.abs())).max().item() * 2 ** 24
