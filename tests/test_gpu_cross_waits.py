"""Cross attention whose bounded waits run out: rows are NaN then, never what the output or the scratch held before.
The waits are made to run out by their limit alone; everything that they wait for happens."""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import serving_mog_decode_gb300 as mog
from serving_mog_decode_gb300 import buildlib
from test_gpu_cross import DEV, D, Made, ints, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    buildlib.build()


CALLS = [  # lens, counts, H, G, T, page
    ((500, 300, 0, 129), (300, 257, 40, 1), 64, 2, 300, 0),       # whole items, several of each CTA, sorted
    ((130,) * 70, (20,) * 70, 8, 4, 20, 64),                      # whole items, too many sequences to sort
    ((5000, 700, 0, 64), (600, 33, 5, 200), 2, 4, 600, 16),       # equal shares and their partials
    ((5000,) * 8, (256,) * 8, 32, 1, 256, 0),                     # sequences alike: whole rounds first
    ((20000, 100), (64, 8), 1, 4, 64, 0),                         # one pair of many CTAs, then a single tile
]


@pytest.mark.parametrize("lens,counts,H,G,T,page,polls", [c + (0,) for c in CALLS] + [CALLS[0] + (1,), CALLS[2] + (1,)])
def test_rows_are_right_or_nan(lens, counts, H, G, T, page, polls):
    m = Made(len(lens) + T, lens, H, page)
    q, cnt = randn(9, len(lens), T, H * G, D), ints(*counts)
    want = mog.cross_attend(*m.cache, m.lengths, m.n_max, q, count=cnt, out=torch.full(q.shape, 2.0, dtype=q.dtype, device=DEV))
    m.check(q, want, G, counts, fill=2.0)
    got = mog.check_cross_wait(*m.cache, m.lengths, m.n_max, q, polls, count=cnt, out=torch.full_like(want, 2.0))
    live = torch.arange(T, device=DEV)[None, :] < cnt[:, None]
    assert (got[~live] == 2).all()
    nan = torch.isnan(got).all(-1)
    assert torch.equal(got[~nan], want[~nan])
    if polls == 0:  # nothing was waited for, and nothing came
        assert nan[live].all()
    # the limit of a call is its own
    again = mog.cross_attend(*m.cache, m.lengths, m.n_max, q, count=cnt, out=torch.full_like(want, 2.0))
    assert torch.equal(again, want)


def test_long_items_outlast_few_polls():
    """Items of half a million keys, one memory for all heads, several of each CTA."""
    n, H, T = 1 << 19, 16, 6400
    K, V = randn(1, 1, 1, n, D).expand(1, H, -1, -1), randn(2, 1, 1, n, D).expand(1, H, -1, -1)
    q = randn(3, 1, T, H, D)
    want = mog.cross_attend(K, V, ints(n), n, q)
    assert torch.isfinite(want).all()
    for polls in (0, 200):
        got = mog.check_cross_wait(K, V, ints(n), n, q, polls, out=torch.full_like(want, 2.0))
        nan = torch.isnan(got).all(-1)
        assert torch.equal(got[~nan], want[~nan]) and (polls or nan.all())


def test_refusals():
    m = Made(5, (100,), 2)
    for q, polls in ((randn(6, 1, 1, 2, D), 5), (randn(6, 1, 4, 2, D), -1)):
        with pytest.raises(mog.MogError, match="INVALID_ARG"):
            mog.check_cross_wait(*m.cache, m.lengths, 100, q, polls)
