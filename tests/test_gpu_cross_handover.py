"""Cross attention where a CTA goes from one item to the next: the place that the partials of a pair of query tiles
pass through is also that of the maxima and sums which the two streams of a single query tile exchange."""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import serving_mog_decode_gb300 as mog
from serving_mog_decode_gb300 import buildlib
from test_gpu_cross import DEV, Made, ints, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    buildlib.build()


def up(a, b):
    return -(-a // b)


def shares(lens, counts, H, G, T, n_max):
    """The CTAs' shares of a call whose work goes out as equal shares of all key tiles: per CTA a list of (sequence, pair,
    first unit, units, units of the item).  None if the call takes whole items."""
    tokens, sms = 128 // G, torch.cuda.get_device_properties(0).multi_processor_count
    tiles, nt, heads = up(T, tokens), up(n_max, 128), len(lens) * H
    most = heads * (tiles // 2 * nt + tiles % 2 * up(nt, 2))
    if up(heads * up(tiles, 2), sms) * (nt if tiles > 1 else up(nt, 2)) <= most // sms + 8:
        return None
    ctas = min(sms, up(most, 4))
    items = []
    for b, (n, c) in enumerate(zip(lens, counts)):
        t, k = up(c, tokens), up(n, 128)
        items += ([(b, True, max(k, 1))] * (t // 2) + [(b, False, max(up(k, 2), 1))] * (t % 2)) * H
    total = sum(u for _, _, u in items)
    limit = total // ctas + total // ctas // 3 + 12
    if max(u for _, _, u in items) <= limit:
        return None  # (may take whole items)
    chunk, out, at = max(up(total, ctas), 4), [[] for _ in range(ctas)], 0
    for b, pair, u in items:
        for p in range(at, at + u):
            c = out[p // chunk]
            if c and c[-1][0] == (b, at):
                c[-1][3] += 1
            else:
                c.append([(b, at), pair, p - at, 1, u])
        at += u
    return out


CALLS = [  # lens, counts, H, G, T, n_max
    ((3968, 100), (64, 8), 1, 4, 64, 4000),
    ((20000, 100), (200, 100), 1, 1, 200, 20000),
    ((9100, 128, 0, 64, 3000, 1), (256, 120, 7, 3, 200, 100), 3, 1, 300, 9100),
    ((30100, 5, 12000, 128), (64, 1, 60, 31), 3, 4, 64, 30100),
]


@pytest.mark.parametrize("page", [0, 64])
@pytest.mark.parametrize("lens,counts,H,G,T,n_max", CALLS)
def test_partial_of_a_pair_then_a_single_tile_of_few_rows(lens, counts, H, G, T, n_max, page):
    if not page:  # (the calls are what they are meant to be)
        assert any(a[1] and a[3] < a[4] and not b[1] and 0 < lens[b[0][0]] <= 128
                   for c in shares(lens, counts, H, G, T, n_max) for a, b in zip(c, c[1:]))
    m = Made(len(lens) + page, lens, H, page, slack=n_max - max(lens))
    q, cnt = randn(9, len(lens), T, H * G, 128), ints(*counts)
    first = torch.full(q.shape, 2.0, dtype=torch.bfloat16, device=DEV)
    mog.cross_attend(*m.cache, m.lengths, n_max, q, count=cnt, out=first)
    m.check(q, first, G, counts, fill=2.0)
    for _ in range(300):
        out = torch.full_like(first, 2.0)
        mog.cross_attend(*m.cache, m.lengths, n_max, q, count=cnt, out=out)
        assert torch.equal(out, first)
