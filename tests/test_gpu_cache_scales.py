"""e4m3 decode where value rows are of very different size: rows of zeros (which kv_store gives the
scale 1) among small ones, large rows without weight, rows that lose their weight later.

The bounds are those of test_gpu_cache, per output element and relative to sum p |v|.  To
them the kernel adds 2^-39 of its unit per row, and the unit is at most 2^15 times the largest weight
p * v_scale among a warp's rows that are not zero: 2^-24 of that weight for each of the few hundred
rows of a warp, whose codes are of comparable size here: 2^-16 of sum p |v|, inside the bounds' 2^-15.
"""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import serving_mog_decode_gb300 as mog
from serving_mog_decode_gb300 import buildlib
from test_gpu_cache import (D, DEV, OUTS, STEP, Made, check, check_dense8, check_diff, gen, one_map, queries, randn,
                            weight_error, weights)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    buildlib.build()
    mog.lib()


class Stored:
    """Rows k, v (float [H, n, D]) of one sequence, written by kv_store, in 64 bits as stored."""

    def __init__(self, k, v, slack):
        self.H, n = k.shape[:2]
        self.lens, self.B, self.n_max = (n,), 1, n + slack
        codes = [torch.zeros((1, self.H, n + slack, D), device=DEV).to(torch.float8_e4m3fn) for _ in range(2)]
        scales = [torch.full((1, self.H, n + slack), float("nan"), device=DEV) for _ in range(2)]
        self.cache = mog.KV8(*codes, *scales), None
        self.lengths = torch.tensor([n], dtype=torch.int32, device=DEV)
        new = [x.transpose(0, 1)[None].bfloat16().contiguous() for x in (k, v)]
        mog.kv_store(*self.cache, torch.zeros_like(self.lengths), None, *new)
        self.rows64 = [c[:, :, :n].double() * s[:, :, :n].double()[..., None] for c, s in zip(codes, scales)]


def check_all(m, q, G, out_type):
    """dense_decode and (up to 8 heads) diff_decode over the cache."""
    out = torch.empty(q.shape, dtype=out_type, device=DEV)
    check_dense8(m, q, mog.dense_decode(*m.cache, m.lengths, m.n_max, q, out=out), G)
    if G <= 8:
        lam, gamma = weights(7)
        mog.diff_decode(*m.cache, m.lengths, m.n_max, q, lam, 0.5, gamma, eps=1e-30, out=out)
        check_diff(m, q, out, G, lam, 0.5, gamma, 1e-30)


FORMS = pytest.mark.parametrize("G,slack", [(1, 0), (4, 0), (4, 3000), (5, 3000), (8, 0), (9, 0), (16, 3000)])


@pytest.mark.parametrize("out_type", OUTS)
@pytest.mark.parametrize("size", [1.0, 1e-3, 1e-6, 1e-8, 1e-12])
@FORMS
def test_rows_of_zeros_among_small_rows(G, slack, size, out_type):
    """Whole tiles of zeros, and single rows of zeros in every other tile."""
    g = gen(1)
    H, n = 2, 700
    k, v = 0.3 * randn(g, H, n, D), size * randn(g, H, n, D)
    v[:, :40] = 0
    v[:, ::16] = 0
    v[:, 320:480] = 0
    check_all(Stored(k, v, slack), 0.3 * queries(2, 1, H * G), G, out_type)


@pytest.mark.parametrize("out_type", OUTS)
@pytest.mark.parametrize("at", [(70,), (0, 1, 2), tuple(range(64, 128)), (699,)])
@FORMS
def test_large_rows_that_some_heads_do_not_see(G, slack, at, out_type):
    """Rows 2^40 times the others: every other head gives them e^-100 of the rest's weight, the
    others all of it."""
    g = gen(3)
    H, n = 2, 700
    k, v = 0.3 * randn(g, H, n, D), 1e-3 * randn(g, H, n, D)
    q = 0.3 * queries(4, 1, H * G)
    for d in (0, 64):
        k[..., d], q[..., d] = 0, 0
        k[:, list(at), d] = -100.0
        q[:, ::2, d] = 8.0
        q[:, 1::2, d] = -8.0
    v[:, list(at)] *= 2.0 ** 40
    check_all(Stored(k, v, slack), q, G, out_type)


@pytest.mark.parametrize("out_type", OUTS)
@pytest.mark.parametrize("first,later,gap", [(2.0 ** 30, 1e-3, 40.0), (2.0 ** 100, 1e-20, 180.0), (0.0, 1e-30, 0.0)])
@FORMS
def test_large_rows_that_lose_their_weight(G, slack, first, later, gap, out_type):
    """Rows `first` in size, then rows `later` in size whose logits are `gap` above theirs."""
    g = gen(5)
    H, n, lead = 2, 900, 200
    k, v = 0.3 * randn(g, H, n, D), randn(g, H, n, D)
    q = 0.3 * queries(6, 1, H * G)
    for d in (0, 64):
        k[..., d], q[..., d] = 0, 11.0
        k[:, lead:, d] = gap
    v[:, :lead] *= first
    v[:, lead:] *= later
    m = Stored(k, v, slack)
    if later > 1e-18:
        return check_all(m, q, G, out_type)
    # (below the floor of check_dense8's comparison: the same values times 2^60 are the same output times 2^60)
    out = torch.empty(q.shape, dtype=out_type, device=DEV)
    mog.dense_decode(*m.cache, m.lengths, m.n_max, q, out=out)
    m.rows64[1] = m.rows64[1] * 2.0 ** 60
    check_dense8(m, q, (out.float() * 2.0 ** 60).to(out_type), G)


@pytest.mark.parametrize("out_type", OUTS)
@pytest.mark.parametrize("G", [4, 9])
@pytest.mark.parametrize("sink", [False, True])
def test_a_long_flat_tail_beside_one_row(G, sink, out_type):
    """300,000 rows of e^-12 of the largest row's weight each, which together outweigh it; that row's
    values zero, or like the others'."""
    g = gen(8)
    n = 300000
    k, v = torch.zeros((1, n, D), device=DEV), 1e-6 * (1 + 0.2 * randn(g, 1, n, D))
    q = 0.1 * queries(9, 1, G)
    for d in (0, 64):
        q[..., d] = 8.0
        k[:, 5, d] = 12.0 * D ** 0.5 / 16
    v[:, ::1000] = 0
    if sink:
        v[:, 5] = 0
    check_all(Stored(k, v, 0), q, G, out_type)


@pytest.mark.parametrize("out_type", OUTS)
@pytest.mark.parametrize("steps", [1, 40])
@pytest.mark.parametrize("size", [1.0, 100.0])
@FORMS
def test_rows_of_zeros_with_the_largest_logits(G, slack, size, steps, out_type):
    """Values whose scales are near the 1 that a row of zeros has, and rows of zeros that take nearly all the
    weight: one first row, or a row in every tile, each a little above the one before."""
    g = gen(17)
    H, n = 2, 40 * 32
    k, v = 0.3 * randn(g, H, n, D), size * randn(g, H, n, D)
    q = 0.3 * queries(18, 1, H * G)
    at = torch.arange(steps, device=DEV) * 32
    for d in (0, 64):
        k[..., d], q[..., d] = 0, 11.0
        k[:, at, d] = 30.0 * (1 + torch.arange(steps, device=DEV)) / steps
    v[:, at] = 0
    check_all(Stored(k, v, slack), q, G, out_type)


@pytest.mark.parametrize("G", [4, 9])
def test_a_row_of_zeros_whose_scale_is_infinite_shows(G):
    """scale * code is NaN there, as in the definition."""
    g = gen(10)
    k, v = 0.3 * randn(g, 2, 200, D), 1e-6 * randn(g, 2, 200, D)
    v[:, ::16] = 0
    m = Stored(k, v, 0)
    q = queries(11, 1, 2 * G)
    m.cache[0].v_scale[0, 0, 48] = float("inf")
    out = mog.dense_decode(*m.cache, m.lengths, m.n_max, q)
    assert torch.isnan(out[0, :G]).all() and torch.isfinite(out[0, G:]).all()


@pytest.mark.parametrize("slack", [0, 3000])
@pytest.mark.parametrize("G", [1, 4, 8])
@pytest.mark.parametrize("n", [1, 5])
def test_bf16_outputs_up_to_eight_heads_are_rounded_once(n, G, slack):
    """Equal keys, so that every weight is 1/n and each output is the mean of n values: within half a bf16
    step of it and the fp32 form's error (weights 2^-22, sums 2^-16).  Weights in one fp16 part, all off by the
    same 2^-11 or less, would carry a few outputs over the next border."""
    g = gen(12)
    H = 8
    k, v = torch.ones((1, H, n, D), device=DEV), randn(g, 1, H, n, D).abs() + 0.1
    scale = v.amax(-1) / 448.0 * (1 + 0.3 * torch.rand((1, H, n), generator=g, device=DEV))
    codes = [x.to(torch.float8_e4m3fn) for x in (k, v / scale[..., None])]
    caps = [torch.zeros((1, H, n + slack, D), device=DEV).to(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.ones((1, H, n + slack), device=DEV) for _ in range(2)]
    for c, x in zip(caps, codes):
        c[:, :, :n].view(torch.uint8).copy_(x.view(torch.uint8))
    scales[1][:, :, :n] = scale
    lengths = torch.tensor([n], dtype=torch.int32, device=DEV)
    q = queries(13, 1, H * G)
    out = torch.empty(q.shape, dtype=torch.bfloat16, device=DEV)
    mog.dense_decode(mog.KV8(*caps, *scales), None, lengths, n + slack, q, out=out)
    ref = (codes[1].double() * scale.double()[..., None]).mean(2)[0].repeat_interleave(G, 0)
    half = 2.0 ** (torch.floor(torch.log2(ref)) - 8)
    assert ((out[0].double() - ref).abs() <= half + (2.0 ** -16 + 2.0 ** -22) * ref).all()


@pytest.mark.parametrize("out_type", OUTS)
@pytest.mark.parametrize("half", [0, 1])
@pytest.mark.parametrize("G,slack", [(2, 0), (2, 3000), (5, 0), (5, 3000), (8, 3000)])
def test_diff_rows_infinite_in_one_half(G, slack, half, out_type):
    """bf16 rows with -inf in one half: without weight in that map, with their usual one in the other.  Each
    map's reference and bound go over the rows that it sees."""
    H, n, w = 1, 300, D // 2
    m = Made(14, (n,), H, 0, e4m3=False, slack=slack)
    q = queries(15, 1, H * G).abs() + 0.5
    rows = [7, 64, 299]
    m.cache[0][0, 0, rows, half * w:(half + 1) * w] = float("-inf")
    lam, gamma = weights(16)
    out = torch.empty(q.shape, dtype=out_type, device=DEV)
    mog.diff_decode(*m.cache, m.lengths, m.n_max, q, lam, 0.5, gamma, out=out)
    seen = torch.ones(n, dtype=torch.bool, device=DEV)
    seen[rows] = False
    maps = []
    for j in range(2):
        K, V = m.cache[0][0, 0, :n].double(), m.cache[1][0, 0, :n].double()
        if j == half:
            K, V = K[seen], V[seen]
        at = slice(j * w, (j + 1) * w)
        maps.append(one_map(q[0, :, at].double(), K[:, at], V, len(V), w ** -0.5))
    bf = out_type == torch.bfloat16
    L = lam.double()
    weight = torch.exp((L[0] * L[1]).sum()) - torch.exp((L[2] * L[3]).sum()) + 0.5
    (a1, e1, s1), (a2, e2, s2) = maps
    a = a1 - weight * a2
    r = torch.sqrt((a * a).mean(-1, keepdim=True) + 1e-5)
    gm = 0.5 * gamma.double()
    ref = a / r * gm
    # as in check_diff
    dw = 200 * STEP * (weight.abs() + 2 * torch.exp((L[:2].abs().prod(0)).sum()))
    E = e1 + weight.abs() * e2 + (2 * weight_error(False, bf) + 4 * STEP) * (s1 + weight.abs() * s2) + dw * s2
    bound = 1.05 * (E / r * gm.abs() + ref.abs() * torch.sqrt((E * E).mean(-1, keepdim=True)) / r) + 16 * STEP * ref.abs()
    check(out[0], ref, bound + (2.0 ** -8 * ref.abs() if bf else 0), half)
