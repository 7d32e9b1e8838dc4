"""The e4m3 cache (kv_store, dense_decode over KV8 / PagedKV8) and differential decode
against plain 64-bit forms.

Tolerances, per output element.  A weight's relative error d moves out = sum w v / sum w by
at most 2 d S, S = sum p |v|.  d adds up, in units of 2^-23 (an fp32 step, the accumulation
on the tensor cores included):
  logits   8 products of 16 terms, each off by two steps of the partial sums, at most
           A = max_i sum_j |q_j k_ij| tau: 16 A, and 4 A for the scale factors;
  exp2     its argument's rounding, 4 A; the function 2;
  sums     at most one step per added tile and merged partial: n/16 + 64;
  weights  fp16 in two parts 2^-22 or, for a bf16 output, one part 2^-12; bf16 in three
           parts 2^-24 or, for a bf16 output, two parts 2^-16 (both parts rounded to 8 bits).
A bf16 output adds half a step, 2^-8 |out|.
Differential: the two maps' bounds add (the second times |lambda|) to E; normalising by
r = sqrt(mean a^2 + eps) passes E/r on and changes r by at most rms(E): |out| rms(E)/r more.
"""
import math

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import serving_mog_decode_gb300 as mog
from serving_mog_decode_gb300 import buildlib

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
D = 128
STEP = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _built():
    buildlib.build()
    mog.lib()


# ------------------------------------------------------------------------------- inputs

def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


class Made:
    """A cache of `lens` sequences (contiguous: page 0) with its rows in 64 bits.  Rows that
    no sequence owns hold NaN, so that a read of one shows."""

    def __init__(self, seed, lens, H, page=0, e4m3=True, heads_first=True, spread=0, slack=0):
        g = gen(seed)
        B, n_max = len(lens), max(max(lens), 1)
        self.lens, self.n_max, self.B, self.H = lens, n_max + slack, B, H
        self.lengths = torch.tensor(lens, dtype=torch.int32, device=DEV)
        cap = n_max + slack if page == 0 else -(-(n_max + slack) // page) * page
        k, v = 1.5 * randn(g, B, H, cap, D), randn(g, B, H, cap, D)
        if spread:  # rows of very different size
            v = v * torch.exp2(torch.randint(-spread, spread + 1, (B, H, cap, 1), generator=g, device=DEV).float())
        dead = torch.arange(cap, device=DEV)[None, None, :, None] >= self.lengths.view(-1, 1, 1, 1)
        rows = [k, v]
        self.scales = None
        if e4m3:
            self.scales, codes = [], []
            for x in rows:
                sc = x.abs().amax(-1) / 448.0
                codes.append((x / sc[..., None]).masked_fill(dead, float("nan")).to(torch.float8_e4m3fn))
                self.scales.append(sc.masked_fill(dead[..., 0], float("nan")))
            self.rows64 = [c.double() * s.double()[..., None] for c, s in zip(codes, self.scales)]
            rows = codes
        else:
            rows = [x.masked_fill(dead, float("nan")).bfloat16() for x in rows]
            self.rows64 = [x.double() for x in rows]
        self.table = None
        if page == 0:
            self.cache = (mog.KV8(*rows, *self.scales), None) if e4m3 else tuple(rows)
            return
        per = cap // page
        n_pages = B * per + 3
        perm = torch.randperm(n_pages, generator=g, device=DEV)[: B * per].view(B, per)
        self.table = perm.int()
        for b, n in enumerate(lens):  # behind the end: pages that do not exist
            self.table[b, -(-n // page):] = -1 if b % 2 else 1 << 30
        self.pools = []
        for x in rows + (self.scales or []):
            p = torch.full((n_pages, H, page) + x.shape[3:], float("nan"), device=DEV).to(x.dtype)
            raw = p.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else p
            src = x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
            raw[perm] = src.unflatten(2, (per, page)).transpose(1, 2)
            if not heads_first:
                p = (p.view(torch.uint8).transpose(1, 2).contiguous().view(x.dtype) if raw is not p
                     else p.transpose(1, 2).contiguous())
            self.pools.append(p)
        if e4m3:
            self.cache = mog.PagedKV8(*self.pools, self.table, page, heads_first), None
        else:
            self.cache = mog.PagedKV(*self.pools, self.table, page, heads_first), None


def one_map(q, K, V, n, tau):
    """(softmax(tau q K^T) V, bound of its error without the weights' rounding, S) in 64 bits."""
    out = torch.zeros((q.shape[0], V.shape[1]), dtype=torch.float64, device=DEV)
    if n == 0:
        return out, out, out
    K, V = K[:n], V[:n]
    p = torch.softmax(q @ K.T * tau, -1)
    a = (q.abs() @ K.abs().T).amax(-1, keepdim=True) * tau
    s = p @ V.abs()
    return p @ V, 2 * STEP * (24 * a + 2 + n / 16 + 64) * s, s


def weight_error(e4m3, bf16_out):
    return (2.0 ** -12 if bf16_out else 2.0 ** -22) if e4m3 else (2.0 ** -16 if bf16_out else 2.0 ** -24)


def check(out, ref, bound, where):
    out = out.double()
    assert torch.isfinite(out).all(), where
    if out.dtype is not None:
        worst = ((out - ref).abs() / (bound + 1e-30)).max().item()
    assert worst <= 1, (where, worst)


def check_dense8(m, q, out, G):
    bf = out.dtype == torch.bfloat16
    for b, n in enumerate(m.lens):
        for h in range(m.H):
            hs = slice(h * G, (h + 1) * G)
            ref, e, s = one_map(q[b, hs].double(), m.rows64[0][b, h], m.rows64[1][b, h], n, D ** -0.5)
            bound = e + 2 * weight_error(True, bf) * s + (2.0 ** -8 * ref.abs() if bf else 0)
            check(out[b, hs], ref, bound, (b, h))


def check_diff(m, q, out, G, lam, li, gamma, eps, e4m3=True, lens=None):
    bf = out.dtype == torch.bfloat16
    w = D // 2
    for b, n in enumerate(lens or m.lens):
        for h in range(m.H):
            hs = slice(h * G, (h + 1) * G)
            K, V, qq = m.rows64[0][b, h], m.rows64[1][b, h], q[b, hs].double()
            L = (lam if lam.dim() == 3 else lam[None].expand(m.H * G, -1, -1))[hs].double()
            weight = (torch.exp((L[:, 0] * L[:, 1]).sum(-1)) - torch.exp((L[:, 2] * L[:, 3]).sum(-1)) + li)[:, None]
            a1, e1, s1 = one_map(qq[:, :w], K[:, :w], V, n, w ** -0.5)
            a2, e2, s2 = one_map(qq[:, w:], K[:, w:], V, n, w ** -0.5)
            a = a1 - weight * a2
            r = torch.sqrt((a * a).mean(-1, keepdim=True) + eps)
            gm = (1 - li) * (gamma.double() if gamma is not None else 1.0)
            ref = a / r * gm
            # lambda: two dot products of 64 terms and their exponentials in fp32
            dw = 200 * STEP * (weight.abs() + 2 * torch.exp((L[:, :2].abs().prod(1)).sum(-1))[:, None])
            E = e1 + weight.abs() * e2 + 2 * weight_error(e4m3, bf) * (s1 + weight.abs() * s2) + dw * s2 + 4 * STEP * (s1 + weight.abs() * s2)
            rE = torch.sqrt((E * E).mean(-1, keepdim=True))
            gmax = gm.abs() if torch.is_tensor(gm) else abs(gm)
            bound = 1.05 * (E / r * gmax + ref.abs() * (rE / r)) + 16 * STEP * ref.abs()
            check(out[b, hs], ref, bound + (2.0 ** -8 * ref.abs() if bf else 0), (b, h))


def queries(seed, B, HG):
    return randn(gen(seed), B, HG, D).bfloat16()


OUTS = [torch.float32, torch.bfloat16]
LAYOUTS = [(0, True), (16, True), (64, False), (128, True), (256, True)]


# ---------------------------------------------------------------------------- dense8

@pytest.mark.parametrize("slack", [0, 3000])  # one launch, clusters; two launches, the tile list split
@pytest.mark.parametrize("out_type", OUTS)
@pytest.mark.parametrize("page,hf", LAYOUTS)
@pytest.mark.parametrize("lens,H,G", [((1,), 1, 1), ((0, 1, 63, 64, 65), 2, 4), ((1000,), 3, 5), ((3001, 17), 2, 8),
                                      ((130, 0, 777), 1, 16), ((500,), 2, 9)])
def test_dense8(lens, H, G, page, hf, out_type, slack):
    m = Made(1, lens, H, page, heads_first=hf, slack=slack)
    assert (mog.dense8_scratch_bytes(m.B, H, H * G, m.n_max) == 0) == (m.n_max <= 2048)
    q = queries(2, m.B, H * G)
    out = torch.full(q.shape, float("nan"), dtype=out_type, device=DEV)
    mog.dense_decode(*m.cache, m.lengths, m.n_max, q, out=out)
    check_dense8(m, q, out, G)


@pytest.mark.parametrize("slack", [5, 3000])
def test_dense8_many_sequences_and_long_ones(slack):
    g = torch.Generator().manual_seed(3)
    lens = tuple(int(x) for x in torch.randint(0, 300, (70,), generator=g))
    m = Made(4, lens, 2, 16, slack=slack)
    q = queries(5, m.B, 4)
    check_dense8(m, q, mog.dense_decode(*m.cache, m.lengths, m.n_max, q), 2)
    m = Made(6, (70001, 33), 1, 64)
    q = queries(7, 2, 4)
    check_dense8(m, q, mog.dense_decode(*m.cache, m.lengths, m.n_max, q), 4)


@pytest.mark.parametrize("slack", [0, 3000])
def test_dense8_scales_far_apart_and_zero(slack):
    m = Made(8, (777, 300), 2, 16, spread=40, slack=slack)
    q = queries(9, 2, 4)
    check_dense8(m, q, mog.dense_decode(*m.cache, m.lengths, m.n_max, q), 2)
    # all value scales zero: zeros, not NaN
    m.pools[3].zero_()
    out = mog.dense_decode(*m.cache, m.lengths, m.n_max, q)
    assert (out == 0).all()


def test_dense8_query_sizes():
    """Queries from 2^-60 to 2^40 times the usual: the power of two that fp16 takes out."""
    m = Made(10, (333,), 1, 0)
    q = queries(11, 1, 4).float()
    q *= torch.tensor([2.0 ** -60, 2.0 ** -9, 1.0, 2.0 ** 4], device=DEV).view(1, 4, 1)
    q = q.bfloat16()
    check_dense8(m, q, mog.dense_decode(*m.cache, m.lengths, m.n_max, q), 4)
    q = (queries(11, 1, 4).float() * 2.0 ** 40).bfloat16()  # one key takes all
    out = mog.dense_decode(*m.cache, m.lengths, m.n_max, q)
    best = (q[0].double() @ m.rows64[0][0, 0, :333].T).argmax(-1)
    want = m.rows64[1][0, 0][best]
    assert torch.allclose(out[0].double(), want, rtol=1e-6, atol=0)


def test_dense8_a_nan_row_shows_and_stays_in_its_head():
    m = Made(12, (200,), 2, 0)
    m.cache[0].k_scale[0, 0, 100] = float("nan")
    q = queries(13, 1, 4)
    out = mog.dense_decode(*m.cache, m.lengths, m.n_max, q)
    assert torch.isnan(out[0, :2]).all()
    m.rows64[0] = m.rows64[0].clone()
    assert torch.isfinite(out[0, 2:]).all()


def test_dense8_pages_that_do_not_exist_are_left_out():
    m = Made(14, (100,), 1, 16)
    q = queries(15, 1, 2)
    keep = torch.ones(100, dtype=torch.bool, device=DEV)
    for slot, bad in ((1, -1), (4, 10 ** 6), (5, -(1 << 31))):
        m.table[0, slot] = bad
        keep[16 * slot:16 * slot + 16] = False
    out = mog.dense_decode(*m.cache, m.lengths, m.n_max, q)
    m.rows64 = [x[:, :, :100][:, :, keep] for x in m.rows64]
    m.lens = (int(keep.sum()),)
    check_dense8(m, q, out, 2)


def test_dense8_lengths_are_clamped():
    m = Made(16, (96,), 1, 0)
    q = queries(17, 1, 1)
    want = mog.dense_decode(*m.cache, m.lengths, 96, q)
    assert torch.equal(mog.dense_decode(*m.cache, m.lengths + 50, 96, q), want)
    assert (mog.dense_decode(*m.cache, m.lengths - 1000, 96, q) == 0).all()


def test_dense8_is_deterministic_and_follows_lengths_in_a_graph():
    m = Made(18, (4000, 1200), 2, 64)
    q = queries(19, 2, 8)
    scratch = torch.empty(mog.dense8_scratch_bytes(2, 2, 8, m.n_max), dtype=torch.uint8, device=DEV)
    assert scratch.numel() > 0
    out = torch.empty(q.shape, dtype=torch.float32, device=DEV)
    call = lambda o: mog.dense_decode(*m.cache, m.lengths, m.n_max, q, out=o, scratch=scratch)  # noqa: E731
    first = call(torch.empty_like(out)).clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out)
    for lens in ((4000, 1200), (1, 0), (3999, 64)):
        m.lengths.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        m.lens = lens
        check_dense8(m, q, out, 4)
        if lens == (4000, 1200):
            assert torch.equal(out, first)


def test_dense8_on_another_stream():
    m = Made(20, (2000,), 2, 16)
    q = queries(21, 1, 4)
    want = mog.dense_decode(*m.cache, m.lengths, m.n_max, q)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = mog.dense_decode(*m.cache, m.lengths, m.n_max, q, stream=s)
    with torch.cuda.stream(s):
        again = mog.dense_decode(*m.cache, m.lengths, m.n_max, q)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(again, want)


def test_store_past_32_bit_strides():
    """Sequences and new rows further apart than 2^31 elements."""
    apart = (1 << 31) + 4096
    big = torch.zeros(2 * apart, dtype=torch.uint8, device=DEV)
    pools = [big[at:].view(torch.float8_e4m3fn).as_strided((2, 1, 4, D), (apart, 512, D, 1)) for at in (0, 1024)]
    scales = [torch.ones((2, 1, 4), device=DEV) for _ in range(2)]
    new = torch.zeros(apart + 4096, dtype=torch.bfloat16, device=DEV)
    x = [new[at:].as_strided((2, 2, 1, D), (apart, D, D, 1)) for at in (0, 512)]
    for i, t in enumerate(x):
        t.copy_(randn(gen(94 + i), 2, 2, 1, D))
    mog.kv_store(mog.KV8(*pools, *scales), None, torch.tensor([1, 2], dtype=torch.int32, device=DEV), None, *x)
    for pool, sc, t in zip(pools, scales, x):
        for b, p0 in ((0, 1), (1, 2)):
            row = t[b, :, 0].double()
            want = row_scale(row)
            assert torch.equal(sc[b, 0, p0:p0 + 2].double(), want)
            assert torch.equal(pool[b, 0, p0:p0 + 2].double(), e4m3_nearest(row / want[:, None]))
            assert (pool[b, 0, :p0].double() == 0).all() and (pool[b, 0, p0 + 2:].double() == 0).all()


def test_dense8_past_32_bit_offsets():
    """One head's rows spread over more than 4 GiB by their stride."""
    n, stride = 40000, 128 * 1024
    big = torch.zeros(n * stride, dtype=torch.uint8, device=DEV)
    K = big.view(torch.float8_e4m3fn).as_strided((1, 1, n, D), (n * stride, n * stride, stride, 1))
    V = big[1024:].view(torch.float8_e4m3fn).as_strided((1, 1, n, D), (n * stride, n * stride, stride, 1))
    m = Made(22, (n,), 1, 0)
    c = m.cache[0]
    K.view(torch.uint8).copy_(c.K.view(torch.uint8))
    V.view(torch.uint8).copy_(c.V.view(torch.uint8))
    q = queries(23, 1, 2)
    out = mog.dense_decode(mog.KV8(K, V, c.k_scale, c.v_scale), None, m.lengths, n, q)
    check_dense8(m, q, out, 2)


# ------------------------------------------------------------------------------ diff

def weights(seed, heads=None):
    g = gen(seed)
    lam = 0.2 * randn(g, *((heads,) if heads else ()), 4, D // 2)
    return lam, 1 + 0.2 * randn(g, D)


@pytest.mark.parametrize("slack", [0, 3000])
@pytest.mark.parametrize("out_type", OUTS)
@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("page,hf", LAYOUTS)
@pytest.mark.parametrize("lens,H,G", [((1,), 1, 1), ((0, 1, 63, 64, 65), 2, 4), ((1000,), 3, 3), ((2001, 17), 2, 8),
                                      ((300, 0, 77), 1, 5)])
def test_diff(lens, H, G, page, hf, e4m3, out_type, slack):
    m = Made(31, lens, H, page, e4m3=e4m3, heads_first=hf, slack=slack)
    q = queries(32, m.B, H * G)
    lam, gamma = weights(33)
    out = torch.full(q.shape, float("nan"), dtype=out_type, device=DEV)
    mog.diff_decode(*m.cache, m.lengths, m.n_max, q, lam, 0.5, gamma=gamma, eps=1e-5, out=out)
    check_diff(m, q, out, G, lam, 0.5, gamma, 1e-5, e4m3)


@pytest.mark.parametrize("e4m3", [True, False])
def test_diff_weights_per_head_and_no_gamma(e4m3):
    m = Made(34, (900, 40), 2, 32, e4m3=e4m3)
    q = queries(35, 2, 6)
    lam, _ = weights(36, 6)
    out = mog.diff_decode(*m.cache, m.lengths, m.n_max, q, lam, 0.2, eps=1e-6)
    check_diff(m, q, out, 3, lam, 0.2, None, 1e-6, e4m3)


@pytest.mark.parametrize("slack", [0, 3000])
@pytest.mark.parametrize("e4m3", [True, False])
def test_diff_many_sequences_and_long_ones(e4m3, slack):
    g = torch.Generator().manual_seed(37)
    lens = tuple(int(x) for x in torch.randint(0, 200, (40,), generator=g))
    lam, gamma = weights(38)
    m = Made(39, lens, 2, 16, e4m3=e4m3, slack=slack)
    q = queries(40, m.B, 4)
    check_diff(m, q, mog.diff_decode(*m.cache, m.lengths, m.n_max, q, lam, 0.5, gamma), 2, lam, 0.5, gamma, 1e-5, e4m3)
    m = Made(41, (50001,), 1, 64, e4m3=e4m3)
    q = queries(42, 1, 5)
    check_diff(m, q, mog.diff_decode(*m.cache, m.lengths, m.n_max, q, lam, 0.5, gamma), 5, lam, 0.5, gamma, 1e-5, e4m3)


def test_diff_equal_maps_cancel_to_lambda():
    """Equal halves: a = (1 - lambda) softmax(.) V, whatever the sizes."""
    m = Made(43, (500,), 1, 0, e4m3=False)
    m.cache[0][..., 64:] = m.cache[0][..., :64]
    m.rows64[0] = m.cache[0].double()
    q = queries(44, 1, 2)
    q[..., 64:] = q[..., :64]
    lam, gamma = weights(45)
    out = mog.diff_decode(*m.cache, m.lengths, 500, q, lam, 0.8, gamma)
    check_diff(m, q, out, 2, lam, 0.8, gamma, 1e-5, False)


def test_diff_infinite_keys_of_one_map_do_not_touch_the_other():
    """-inf in a row's second half gives that row no weight in the second map and its usual
    weight in the first."""
    m = Made(46, (300,), 1, 0, e4m3=False)
    q = queries(47, 1, 2).abs() + 0.5
    K = m.cache[0]
    K[0, 0, 7, 64:] = float("-inf")
    m.rows64[0] = K.double()
    lam, gamma = weights(48)
    out = mog.diff_decode(*m.cache, m.lengths, 300, q, lam, 0.5, gamma)
    # (the bound's largest |q||k| leaves the infinite row out)
    m.rows64[0] = m.rows64[0].clone()
    m.rows64[0][0, 0, 7, 64:] = -1e3
    check_diff(m, q, out, 2, lam, 0.5, gamma, 1e-5, False)


def test_diff_bf16_pages_that_do_not_exist_are_left_out():
    m = Made(49, (100,), 1, 16, e4m3=False)
    q = queries(50, 1, 2)
    lam, gamma = weights(51)
    keep = torch.ones(100, dtype=torch.bool, device=DEV)
    for slot, bad in ((0, -1), (3, 10 ** 6)):
        m.table[0, slot] = bad
        keep[16 * slot:16 * slot + 16] = False
    out = mog.diff_decode(*m.cache, m.lengths, m.n_max, q, lam, 0.5, gamma)
    m.rows64 = [x[:, :, :100][:, :, keep] for x in m.rows64]
    check_diff(m, q, out, 2, lam, 0.5, gamma, 1e-5, False, lens=(int(keep.sum()),))


@pytest.mark.parametrize("slack", [0, 3000])
@pytest.mark.parametrize("e4m3", [True, False])
def test_diff_in_a_graph(e4m3, slack):
    m = Made(52, (2000, 100), 2, 16, e4m3=e4m3, slack=slack)
    q = queries(53, 2, 4)
    lam, gamma = weights(54)
    mog.diff_decode(*m.cache, m.lengths, m.n_max, q, lam, 0.5, gamma)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = mog.diff_decode(*m.cache, m.lengths, m.n_max, q, lam, 0.5, gamma)
    for lens in ((2000, 100), (5, 0), (1999, 65)):
        m.lengths.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        check_diff(m, q, out, 2, lam, 0.5, gamma, 1e-5, e4m3, lens=lens)


# ----------------------------------------------------------------------------- store

def pow2(e):
    """2^e in 64 bits, from its bits (torch.ldexp goes through a 32-bit power)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def e4m3_nearest(y):
    """float64 y to the nearest e4m3 value (ties to even, saturating), in 64 bits."""
    m, e = torch.frexp(y)
    step = pow2((e - 1).clamp_min(-6) - 3)
    return (torch.round(y / step) * step).clamp(-448, 448)


def row_scale(x):
    """The least power of two with amax <= 448 * scale, by comparison with every candidate."""
    amax = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)
    cand = pow2(torch.arange(-126, 121, device=DEV))
    at = (448 * cand < amax[..., None]).sum(-1).clamp_max(246)
    return torch.where(amax > 0, cand[at], 1.0)


def store_rows(seed, B, T, H):
    g = gen(seed)
    x = randn(g, B, T, 2 * H, D) * torch.exp2(torch.randint(-30, 30, (B, T, 2 * H, 1), generator=g, device=DEV).float())
    x = x.bfloat16()
    if T >= 6:
        x[0, 0] = 0
        x[0, 1, :, 5] = float("inf")
        x[0, 2, :, 6] = float("-inf")
        x[0, 3, :, 7] = float("nan")
        x[0, 4] = 0
        x[0, 4, :, 3] = 448 * 2.0 ** -9  # exactly at the border of a scale
        x[0, 5] = 1e-39                  # a subnormal row
    return x


@pytest.mark.parametrize("page,hf", [(0, True), (16, True), (64, False)])
@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("B,T,H", [(1, 1, 1), (3, 37, 2), (2, 300, 8), (5, 1, 32)])
def test_store(B, T, H, e4m3, page, hf):
    g = gen(61)
    x = store_rows(62, B, T, H)
    k_new, v_new = x[:, :, :H], x[:, :, H:]
    pos = torch.randint(0, 50, (B,), generator=g, device=DEV).int()
    count = torch.randint(0, T + 1, (B,), generator=g, device=DEV).int()
    count[0] = T
    cap = 50 + T
    dt = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    if page:
        per = -(-cap // page)
        n_pages = B * per + 2
        shape = (n_pages, H, page) if hf else (n_pages, page, H)
        table = torch.randperm(n_pages, generator=g, device=DEV)[: B * per].view(B, per).int().contiguous()
    else:
        shape, table = (B, H, cap), None
    pools = [(0.5 * randn(g, *shape, D)).to(dt) for _ in range(2)]
    scales = [torch.full(shape, 3.0, device=DEV) for _ in range(2)] if e4m3 else []
    want = [p.double() for p in pools] + [s.double() for s in scales]
    if page:
        cls = mog.PagedKV8 if e4m3 else mog.PagedKV
        cache = (cls(*pools, *scales, table, page, hf), None)
    else:
        cache = (mog.KV8(*pools, *scales), None) if e4m3 else tuple(pools)
    mog.kv_store(*cache, pos, count, k_new, v_new)
    for i, new in enumerate((k_new, v_new)):
        sc = row_scale(new.double()) if e4m3 else None
        val = e4m3_nearest(new.double() / sc[..., None]) if e4m3 else new.double()
        for b in range(B):
            n, p0 = int(count[b]), int(pos[b])
            at = torch.arange(p0, p0 + n, device=DEV)
            if page:
                pg, row = table[b].long()[at // page], at % page
                idx = (pg, slice(None), row) if hf else (pg, row)
            else:
                idx = (b, slice(None), at)
            rows = val[b, :n] if page else val[b, :n].transpose(0, 1)
            want[i][idx] = rows
            if e4m3:
                want[2 + i][idx] = sc[b, :n] if page else sc[b, :n].transpose(0, 1)
    for got, ref in zip(pools + scales, want):
        assert torch.equal(torch.nan_to_num(got.double(), nan=1e9), torch.nan_to_num(ref, nan=1e9))


def test_store_leaves_out_what_is_outside():
    """Positions before, behind and in no page; a count above T; no counts at all."""
    H, page = 2, 16
    pool = [torch.zeros((4, H, page, D), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    table = torch.tensor([[0, -1], [4, 1], [2, 3]], dtype=torch.int32, device=DEV)
    x = torch.ones((3, 20, H, D), dtype=torch.bfloat16, device=DEV)
    cache = mog.PagedKV(*pool, table, page)
    pos = torch.tensor([-4, 8, 20], dtype=torch.int32, device=DEV)
    mog.kv_store(cache, None, pos, torch.tensor([20, 99, -3], dtype=torch.int32, device=DEV), x, x)
    want = torch.zeros((4, page))
    want[0, :16] = 1   # positions -4..-1 left out, 0..15 written
    want[1, :12] = 1   # positions 8..15 in no page, 16..27 written
    assert torch.equal(pool[0][:, 0, :, 0].float().cpu(), want)
    mog.kv_store(cache, None, pos, None, x, x)
    want[3, 4:] = 1    # 20..31 written, 32..39 behind the table
    assert torch.equal(pool[1][:, 1, :, 5].float().cpu(), want)


def test_store_takes_strided_rows_and_refuses_others():
    g = gen(63)
    x = randn(g, 2, 3, 4, 3 * D).bfloat16()
    K = torch.zeros((2, 4, 8, D), dtype=torch.bfloat16, device=DEV)
    V = torch.zeros_like(K)
    pos = torch.zeros(2, dtype=torch.int32, device=DEV)
    mog.kv_store(K, V, pos, None, x[..., :D], x[..., D:2 * D])
    assert torch.equal(K[:, :, :3], x[..., :D].transpose(1, 2)) and torch.equal(V[:, :, :3], x[..., D:2 * D].transpose(1, 2))
    with pytest.raises(mog.MogError, match="INVALID_ARG"):
        mog.kv_store(K, V, pos, None, x[..., 4:4 + D], x[..., D + 4:2 * D + 4])  # not on 16 bytes
    for bad in (x[..., :64], x[:1, :, :, :D], x[..., :D].float()):
        with pytest.raises(ValueError):
            mog.kv_store(K, V, pos, None, bad, bad)
    with pytest.raises(ValueError):
        mog.kv_store(K, V, pos.long(), None, x[..., :D], x[..., D:2 * D])
    mog.kv_store(K, V, pos, None, x[:, :0, :, :D], x[:, :0, :, :D])  # nothing to store


def test_python_refusals():
    m = Made(64, (64,), 2, 16)
    c = m.cache[0]
    q = queries(65, 1, 4)
    lam, gamma = weights(66)
    ok = dict(lengths_dev=m.lengths, n_max=64, q=q)
    bad = [dict(q=q.float()), dict(q=q[:, :, :64].contiguous()), dict(q=q.transpose(1, 2)), dict(n_max=65), dict(n_max=0),
           dict(lengths_dev=m.lengths.long()), dict(lengths_dev=torch.zeros(2, dtype=torch.int32, device=DEV)),
           dict(out=torch.empty((1, 4, D), dtype=torch.float16, device=DEV)), dict(lengths_dev=m.lengths.cpu()),
           dict(out=torch.empty((1, 3, D), device=DEV))]
    for kw in bad:
        with pytest.raises(ValueError):
            mog.dense_decode(c, None, **{**ok, **kw})
        with pytest.raises(ValueError):
            mog.diff_decode(c, None, **{**ok, **kw}, lam=lam, lambda_init=0.5)
    long = Made(64, (64,), 2, 16, slack=4000)
    with pytest.raises(mog.MogError, match="ARENA"):
        mog.dense_decode(long.cache[0], None, long.lengths, long.n_max, q,
                         scratch=torch.empty(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(mog.MogError, match="SHAPE"):
        mog.diff_decode(c, None, m.lengths, 64, queries(67, 1, 18), lam, 0.5)
    for w in (lam.double(), lam[:3], lam[:, :32].contiguous(), lam[None].expand(3, -1, -1).contiguous()):
        with pytest.raises(ValueError):
            mog.diff_decode(c, None, **ok, lam=w, lambda_init=0.5)
    with pytest.raises(ValueError):
        mog.diff_decode(c, None, **ok, lam=lam, lambda_init=0.5, gamma=gamma[:64])
    with pytest.raises(ValueError):
        mog.dense_decode_noalloc(c, None, m.lengths, 64, q, torch.empty((1, 4, D), device=DEV))
    with pytest.raises(ValueError):  # an e4m3 cache has no MoG index
        mog.build(c, None, [64], mog.make_params(1, 2, 4, 64))


# ---------------------------------------------------------- bounds, streams, large batches

@pytest.mark.parametrize("lens,H,G,page", [((5000,), 1, 4, 16), ((3000, 10, 0, 4000), 3, 16, 64), ((2500,) * 3, 2, 9, 0)])
def test_nothing_is_written_behind_scratch_and_output(lens, H, G, page):
    m = Made(71, lens, H, page)
    q = queries(72, m.B, H * G)
    for diff in ([False, True] if G <= 8 else [False]):
        need = (mog.diff_scratch_bytes if diff else mog.dense8_scratch_bytes)(m.B, H, H * G, m.n_max)
        assert need > 0
        buf = torch.full((need + 8192,), 0xA5, dtype=torch.uint8, device=DEV)
        big = torch.full((m.B + 2, H * G, D), 7.5, device=DEV)
        out, scratch = big[1:-1], buf[4096:4096 + need]
        if diff:
            lam, gamma = weights(73)
            mog.diff_decode(*m.cache, m.lengths, m.n_max, q, lam, 0.5, gamma, out=out, scratch=scratch)
            check_diff(m, q, out, G, lam, 0.5, gamma, 1e-5)
        else:
            mog.dense_decode(*m.cache, m.lengths, m.n_max, q, out=out, scratch=scratch)
            check_dense8(m, q, out, G)
        assert (buf[:4096] == 0xA5).all() and (buf[4096 + need:] == 0xA5).all()
        assert (big[0] == 7.5).all() and (big[-1] == 7.5).all()


@pytest.mark.parametrize("n", [40, 1000])
def test_large_batches_of_short_sequences(n):
    """More units than CTAs: a warp per head folds one or two partials."""
    g = torch.Generator().manual_seed(74)
    lens = tuple(int(x) for x in torch.randint(0, n + 1, (300,), generator=g))
    m = Made(75, lens, 2, 16)
    q = queries(76, m.B, 4)
    lam, gamma = weights(77)
    assert mog.dense8_scratch_bytes(m.B, 2, 4, m.n_max) > 0
    check_dense8(m, q, mog.dense_decode(*m.cache, m.lengths, m.n_max, q), 2)
    check_diff(m, q, mog.diff_decode(*m.cache, m.lengths, m.n_max, q, lam, 0.5, gamma), 2, lam, 0.5, gamma, 1e-5)


def test_two_streams_at_once():
    """Calls that overlap, each with scratch of its own."""
    ms = [Made(78 + i, (20000 + 999 * i,), 2, 16 * i) for i in range(2)]
    qs = [queries(80 + i, 1, 8) for i in range(2)]
    want = [mog.dense_decode(*m.cache, m.lengths, m.n_max, q) for m, q in zip(ms, qs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            got[i].append(mog.dense_decode(*ms[i].cache, ms[i].lengths, ms[i].n_max, qs[i], stream=s))
    for s in streams:
        s.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])


def test_graphs_of_two_calls_with_their_own_scratch():
    """Scratch that a captured call takes by itself belongs to the graph."""
    m = Made(82, (9000, 400), 2, 64)
    q = queries(83, 2, 8)
    lam, gamma = weights(84)
    want = (mog.dense_decode(*m.cache, m.lengths, m.n_max, q), mog.diff_decode(*m.cache, m.lengths, m.n_max, q, lam, 0.5, gamma))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = (mog.dense_decode(*m.cache, m.lengths, m.n_max, q), mog.diff_decode(*m.cache, m.lengths, m.n_max, q, lam, 0.5, gamma))
    for _ in range(3):
        noise = [torch.full((1 << 20,), float("nan"), device=DEV) for _ in range(8)]  # takes freed memory outside
        del noise
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_paged_cache_whose_attributes_are_set_anew():
    """A PagedKV is read as it is at each call, in place of what an earlier call saw."""
    a, b = Made(85, (300,), 2, 16, e4m3=False), Made(86, (300,), 2, 16, e4m3=False)
    q = queries(87, 1, 4)
    lam, gamma = weights(88)
    pk = a.cache[0]
    mog.diff_decode(pk, None, a.lengths, 300, q, lam, 0.5, gamma)
    pk.K, pk.V, pk.block_table = b.cache[0].K, b.cache[0].V, b.table
    check_diff(b, q, mog.diff_decode(pk, None, b.lengths, 300, q, lam, 0.5, gamma), 2, lam, 0.5, gamma, 1e-5, False)
    pk.K.data = a.pools[0]  # (the same tensor object over other memory)
    pk.V.data, pk.block_table.data = a.pools[1], a.table
    check_diff(a, q, mog.diff_decode(pk, None, a.lengths, 300, q, lam, 0.5, gamma), 2, lam, 0.5, gamma, 1e-5, False)


def test_pages_past_32_bit_offsets():
    """Pools whose pages lie 128 KB apart over more than 4 GiB: stored, forked, moved and read."""
    n_pages, R, apart = 40000, 16, 1 << 17
    big = torch.zeros(n_pages * apart, dtype=torch.uint8, device=DEV)

    def pool(at):
        return big[at:].view(torch.float8_e4m3fn).as_strided((n_pages, 1, R, D), (apart, R * D, D, 1))

    K, V = pool(0), pool(apart // 2)
    scales = [torch.ones((n_pages, 1, R), device=DEV) for _ in range(2)]
    refs = torch.ones(n_pages, dtype=torch.int32, device=DEV)  # all but the last pages are taken
    refs[-40:] = 0
    p = mog.PagePool(K, V, 2, 8, k_scale=scales[0], v_scale=scales[1], refs=refs)
    n = torch.tensor([100, 0], dtype=torch.int32, device=DEV)
    pos, granted = p.grow(n)
    assert granted.tolist() == [100, 0] and int(p.block_table[0, 0]) == n_pages - 40
    x = randn(gen(89), 2, 100, 2, D).bfloat16()
    mog.kv_store(p.cache(), None, pos, granted, x[:, :, :1], x[:, :, 1:])
    p.assign(torch.tensor([0, 0], dtype=torch.int32, device=DEV))
    p.grow(torch.tensor([0, 1], dtype=torch.int32, device=DEV))  # a copied last page
    p.lengths.fill_(100)                                          # (its new row is not written)
    rows = [e4m3_nearest(x[0, :, i].double() / row_scale(x[0, :, i].double())[:, None])
            * row_scale(x[0, :, i].double())[:, None] for i in range(2)]
    q = queries(90, 2, 4)
    ref, e, s = one_map(q[0].double(), *rows, 100, D ** -0.5)
    out = mog.dense_decode(p.cache(), None, p.lengths, 128, q)
    check(out[0], ref, e + 2 * weight_error(True, False) * s, "first")
    ref, e, s = one_map(q[1].double(), *rows, 100, D ** -0.5)
    check(out[1], ref, e + 2 * weight_error(True, False) * s, "copied")
    p.refs[:100] = 0  # pages at the front come free: the sequences' pages move there
    p.compact()
    assert int(p.block_table.max()) < n_pages - 40 and p.status() == 0
    assert torch.equal(mog.dense_decode(p.cache(), None, p.lengths, 128, q), out)


def test_diff_a_map_of_infinitely_small_logits_is_zero():
    """-inf in the second half of every row: the first map alone is left."""
    m = Made(91, (100,), 1, 0, e4m3=False)
    q = queries(92, 1, 2).abs() + 0.5
    m.cache[0][..., 64:] = float("-inf")
    lam, gamma = weights(93)
    out = mog.diff_decode(*m.cache, m.lengths, 100, q, lam, 0.5, gamma)
    K, V = m.rows64[0][0, 0], m.rows64[1][0, 0]
    a, e, s = one_map(q[0, :, :64].double(), K[:, :64], V, 100, 64 ** -0.5)
    r = torch.sqrt((a * a).mean(-1, keepdim=True) + 1e-5)
    E = e + 2 * weight_error(False, False) * s
    ref = 0.5 * gamma.double() * a / r
    rE = torch.sqrt((E * E).mean(-1, keepdim=True))
    check(out[0], ref, 1.05 * (0.5 * gamma.double().abs() * E / r + ref.abs() * rE / r) + 16 * STEP * ref.abs(), "map")
