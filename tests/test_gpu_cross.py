"""Cross attention against a plain implementation in 64 bits: query counts, lengths and heads around the
tiles, pages, strides, masked rows that hold NaN, and its refusals."""
import math

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import serving_mog_decode_gb300 as mog
from serving_mog_decode_gb300 import buildlib

pytestmark = pytest.mark.gpu
DEV, D = "cuda", 128
BF = 2.0 ** -8  # half a step of bf16, relative


@pytest.fixture(scope="module", autouse=True)
def built():
    buildlib.build()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def randn(seed, *shape):
    return torch.randn(shape, generator=gen(seed), device=DEV).bfloat16()


class Made:
    """A bf16 cache of `lens` sequences whose rows behind the end hold NaN and infinities; pages that no
    sequence owns too."""

    def __init__(self, seed, lens, H, page=0, heads_first=True, slack=0):
        self.lens, self.H, self.n_max = lens, H, max(max(lens), 1) + slack
        B, cap = len(lens), self.n_max if page == 0 else -(-self.n_max // page) * page
        self.lengths = ints(*lens)
        self.rows = [randn(seed, B, H, cap, D), randn(seed + 1, B, H, cap, D)]
        dead = torch.arange(cap, device=DEV)[None, None, :, None] >= self.lengths.view(-1, 1, 1, 1)
        t = [x.masked_fill(dead, v) for x, v in zip(self.rows, (float("nan"), float("inf")))]
        t[1][..., ::3] = t[1][..., ::3].masked_fill(dead.expand_as(t[1])[..., ::3], float("nan"))
        if page == 0:
            self.cache = tuple(t)
            return
        per = cap // page
        perm = torch.randperm(B * per + 2, generator=gen(seed + 2), device=DEV)[: B * per].view(B, per)
        self.table = perm.int()
        for b, n in enumerate(lens):
            self.table[b, -(-n // page):] = -1 if b % 2 else 1 << 30
        pools = []
        for x in t:
            p = torch.full((B * per + 2, H, page, D), float("nan"), device=DEV, dtype=torch.bfloat16)
            p[perm] = x.unflatten(2, (per, page)).transpose(1, 2)
            pools.append(p if heads_first else p.transpose(1, 2).contiguous())
        self.cache = mog.PagedKV(*pools, self.table, page, heads_first), None

    def check(self, q, out, G, count=None, keep=None, fill=None):
        """Largest error against its bound, and the 2-norm of the errors: the weights' rounding and the output's,
        each uniform in half a step (2^-8 / sqrt 3 of a value at most)."""
        off = size2 = 0.0
        for b, n in enumerate(self.lens):
            t = q.shape[1] if count is None else min(max(count[b], 0), q.shape[1])
            if fill is not None:
                assert (out[b, t:] == fill).all()
            for h in range(self.H):
                got = out[b, :t, h * G:(h + 1) * G].double().reshape(-1, D)
                K, V = (x[b, h, :n].double() for x in self.rows)
                if keep is not None:
                    K, V = K[keep[b][:n]], V[keep[b][:n]]
                if K.shape[0] == 0:
                    assert (got == 0).all()
                    continue
                x = q[b, :t, h * G:(h + 1) * G].double().reshape(-1, D)
                p = torch.softmax(x @ K.T / math.sqrt(D), -1)
                want, size = p @ V, p @ V.abs()
                assert torch.isfinite(got).all()
                # weights to half a step of bf16; logits (below 2^6) to 2^-20, so weights to 2^-14; the output's rounding
                assert ((got - want).abs() <= (BF + 2.0 ** -14) * (1 + BF) * size + BF * want.abs()).all(), (b, h)
                off += float(((got - want) ** 2).sum())
                size2 += float((want ** 2).sum() + ((p * p) @ (V * V)).sum())
        if size2:
            assert math.sqrt(off / size2) <= BF / math.sqrt(3) * 1.05 + 2.0 ** -14  # (5%: few samples)


CASES = [  # lens, T, H, G, page
    ((1,), 1, 1, 1, 0), ((128,), 1, 1, 1, 0), ((129, 0, 77), 2, 2, 1, 0), ((256,), 128, 1, 1, 0), ((257, 1000), 129, 1, 1, 0),
    ((300, 5, 640), 30, 2, 4, 0), ((1500, 700), 50, 2, 5, 0), ((1000,), 17, 1, 16, 0), ((127, 128, 129), 100, 1, 3, 16),
    ((500, 33), 40, 2, 8, 32), ((1111, 2000), 1, 2, 4, 64), ((777,), 200, 2, 2, 128), ((900, 300), 70, 1, 7, 256),
    ((20000,), 3, 2, 5, 64), ((20000, 9000), 1, 4, 4, 0), ((6000,), 300, 1, 1, 16),
    ((20000, 19000, 20000, 17000), 16, 16, 5, 64), ((15000, 16384), 80, 20, 4, 0),  # long streams, one query tile and two
    ((5000,) * 8, 256, 32, 1, 0), ((5000, 4999, 5120, 5000, 4993, 5001, 5000, 5000), 300, 24, 1, 64),  # sequences alike: whole rounds first
]


@pytest.mark.parametrize("lens,T,H,G,page", CASES)
def test_cross(lens, T, H, G, page):
    m = Made(T + page, lens, H, page)
    q = randn(9, len(lens), T, H * G, D)
    m.check(q, mog.cross_attend(*m.cache, m.lengths, m.n_max, q), G)


@pytest.mark.parametrize("page", [0, 16, 64])
def test_counts_strides_and_slack(page):
    m = Made(20, (260, 0, 400, 31), 2, page, heads_first=False, slack=500)
    G, T = 3, 150
    qkv = randn(21, 4, T, 2 * G + 4, D)
    q = qkv[:, :, 2:2 + 2 * G]
    count = (150, 20, 1, -4)
    out = torch.full((4, 2 * G, T, D), 5.0, dtype=torch.bfloat16, device=DEV).transpose(1, 2)
    got = mog.cross_attend(*m.cache, m.lengths, m.n_max, q, count=ints(*count), out=out)
    assert got is out
    m.check(q, out, G, count, fill=5.0)
    # lengths are clamped
    again = mog.cross_attend(*m.cache, m.lengths - torch.tensor([0, 1000, 0, 0], dtype=torch.int32, device=DEV), m.n_max, q)
    m.check(q, again, G)  # (not its bits: how the work is shared depends on all lengths and counts)
    big = Made(22, (300,), 1)
    a = mog.cross_attend(*big.cache, ints(1 << 30), 300, q[:1, :, :2])
    assert torch.equal(a, mog.cross_attend(*big.cache, ints(300), 300, q[:1, :, :2]))


@pytest.mark.parametrize("page", [0, 32])
@pytest.mark.parametrize("T,H,G,longest", [(1, 8, 2, 700), (40, 4, 4, 700), (100, 3, 3, 500), (300, 4, 1, 130), (7, 2, 1, 6000)])
def test_many_sequences(T, H, G, longest, page):
    """Lists of many short items, one query tile and two, with sequences that have no rows and no tokens."""
    g = torch.Generator().manual_seed(T)
    B = 45
    lens = torch.randint(0, longest, (B,), generator=g)
    lens[torch.tensor([0, 7, 8, B - 1])] = torch.tensor([0, 0, 128, 0])
    count = torch.randint(-2, T + 3, (B,), generator=g)
    count[torch.tensor([3, 4, B - 2])] = 0
    m = Made(T, tuple(lens.tolist()), H, page)
    q = randn(9, B, T, H * G, D)
    out = torch.full(q.shape, 2.0, dtype=torch.bfloat16, device=DEV)
    cnt = count.to(torch.int32).to(DEV)
    mog.cross_attend(*m.cache, m.lengths, m.n_max, q, count=cnt, out=out)
    m.check(q, out, G, count.tolist(), fill=2.0)
    again = mog.cross_attend(*m.cache, m.lengths, m.n_max, q, count=cnt, out=torch.full_like(out, 2.0))
    assert torch.equal(again, out)
    cnt.zero_()
    assert (mog.cross_attend(*m.cache, m.lengths, m.n_max, q, count=cnt, out=torch.full_like(out, 2.0)) == 2).all()


def test_pages_that_do_not_exist_are_left_out():
    for T in (3, 200):
        m = Made(30, (500, 300), 1, 16)
        keep = [torch.ones(n, dtype=torch.bool, device=DEV) for n in m.lens]
        for b, slot, bad in ((0, 1, -1), (0, 30, 10 ** 6), (0, 31, -(1 << 31)), (1, 0, -1), (1, 18, 99999)):
            m.table[b, slot] = bad
            keep[b][16 * slot:16 * slot + 16] = False
        q = randn(31, 2, T, 2, D)
        m.check(q, mog.cross_attend(*m.cache, m.lengths, m.n_max, q), 2, keep=keep)
        m.table.fill_(-1)
        assert (mog.cross_attend(*m.cache, m.lengths, m.n_max, q) == 0).all()
    # whole tiles of such pages
    m = Made(32, (1000,), 1, 128)
    m.table[0, 2:7] = -1
    keep = [torch.ones(1000, dtype=torch.bool, device=DEV)]
    keep[0][256:896] = False
    q = randn(33, 1, 140, 1, D)
    m.check(q, mog.cross_attend(*m.cache, m.lengths, 1000, q), 1, keep=keep)


def test_rising_and_large_logits():
    """Maxima that rise from tile to tile, by little and by much, fall, and reach 2^40."""
    n, T = 1024, 130
    for step in (0.5, 4.0, 300.0, -4.0):
        m = Made(40, (n,), 1)
        q = randn(41, 1, T, 1, D)
        q[..., 0] = 16.0
        tile = torch.arange(n, device=DEV) // 64
        m.rows[0][0, 0, :, 0] = (step * tile * math.sqrt(D) / 16).bfloat16()
        m.rows[0][0, 0, :, 1:] *= 0.25
        m.cache = tuple(m.rows)
        out = mog.cross_attend(*m.cache, m.lengths, n, q)
        K, V = (x[0, 0].double() for x in m.rows)
        logits = q[0, :, 0].double() @ K.T / math.sqrt(D)
        p = torch.softmax(logits, -1)
        rel = 2.0 ** -21 * (q[0, :, 0].double().abs() @ K.abs().T / math.sqrt(D)).amax(-1, keepdim=True)  # of the logits
        assert ((out[0, :, 0].double() - p @ V).abs() <= (2 * BF + 4 * rel) * (p @ V.abs()) + 1e-30).all(), step
    m = Made(42, (n,), 1)
    q = (randn(43, 1, T, 1, D).float() * 2.0 ** 40).bfloat16()
    out = mog.cross_attend(*m.cache, m.lengths, n, q)
    best = (q[0, :, 0].double() @ m.rows[0][0, 0].double().T).argmax(-1)
    assert torch.equal(out[0, :, 0], m.rows[1][0, 0][best])


def test_infinite_and_nan_rows():
    m = Made(50, (300, 300), 2)
    m.rows[0][0, 0, 200] = float("nan")  # a key that everybody sees
    m.rows[1][1, 0, 7] = float("inf")
    m.cache = tuple(m.rows)
    q = randn(51, 2, 4, 2, D)
    out = mog.cross_attend(*m.cache, m.lengths, 300, q)
    assert torch.isnan(out[0, :, 0]).all() and torch.isfinite(out[0, :, 1]).all()
    assert (out[1, :, 0] == float("inf")).all() and torch.isfinite(out[1, :, 1]).all()
    # logits that are all -infinity: zeros
    m = Made(52, (40,), 1)
    m.rows[0][:] = 0
    m.rows[0][..., 0] = -float("inf")
    m.cache = tuple(m.rows)
    q = torch.zeros((1, 3, 1, D), dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 1
    assert (mog.cross_attend(*m.cache, m.lengths, 40, q) == 0).all()
    # a query row of NaN stays with itself
    m = Made(53, (333,), 1)
    q = randn(54, 1, 200, 1, D)
    want = mog.cross_attend(*m.cache, m.lengths, 333, q)
    q[0, 100, 0, 3] = float("nan")
    out = mog.cross_attend(*m.cache, m.lengths, 333, q)
    assert torch.isnan(out[0, 100]).all()
    rest = torch.arange(200, device=DEV) != 100
    assert torch.equal(out[0, rest], want[0, rest])


def test_one_memory_for_every_sequence():
    """States expanded over the batch (stride 0), and over the heads."""
    K, V = randn(60, 1, 2, 500, D), randn(61, 1, 2, 500, D)
    q, L = randn(62, 3, 9, 4, D), ints(500, 123, 0)
    a = mog.cross_attend(K.expand(3, -1, -1, -1), V.expand(3, -1, -1, -1), L, 500, q)
    b = mog.cross_attend(K.repeat(3, 1, 1, 1), V.repeat(3, 1, 1, 1), L, 500, q)
    assert torch.equal(a, b)
    a = mog.cross_attend(K[:, :1].expand(3, 2, -1, -1), V[:, :1].expand(3, 2, -1, -1), L, 500, q)
    b = mog.cross_attend(K[:, :1].repeat(3, 2, 1, 1), V[:, :1].repeat(3, 2, 1, 1), L, 500, q)
    assert torch.equal(a, b)


def test_one_token_is_the_decode_step():
    m = Made(63, (3000, 129), 4, 64)
    q = randn(64, 2, 1, 16, D)
    out = mog.cross_attend(*m.cache, m.lengths, m.n_max, q)
    want = mog.dense_decode(*m.cache, m.lengths, m.n_max, q[:, 0].contiguous())
    assert ((out[:, 0].double() - want.double()).norm() / want.double().norm()) < 2 * BF / math.sqrt(3)


@pytest.mark.parametrize("G", [1, 5, 16])
@pytest.mark.parametrize("page", [0, 32])
def test_one_token_with_strides_and_counts(G, page):
    lens, H = (700, 0, 5000, 33, 64), 3
    m = Made(100 + G, lens, H, page)
    qkv = randn(101, 5, 1, (G + 2) * H, D)
    q = qkv[:, :, H:(G + 1) * H]
    out = torch.full((5, 1, 2 * G * H, D), 4.0, dtype=torch.bfloat16, device=DEV)
    part = out[:, :, G * H:]
    count = (1, 1, 0, 7, -2)
    mog.cross_attend(*m.cache, m.lengths, m.n_max, q, count=ints(*count), out=part)
    m.check(q, part, G, count, fill=4.0)
    assert (out[:, :, : G * H] == 4).all()
    long = Made(102, (60000,), 2, page)  # the split form
    q = randn(103, 1, 1, 2 * G, D)
    got = mog.cross_attend(*long.cache, long.lengths, long.n_max, q)
    long.check(q, got, G)
    keep = torch.full_like(got, 9.0)
    mog.cross_attend(*long.cache, long.lengths, long.n_max, q, count=ints(0), out=keep)
    assert (keep == 9).all()


def test_read_back_from_8_bits_then_attended():
    """An int8 cache's rows read back are what several query tokens attend to."""
    g = gen(65)
    codes = [torch.randint(-127, 128, (2, 2, 192, D), generator=g, device=DEV, dtype=torch.int8) for _ in range(2)]
    s = [torch.rand((2, 2, 6), generator=g, device=DEV) / 64 for _ in range(2)]
    c = mog.KVI8(*codes, *s, 32)
    K, V = (torch.zeros((2, 2, 192, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    mog.kv_load(c, None, ints(0, 0), None, K.transpose(1, 2), V.transpose(1, 2))
    m = Made(66, (192, 100), 2)
    m.rows = [K, V]
    q = randn(67, 2, 12, 4, D)
    m.check(q, mog.cross_attend(K, V, m.lengths, 192, q), 2)


def test_deterministic_captured_and_on_another_stream():
    m = Made(70, (5000, 3000), 2, 64)
    q, count = randn(71, 2, 6, 8, D), ints(6, 6)
    scratch = torch.empty(mog.cross_scratch_bytes(2, 2, 8, 6, m.n_max), dtype=torch.uint8, device=DEV)
    assert scratch.numel() > 0
    out = torch.zeros_like(q)
    call = lambda o: mog.cross_attend(*m.cache, m.lengths, m.n_max, q, count=count, out=o, scratch=scratch)  # noqa: E731
    first = call(torch.zeros_like(q))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    other = torch.zeros_like(q)
    torch.cuda.synchronize()
    assert torch.equal(mog.cross_attend(*m.cache, m.lengths, m.n_max, q, out=other, stream=s), other)
    s.synchronize()
    assert torch.equal(other, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out)
    for lens, cnt in (((5000, 3000), (6, 6)), ((1, 0), (6, 2)), ((128, 2999), (0, 5))):
        m.lengths.copy_(torch.tensor(lens, dtype=torch.int32))
        count.copy_(torch.tensor(cnt, dtype=torch.int32))
        out.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        m.lens = lens
        m.check(q, out, 4, cnt, fill=3.0)
        if lens == (5000, 3000):
            assert torch.equal(out, first)


@pytest.mark.parametrize("page", [0, 64])
def test_how_the_work_is_shared_follows_the_lengths(page):
    """One captured call, whose largest lengths ask for equal shares: sequences that balance as whole items, that do
    not, that are alike, that are empty, and counts of their own."""
    m = Made(85, (4000, 3100, 2000, 1100), 4, page)
    q = randn(87, 4, 700, 16, D)
    count, out = ints(700, 700, 700, 700), torch.empty_like(q)
    rows = m.lens
    for _ in range(2):
        mog.cross_attend(*m.cache, m.lengths, m.n_max, q, count=count, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mog.cross_attend(*m.cache, m.lengths, m.n_max, q, count=count, out=out)
    for lens, cnt in (((4000, 3100, 2000, 1100), (700,) * 4), ((4000, 700, 600, 500), (700,) * 4), ((1100,) * 4, (700,) * 4),
                      ((0, 0, 2000, 1), (700, 0, 333, 32)), ((4000, 3100, 2000, 1100), (33, 700, 1, 640)), ((0,) * 4, (700, 1, 0, 65))):
        lens = tuple(min(n, r) for n, r in zip(lens, rows))
        m.lengths.copy_(torch.tensor(lens, dtype=torch.int32))
        count.copy_(torch.tensor(cnt, dtype=torch.int32))
        out.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        m.lens = lens
        m.check(q, out, 4, cnt, fill=3.0)


def test_past_32_bit_offsets():
    """Rows of one head spread over more than 4 GiB by their stride, and queries as far apart."""
    n, stride = 40000, 64 * 1024
    big = torch.zeros(n * stride + 4096, dtype=torch.bfloat16, device=DEV)
    K, V = (big[at:].as_strided((1, 1, n, D), (n * stride, n * stride, stride, 1)) for at in (0, 1024))
    m = Made(80, (n,), 1)
    K.copy_(m.rows[0])
    V.copy_(m.rows[1])
    q = big[2048:].as_strided((1, 2, 1, D), (0, (n - 2) * stride, D, 1))
    out = big[4096 - 1024:].as_strided((1, 2, 1, D), (0, (n - 2) * stride, D, 1))
    q.copy_(randn(81, 1, 2, 1, D))
    mog.cross_attend(K, V, m.lengths, n, q, out=out)
    m.check(q, out, 1)


def test_refusals():
    m = Made(90, (100, 50), 2)
    q = randn(91, 2, 3, 4, D)
    call = lambda q=q, L=m.lengths, n=100, **kw: mog.cross_attend(*m.cache, L, n, q, **kw)  # noqa: E731
    for bad in (q.float(), q[:1], q[0], q[..., :64], randn(1, 2, 3, 4, 2 * D)[..., ::2], q.cpu()):
        with pytest.raises(ValueError):
            call(bad)
    for kw in (dict(L=ints(1)), dict(L=m.lengths.long()), dict(n=0), dict(n=101), dict(count=ints(1)),
               dict(out=torch.empty((2, 3, 4, D), device=DEV)), dict(out=q[:, :, :1].expand(-1, -1, 4, -1)),
               dict(scratch=torch.empty(64, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(mog.MogError, match="SHAPE"):
        call(randn(1, 2, 3, 5, D))  # 5 heads over 2
    with pytest.raises(mog.MogError, match="SHAPE"):
        call(randn(1, 2, 3, 34, D))  # more than 16 per KV head
    with pytest.raises(ValueError, match="bf16"):
        k = torch.zeros((2, 2, 64, D), dtype=torch.int8, device=DEV)
        s = torch.ones((2, 2, 1), device=DEV)
        mog.cross_attend(mog.KVI8(k, k.clone(), s, s.clone(), 64), None, m.lengths, 64, q)
    assert call(q[:, :0]).shape == (2, 0, 4, D)
