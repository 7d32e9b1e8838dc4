"""Rotary positions, int8 caches with a scale per block, and rows read back: against plain
implementations, at the sizes, positions and values where they can go wrong."""
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
LEAST = 2.0 ** -126


@pytest.fixture(scope="module", autouse=True)
def built():
    buildlib.build()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def rows(seed, *shape, spread=1.0):
    g = gen(seed)
    x = torch.randn(shape, generator=g, device=DEV)
    return (x * torch.exp2(spread * torch.randn(shape[:-1] + (1,), generator=g, device=DEV))).bfloat16()


# ------------------------------------------------------------------- rotary positions, alone

def turned(x, p, freq, factor, rot, pairs, inverse=False):
    """(turned rows, bound of the error before the last rounding) in 64 bits: x [T, H, D], p [T]."""
    x = x.double()
    z = p.double()[:, None, None] * torch.as_tensor(freq, dtype=torch.float64, device=DEV) * (-1 if inverse else 1)
    c, s = torch.cos(z) * factor, torch.sin(z) * factor
    out, mag = x.clone(), torch.zeros_like(x)
    if pairs:
        ia, ib = torch.arange(0, rot, 2, device=DEV), torch.arange(1, rot, 2, device=DEV)
    else:
        ia = torch.arange(rot // 2, device=DEV)
        ib = ia + rot // 2
    a, b = x[..., ia], x[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = mag[..., ib] = (a.abs() + b.abs()) * abs(factor)
    # the angle to 2^-32 turns and 2^-24 of itself (2^-24 pi), sincospi to 2 units (2^-22), factor and products: 3 roundings
    return out, 2.0 ** -20 * mag


def check_turned(got, want, bound, where=None):
    off = (got.double() - want).abs()
    assert (off <= BF * want.abs() + (1 + BF) * bound + 1e-38).all(), (where, off.max().item())


@pytest.mark.parametrize("rot", [16, 48, 64, 128])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("T,H,B", [(1, 1, 1), (1, 40, 3), (17, 3, 2), (33, 48, 1), (300, 7, 2)])
def test_rope(rot, pairs, T, H, B):
    r = mog.Rope(rot, base=500000.0, interleaved=pairs, factor=1.25)
    freq = mog.rope_frequencies(rot, 500000.0)[0]
    x = rows(rot + T, B, T, H, D)
    pos = torch.randint(0, 1 << 20, (B,), generator=gen(T), device=DEV, dtype=torch.int32)
    out = mog.rope(x, pos, r)
    for b in range(B):
        check_turned(out[b], *turned(x[b], pos[b] + torch.arange(T, device=DEV), freq, 1.25, rot, pairs))
    assert torch.equal(out[..., rot:], x[..., rot:])
    back = mog.rope(out, pos, mog.Rope(rot, base=500000.0, interleaved=pairs, factor=0.8), inverse=True)
    for b in range(B):
        want, bound = turned(out[b], pos[b] + torch.arange(T, device=DEV), freq, 0.8, rot, pairs, inverse=True)
        check_turned(back[b], want, bound)


@pytest.mark.parametrize("rot,pairs,inverse", [(128, False, False), (96, True, True), (16, False, True)])
def test_rope_rounds_once(rot, pairs, inverse):
    """Before the rounding to bf16, an element is off by no more than 3 * 2^-24 of its pair: the angle is within an eighth
    of a turn of whole quarters and rounded there (pi 2^-27, times a slope of at most 0.71: 0.28 * 2^-24) and cut to 2^-32
    turns (0.03), sincospi to one unit (1), the factor's product (0.5), and the two roundings of x c - y s (1.0)."""
    r = mog.Rope(rot, base=500000.0, interleaved=pairs, factor=1.25)
    x = rows(3, 1, 4000, 4, D)
    for start in (0, 1 << 20):
        out = mog.rope(x, ints(start), r, inverse=inverse)
        want, bound = turned(x[0], start + torch.arange(4000, device=DEV), mog.rope_frequencies(rot, 500000.0)[0], 1.25, rot, pairs, inverse)
        half = torch.exp2(torch.frexp(want).exponent.double() - 9)  # half a step of bf16
        assert ((out[0].double() - want).abs() <= half + 3 * 2.0 ** -24 * (bound / 2.0 ** -20)).all()


@pytest.mark.parametrize("start", [(1 << 31) - 9, -(1 << 31), -5, 16777217])
def test_rope_far_positions(start):
    """Any int32: angles of 2^31 radians and more (64-bit reference: 2^-53 of 2^32 radians is 2^-21)."""
    r = mog.Rope(64, base=10000.0)
    x = rows(5, 1, 9, 2, D)
    p = start + torch.arange(9, device=DEV, dtype=torch.int64)
    out = mog.rope(x, ints(start), r)
    want, bound = turned(x[0], p, mog.rope_frequencies(64, 10000.0)[0], 1.0, 64, False)
    check_turned(out[0], want, 4 * bound)


def test_rope_positions_of_each_token_counts_and_strides():
    r = mog.Rope(96, base=10000.0, interleaved=True)
    freq = mog.rope_frequencies(96, 10000.0)[0]
    qkv = rows(6, 3, 21, 12, D)
    x = qkv[:, :, 2:7]  # a slice of a fused projection
    pos = torch.randint(-50, 5000, (3, 21), generator=gen(7), device=DEV, dtype=torch.int32)
    count = ints(21, 0, 5)
    out = torch.full((3, 5, 21, D), 7.0, dtype=torch.bfloat16, device=DEV).transpose(1, 2)  # heads first
    got = mog.rope(x, pos, r, count=count, out=out)
    assert got is out
    for b in range(3):
        n = int(count[b])
        check_turned(out[b, :n], *turned(x[b, :n], pos[b, :n], freq, 1.0, 96, True))
        assert (out[b, n:] == 7).all()
    # counts are clamped
    out2 = mog.rope(x, pos, r, count=ints(1000, -3, 21))
    assert torch.equal(out2[0], out[0])
    # in place: the rest of the projection is left alone
    keep = qkv.clone()
    mog.rope(x, pos, r, out=x)
    assert torch.equal(qkv[:, :, :2], keep[:, :, :2]) and torch.equal(qkv[:, :, 7:], keep[:, :, 7:])
    assert torch.equal(x[0], out[0])


def test_rope_gradient():
    """The inverse turn is the gradient: against differences of a weighted sum, in 64 bits of the formula."""
    r = mog.Rope(64, base=100.0, factor=1.5)
    freq = mog.rope_frequencies(64, 100.0)[0]
    x, w = rows(8, 1, 4, 2, D), rows(9, 1, 4, 2, D)
    grad = mog.rope(w, ints(11), r, inverse=True)
    p = 11 + torch.arange(4, device=DEV)
    f = lambda y: (turned(y, p, freq, 1.5, 64, False)[0] * w[0].double()).sum()  # noqa: E731
    y = x[0].double()
    for t, h, j in ((0, 0, 0), (1, 1, 33), (3, 0, 31), (2, 1, 63), (3, 1, 100)):
        d = torch.zeros_like(y)
        d[t, h, j] = 1e-3
        diff = float((f(y + d) - f(y - d)) / 2e-3)  # (linear: no error of the step's second order)
        k = j if j >= 64 else (j + 32) % 64
        mag = 1.5 * float(w[0, t, h, j].abs() + w[0, t, h, k].abs())
        assert abs(float(grad[0, t, h, j]) - diff) <= BF * abs(diff) + 2.0 ** -19 * mag + 1e-9, (t, h, j)


def test_rope_refusals():
    r, x = mog.Rope(64), rows(10, 2, 3, 4, D)
    for bad in (x.float(), x[..., :64], x[0], rows(1, 2, 3, 4, 256)[..., ::2]):
        with pytest.raises(ValueError):
            mog.rope(bad, ints(0, 0), r)
    for pos in (ints(0), ints(0, 0).long(), ints(0, 0).cpu(), torch.zeros((2, 4), dtype=torch.int32, device=DEV)):
        with pytest.raises(ValueError, match="pos"):
            mog.rope(x, pos, r)
    with pytest.raises(ValueError, match="count"):
        mog.rope(x, ints(0, 0), r, count=ints(1))
    with pytest.raises(ValueError, match="out"):
        mog.rope(x, ints(0, 0), r, out=torch.empty((2, 3, 4, D), device=DEV))
    with pytest.raises(ValueError, match="share memory"):
        mog.rope(x, ints(0, 0), r, out=x[:1].expand(2, -1, -1, -1))
    with pytest.raises(ValueError, match="Rope is on cpu"):
        mog.rope(x, ints(0, 0), mog.Rope(64, device="cpu"))
    assert mog.rope(x[:, :0], ints(0, 0), r).shape == (2, 0, 4, D)


# ------------------------------------------------------------------------ int8 block caches

class Cache8:
    """An int8 cache and the same state as a plain model: codes [B, H, cap, D], scales [B, H, blocks]."""

    def __init__(self, seed, B, H, cap, block, page=0, heads_first=True):
        self.B, self.H, self.cap, self.block, self.page = B, H, cap, block, page
        g = gen(seed)
        blocks = -(-cap // block)
        stale = lambda: torch.randint(-127, 128, (B, H, cap, D), generator=g, device=DEV, dtype=torch.int8)  # noqa: E731
        self.codes = [stale(), stale()]  # (what was there before: it must count for nothing)
        self.scales = [torch.rand((B, H, blocks), generator=g, device=DEV) * 100 for _ in range(2)]
        if page == 0:
            self.K, self.V = (x.clone() for x in self.codes)
            self.ks, self.vs = (x.clone() for x in self.scales)
            self.cache = mog.KVI8(self.K, self.V, self.ks, self.vs, block)
            return
        per = cap // page
        self.table = torch.randperm(B * per + 2, generator=g, device=DEV)[: B * per].view(B, per).int()
        pools = []
        for x, rows_ in ((self.codes[0], page), (self.codes[1], page), (self.scales[0], page // block),
                         (self.scales[1], page // block)):
            p = torch.zeros((B * per + 2, H, rows_) + x.shape[3:], device=DEV).to(x.dtype)
            p[self.table.long()] = x.unflatten(2, (per, rows_)).transpose(1, 2)
            pools.append(p if heads_first else p.transpose(1, 2).contiguous())
        self.heads_first, self.pools = heads_first, pools
        self.cache = mog.PagedKVI8(*pools, self.table, page, block, heads_first)

    def state(self):
        """(codes, scales) of K and V as the cache holds them."""
        if self.page == 0:
            return [self.K, self.V], [self.ks, self.vs]
        got = []
        for p in self.pools:
            p = p if self.heads_first else p.transpose(1, 2)
            got.append(p[self.table.long()].transpose(1, 2).flatten(2, 3))
        return got[:2], got[2:]

    def store(self, pos, count, new):
        """The plain model of kv_store: new = (k, v) [B, T, H, D]; rounding in fp32 as defined."""
        for codes, scales, x in zip(self.codes, self.scales, new):
            for b in range(self.B):
                lo, hi = max(pos[b], 0), min(pos[b] + min(count[b], x.shape[1]), self.cap)  # (counts are clamped)
                while lo < hi:
                    blk, end = lo // self.block, min((lo // self.block + 1) * self.block, hi)
                    y = x[b, lo - pos[b]:end - pos[b]].float().transpose(0, 1)  # [H, rows, D]
                    first = blk * self.block
                    old = scales[b, :, blk] if lo > first else torch.zeros(self.H, device=DEV)
                    amax = torch.where(torch.isfinite(y), y.abs(), 0.0).amax((1, 2))
                    inv127 = torch.full((), 1.0, device=DEV) / torch.full((), 127.0, device=DEV)
                    s = torch.maximum(torch.maximum(old, amax * inv127), torch.full_like(old, LEAST))
                    s = torch.where(torch.isnan(y).any(-1).any(-1) | torch.isnan(old), float("nan"), s)
                    code = torch.round(y * (1.0 / s)[:, None, None]).clamp(-127, 127)
                    grow = s > old
                    held = codes[b, :, first:lo].float()
                    held = torch.where(grow[:, None, None], torch.round(held * (old / s)[:, None, None]), held)
                    ok = ~torch.isnan(s)[:, None, None]
                    codes[b, :, first:lo] = torch.where(ok, held, codes[b, :, first:lo].float()).to(torch.int8)
                    codes[b, :, lo:end] = torch.where(ok, code, codes[b, :, lo:end].float()).to(torch.int8)
                    scales[b, :, blk] = s
                    lo = end

    def check(self):
        codes, scales = self.state()
        for got, want, gs, ws in zip(codes, self.codes, scales, self.scales):
            assert torch.equal(torch.nan_to_num(gs, nan=-1.0), torch.nan_to_num(ws, nan=-1.0))
            good = ~torch.isnan(ws).repeat_interleave(self.block, -1)[..., : self.cap, None].expand_as(want)
            assert torch.equal(got[good], want[good])


def store(c, pos, count, k, v):
    mog.kv_store(c.cache, None, ints(*pos), None if count is None else ints(*count), k, v)
    c.store(pos, [k.shape[1]] * c.B if count is None else count, (k, v))


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("page,heads_first", [(0, True), (128, True), (128, False)])
def test_store_rounds_and_grows(block, page, heads_first):
    """Prompts of ragged lengths, then steps of one and of a few tokens, of growing rows."""
    B, H, cap = 3, 3, 384 if page else 333
    c = Cache8(block, B, H, cap, block, page, heads_first)
    k, v = rows(1, B, 150, H, D), rows(2, B, 150, H, D)
    store(c, [0, 0, 7], [150, 1, 77], k, v)
    c.check()
    pos = [150, 1, 84]
    for step in range(6):
        T = (1, 1, 5, 1, 33, 1)[step]
        k, v = (rows(10 * step + i, B, T, H, D, spread=1.0 + step / 2) for i in range(2))
        store(c, pos, None, k, v)
        c.check()
        pos = [p + T for p in pos]
    # back to an earlier position: what lies behind is given up
    store(c, [40, 0, 80], [3, 2, 0], k, v)
    c.check()


def test_store_error_is_half_a_step():
    """In 64 bits: a block written at once is within half a step, and the largest magnitude has the code 127."""
    c = Cache8(3, 2, 4, 256, 64)
    k, v = rows(4, 2, 256, 4, D), rows(5, 2, 256, 4, D)
    store(c, [0, 0], None, k, v)
    for codes, s, x in zip((c.K, c.V), (c.ks, c.vs), (k, v)):
        x = x.double().transpose(1, 2).unflatten(2, (4, 64))
        s, codes = s.double()[..., None, None], codes.double().unflatten(2, (4, 64))
        assert ((x - codes * s).abs() <= s * (0.5 + 128 * 2.0 ** -22)).all()  # x * (1/s): two roundings of up to 127
        assert (codes.abs().amax((-1, -2)) == 127).all()
        assert ((s - x.abs().amax((-1, -2), keepdim=True) / 127).abs() <= 2.0 ** -22 * s).all()


def test_store_extreme_values():
    c = Cache8(6, 1, 6, 64, 32)
    k = rows(7, 1, 40, 6, D, spread=0.0)
    k[0, :, 0] = 0  # nothing: the least scale, codes 0
    k[0, 3, 1, 5], k[0, 35, 1, 9] = float("inf"), -float("inf")
    k[0, 20, 2, 0] = float("nan")
    k[0, :, 3] = (k[0, :, 3].float() * 1e-39).bfloat16()  # subnormal
    k[0, :, 4] = (k[0, :, 4].float().clamp(-3, 3) * 1.1e38).bfloat16()
    k[0, :, 5] = float("inf")  # no finite magnitude
    store(c, [0], None, k, k.flip(1))
    c.check()
    assert (c.ks[0, 0] == LEAST).all() and torch.isnan(c.ks[0, 2, 0]) and torch.isfinite(c.ks[0, 2, 1])
    assert c.K[0, 1, 3, 5] == 127 and c.K[0, 1, 35, 9] == -127 and (c.K[0, 5, :40] == 127).all()
    # a NaN block stays one while rows join it, and starts afresh
    k = rows(8, 1, 1, 6, D)
    store(c, [31], None, k, k)
    c.check()
    assert torch.isnan(c.ks[0, 2, 0])
    store(c, [0], None, k, k)
    c.check()
    assert torch.isfinite(c.ks[0, 2, 0])


@pytest.mark.parametrize("rope", [False, True])
def test_store_leaves_out_positions_outside_and_pages_that_do_not_exist(rope):
    c = Cache8(9, 3, 2, 128, 32, 32)
    before = [x.clone() for x in c.pools]
    c.table[0, 1], c.table[0, 2] = -1, 1 << 30
    k, v = rows(10, 3, 100, 2, D), rows(11, 3, 100, 2, D)
    pos, count = [10, -40, 120], [100, 90, 100]
    if rope:
        r = mog.Rope(128)
        mog.rope_store(c.cache, None, ints(*pos), ints(*count), k, k, v, r)
        k = mog.rope(k, ints(*pos), r)
    else:
        mog.kv_store(c.cache, None, ints(*pos), ints(*count), k, v)
    c.store(pos, count, (k, v))
    real = torch.ones_like(c.table, dtype=torch.bool)
    real[0, 1] = real[0, 2] = False
    touched = torch.zeros(c.pools[0].shape[0], dtype=torch.bool, device=DEV)
    for p, codes in zip(c.pools[:2], c.codes):
        want = codes.unflatten(2, (4, 32)).transpose(1, 2)
        assert torch.equal(p[c.table[real].long()], want[real])
    for p, scales in zip(c.pools[2:], c.scales):
        want = scales.unflatten(2, (4, 1)).transpose(1, 2)
        assert torch.equal(p[c.table[real].long()], want[real])
    touched[c.table[real].long()] = True
    for p, old in zip(c.pools, before):
        assert torch.equal(p[~touched], old[~touched])
    # positions at the end of int32
    mog.kv_store(c.cache, None, ints((1 << 31) - 2, -(1 << 31), 128), None, k, v)
    assert torch.equal(c.pools[0][~touched], before[0][~touched])


# ------------------------------------------------------------------------------- read back

def caches(kind, seed, B, H, cap, page=0):
    """(cache arguments, rows [B, H, cap, D] of K and V as bf16 values) of a full cache."""
    g = gen(seed)
    x = [rows(seed + i, B, H, cap, D) for i in range(2)]
    if kind == "bf16":
        t, want = x, [y.clone() for y in x]
    elif kind == "e4m3":
        s = [torch.rand((B, H, cap), generator=g, device=DEV) + 0.5 for _ in x]
        t = [(y.float() / 8).to(torch.float8_e4m3fn) for y in x]
        want = [(y.float() * z[..., None]).bfloat16() for y, z in zip(t, s)]
        t = t + s
    else:
        block = 32
        s = [torch.rand((B, H, -(-cap // block)), generator=g, device=DEV) + 0.5 for _ in x]
        t = [torch.randint(-128, 128, y.shape, generator=g, device=DEV, dtype=torch.int8) for y in x]
        want = [(y.float() * z.repeat_interleave(block, -1)[..., :cap, None]).bfloat16() for y, z in zip(t, s)]
        t = t + s
    if page == 0:
        return {"bf16": lambda: tuple(t), "e4m3": lambda: (mog.KV8(*t), None), "i8": lambda: (mog.KVI8(*t, 32), None)}[kind](), want
    per = cap // page
    table = torch.randperm(B * per, generator=g, device=DEV).view(B, per)
    pools = []
    for y in t:
        n = y.shape[2] // per
        raw = y.view(torch.uint8) if y.dtype == torch.float8_e4m3fn else y
        p = torch.empty((B * per, H, n) + raw.shape[3:], dtype=raw.dtype, device=DEV)
        p[table] = raw.unflatten(2, (per, n)).transpose(1, 2)
        pools.append(p.view(y.dtype))
    table = table.int()
    if kind == "bf16":
        return (mog.PagedKV(*pools, table, page), None), want
    return (mog.PagedKV8(*pools, table, page) if kind == "e4m3" else mog.PagedKVI8(*pools, table, page, 32), None), want


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("page", [0, 64])
def test_load(kind, page):
    B, H, cap = 3, 5, 192
    (K, V), want = caches(kind, 20, B, H, cap, page)
    pos, count = ints(0, 17, 150), ints(1, 130, 100)  # (the last sequence: rows behind its end)
    T = 131
    out = [torch.full((B, H, T, D), 3.0, dtype=torch.bfloat16, device=DEV).transpose(1, 2) for _ in range(2)]
    got = mog.kv_load(K, V, pos, count, *out)
    assert got[0] is out[0] and got[1] is out[1]
    for o, w in zip(out, want):
        for b, (p, n) in enumerate(((0, 1), (17, 130), (150, 42))):
            assert torch.equal(o[b, :n], w[b, :, p:p + n].transpose(0, 1))
            assert (o[b, n:] == 3).all()
    out = [torch.zeros((B, 7, H, D), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    mog.kv_load(K, V, ints(-3, 5, 190), None, *out)
    for o, w in zip(out, want):
        assert (o[0, :3] == 0).all() and torch.equal(o[0, 3:], w[0, :, :4].transpose(0, 1))
        assert torch.equal(o[1], w[1, :, 5:12].transpose(0, 1)) and (o[2, 2:] == 0).all()


def test_load_leaves_rows_in_no_page_and_reads_nan():
    (K, V), want = caches("i8", 21, 1, 2, 128, 32)
    K.block_table[0, 1] = -7
    K.k_scale[K.block_table[0, 2].long()] = float("nan")
    out = [torch.full((1, 128, 2, D), 9.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    mog.kv_load(K, V, ints(0), None, *out)
    assert (out[0][0, 32:64] == 9).all() and (out[1][0, 32:64] == 9).all()
    assert torch.isnan(out[0][0, 64:96]).all() and torch.equal(out[1][0, 64:], want[1][0, :, 64:].transpose(0, 1))


def test_load_refusals():
    (K, V), _ = caches("i8", 22, 2, 2, 64)
    ok = lambda: torch.empty((2, 4, 2, D), dtype=torch.bfloat16, device=DEV)  # noqa: E731
    for k, v in ((ok().float(), ok()), (ok()[:1], ok()), (ok(), ok()[:, :3]), (ok(), ok().transpose(1, 2).contiguous().transpose(1, 2)),
                 (ok()[:, :, :1].expand(-1, -1, 2, -1),) * 2):
        with pytest.raises(ValueError):
            mog.kv_load(K, V, ints(0, 0), None, k, v)
    with pytest.raises(ValueError, match="pos"):
        mog.kv_load(K, V, ints(0), None, ok(), ok())


# --------------------------------------------------------- turned and stored in one launch

@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("page", [0, 64])
@pytest.mark.parametrize("T,H,G,rot,pairs", [(1, 8, 4, 128, False), (1, 1, 1, 16, True), (5, 3, 5, 64, True),
                                             (100, 2, 1, 96, False), (70, 8, 8, 128, True)])
def test_rope_store_is_rope_then_store(kind, page, T, H, G, rot, pairs):
    B, cap = 3, 256
    made = [caches(kind, 30, B, H, cap, page)[0] for _ in range(2)]
    r = mog.Rope(rot, base=10000.0, interleaved=pairs, factor=1.1)
    qkv = rows(31, B, T, (G + 2) * H, D)
    q, k, v = qkv[:, :, : G * H], qkv[:, :, G * H:(G + 1) * H], qkv[:, :, (G + 1) * H:]
    pos, count = ints(0, 37, cap - T // 2 - 1), ints(T, max(T - 2, 0), T)
    got = mog.rope_store(*made[0], pos, count, q, k, v, r)
    want = mog.rope(q, pos, r)
    for b in range(B):
        n = int(count[b])
        assert torch.equal(got[b, :n], want[b, :n])
    mog.kv_store(*made[1], pos, count, mog.rope(k, pos, r), v.contiguous())

    def held(c):
        c = c[0] if c[1] is None else c
        t = c if isinstance(c, tuple) else [x for x in (c.K, c.V, getattr(c, "k_scale", None), getattr(c, "v_scale", None)) if x is not None]
        return [x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x for x in t]

    for x, y in zip(held(made[0]), held(made[1])):
        assert torch.equal(x, y)
    # queries in place
    mog.rope_store(*made[0], pos, count, q, k, v, r, q_out=q)
    assert torch.equal(q[0], want[0])


def test_rope_store_refusals():
    (K, V), _ = caches("i8", 40, 2, 2, 64)
    r, x = mog.Rope(64), rows(41, 2, 3, 2, D)
    q = rows(42, 2, 3, 8, D)
    for args in ((q.float(), x, x), (q[:1], x, x), (q, x[:, :2], x), (q, x, x.float()), (q, x, rows(1, 2, 3, 4, D)[:, :, :2]),
                 (q[:, :2], x, x)):
        with pytest.raises(ValueError):
            mog.rope_store(K, V, ints(0, 0), None, *args, r)
    with pytest.raises(ValueError, match="Rope is on cpu"):
        mog.rope_store(K, V, ints(0, 0), None, q, x, x, mog.Rope(64, device="cpu"))
    with pytest.raises(ValueError, match="share memory"):
        mog.rope_store(K, V, ints(0, 0), None, q, x, x, r, q_out=q[:1].expand(2, -1, -1, -1))


def test_int8_cache_refusals():
    K = torch.zeros((4, 2, 64, D), dtype=torch.int8, device=DEV)
    s = torch.ones((4, 2, 2), device=DEV)
    table = torch.zeros((2, 2), dtype=torch.int32, device=DEV)
    mog.KVI8(K, K.clone(), s, s.clone(), 32)
    for args in ((K, K.float(), s, s, 32), (K, K.clone(), s, s, 24), (K, K.clone(), s, s, 64), (K, K.clone(), s, s.double(), 32),
                 (K, K[:, :, :32], s, s, 32), (K, K.clone(), s, s.transpose(0, 1).contiguous().transpose(0, 1), 32)):
        with pytest.raises(ValueError):
            mog.KVI8(*args)
    with pytest.raises(ValueError, match="page_rows"):
        mog.PagedKVI8(K, K.clone(), s, s.clone(), table, 32, 32)
    with pytest.raises(ValueError, match="block_table"):
        mog.PagedKVI8(K, K.clone(), s, s.clone(), table.long(), 64, 32)
    with pytest.raises(ValueError, match="16 bytes"):
        mog.PagePool(K[:, :1].contiguous(), K[:, :1].contiguous(), 2, 2, k_scale=s[:, :1].contiguous(), v_scale=s[:, :1].contiguous())
    with pytest.raises(ValueError):
        mog.build(mog.KVI8(K, K.clone(), s, s.clone(), 32), None, [64] * 4, mog.make_params(4, 2, 2, 64))


# ----------------------------------------------------------------- attention over int8 blocks

def attended(q, K, V):
    """(softmax(q K^T / sqrt D) V, sum of weights times |V|) in 64 bits."""
    p = torch.softmax(q.double() @ K.T / math.sqrt(D), -1)
    return p @ V, p @ V.abs()


@pytest.mark.parametrize("G", [1, 4, 7, 12, 16])
@pytest.mark.parametrize("lens,page,block", [((1, 0, 1000), 16, 16), ((300, 77), 64, 32), ((129, 5000), 0, 128), ((70000,), 128, 64)])
@pytest.mark.parametrize("bf16_out", [False, True])
def test_dense_over_int8_blocks(G, lens, page, block, bf16_out):
    B, H, n_max = len(lens), 2, max(lens)
    cap = n_max if page == 0 else -(-n_max // page) * page
    c = Cache8(50, B, H, cap, block, page)
    for s in c.pools[2:] if page else (c.ks, c.vs):
        s.mul_(2.0 ** -10)  # scales of rows of size one
    q = rows(51, B, H * G, D, spread=0.0)
    lengths = ints(*lens)
    out = torch.empty(q.shape, dtype=torch.bfloat16 if bf16_out else torch.float32, device=DEV)
    mog.dense_decode(c.cache, None, lengths, n_max, q, out=out)
    codes, scales = c.state()
    for b, n in enumerate(lens):
        for h in range(H):
            got = out[b, h * G:(h + 1) * G].double()
            if n == 0:
                assert (got == 0).all()
                continue
            K, V = (x[b, h, :n].double() * s[b, h].double().repeat_interleave(block)[:n, None] for x, s in zip(codes, scales))
            want, size = attended(q[b, h * G:(h + 1) * G], K, V)
            # logits to 2^-22 of |q||k| sums (up to about 60 here: 2^-16), weights to 2^-22 (one part: 2^-11), sums of n / 16 tiles
            one_part = bf16_out and G > 8
            rel = 2.0 ** -15 + (2.0 ** -10 if one_part else 2.0 ** -21)
            assert ((got - want).abs() <= rel * size + (BF * want.abs() if bf16_out else 0)).all(), (b, h)


@pytest.mark.parametrize("G", [2, 12])
@pytest.mark.parametrize("spread", [0, 12, 40])
def test_dense_over_int8_blocks_of_very_different_scales(G, spread):
    """Value scales up to 2^spread apart, blocks of zeros as a store leaves them (the least scale), and a scale of 0."""
    g = gen(90 + spread)
    n, block = 2000, 32
    blocks = -(-n // block)
    codes = [torch.randint(-127, 128, (1, 2, n, D), generator=g, device=DEV, dtype=torch.int8) for _ in range(2)]
    ks = torch.full((1, 2, blocks), 1 / 64, device=DEV)
    vs = torch.exp2(torch.randint(-spread, spread + 1, (1, 2, blocks), generator=g, device=DEV).float())
    for i in range(0, blocks, 3):
        codes[1][:, :, i * block:(i + 1) * block] = 0
        vs[:, :, i] = LEAST
    vs[0, 1, 4], ks[0, 1, 7] = 0.0, 0.0
    q = rows(91, 1, 2 * G, D, spread=0.0)
    out = mog.dense_decode(mog.KVI8(*codes, ks, vs, block), None, ints(n), n, q)
    for h in range(2):
        K, V = (x[0, h].double() * s[0, h].double().repeat_interleave(block)[:n, None] for x, s in zip(codes, (ks, vs)))
        want, size = attended(q[0, h * G:(h + 1) * G], K, V)
        # as above; and a weight * scale is held to 2^-24 of the largest one of a row that is not zero
        p = torch.softmax(q[0, h * G:(h + 1) * G].double() @ K.T / math.sqrt(D), -1)
        top = (p * vs[0, h].double().repeat_interleave(block)[:n]).amax(-1, keepdim=True) * 127 * n * 2.0 ** -24
        assert ((out[0, h * G:(h + 1) * G].double() - want).abs() <= 2.0 ** -14 * size + top).all(), h


def test_dense_over_stored_zeros_and_nan():
    """Zeros stored as keys and values weigh in; a NaN row shows in its head alone."""
    c = Cache8(95, 1, 3, 128, 32)
    k, v = rows(96, 1, 100, 3, D, spread=0.0), rows(97, 1, 100, 3, D, spread=0.0)
    k[:, 32:64], v[:, 32:64] = 0, 0
    v[0, 99, 2, 5] = float("nan")
    mog.kv_store(c.cache, None, ints(0), None, k, v)
    q = rows(98, 1, 3, D, spread=0.0)
    out = mog.dense_decode(c.cache, None, ints(100), 100, q)
    for h in range(2):
        K, V = (x[0, h, :100].double() * s[0, h].double().repeat_interleave(32)[:100, None] for x, s in ((c.K, c.ks), (c.V, c.vs)))
        assert (K[32:64] == 0).all() and (V[32:64] == 0).all()
        want, size = attended(q[0, h:h + 1], K, V)
        assert ((out[0, h].double() - want[0]).abs() <= 2.0 ** -14 * size[0]).all()
    assert torch.isnan(out[0, 2]).all()


def test_diff_over_int8_blocks():
    """The same rows in 16-bit products: the differential step over int8 blocks and over their bf16 values.
    int8 codes with power-of-two scales are bf16 values, so both steps read the same rows."""
    g = gen(52)
    B, H, G, n = 2, 2, 3, 700
    codes = [torch.randint(-127, 128, (B, H, n, D), generator=g, device=DEV, dtype=torch.int8) for _ in range(2)]
    scales = [torch.exp2(torch.randint(-7, -4, (B, H, -(-n // 64)), generator=g, device=DEV).float()) for _ in range(2)]
    K, V = ((x.float() * s.repeat_interleave(64, -1)[..., :n, None]).bfloat16() for x, s in zip(codes, scales))
    q, lam = rows(53, B, H * G, D, spread=0.0), 0.1 * torch.randn((4, 64), generator=g, device=DEV)
    lengths = ints(n, 333)
    a = mog.diff_decode(mog.KVI8(*codes, *scales, 64), None, lengths, n, q, lam, 0.4)
    b = mog.diff_decode(K, V, lengths, n, q, lam, 0.4)
    assert ((a - b).abs() <= 2.0 ** -13 * b.abs().amax(-1, keepdim=True)).all()  # (both within 2^-14 of the 64-bit result)


def test_dense_over_int8_rows_of_the_code_minus_128():
    """A byte that a store never writes, and that an e4m3 reader would take for a zero."""
    V = torch.full((1, 1, 100, D), -128, dtype=torch.int8, device=DEV)
    K = torch.zeros_like(V)
    s = torch.full((1, 1, 4), 0.5, device=DEV)
    out = mog.dense_decode(mog.KVI8(K, V, s, s.clone(), 32), None, ints(100), 100, rows(54, 1, 2, D))
    assert ((out + 64).abs() <= 64 * 2.0 ** -20).all()


def test_prompt_forked_grown_and_attended_over_int8_pages():
    """Rotary store, fork, growth with copy on write, a step, attention and read-back together."""
    B, H, G, R, block, n = 3, 4, 2, 32, 16, 45
    K, V = (torch.zeros((16, H, R, D), dtype=torch.int8, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros((16, H, R // block), device=DEV) for _ in range(2))
    pool = mog.PagePool(K, V, B, 4, k_scale=ks, v_scale=vs)
    c, r = pool.cache(), mog.Rope(64, base=10000.0)
    assert isinstance(c, mog.PagedKVI8) and c.block_rows == block
    model = [torch.zeros((B, H, 128, D), dtype=torch.float64, device=DEV) for _ in range(2)]

    def step(seed, *counts):
        pos, granted = pool.grow(ints(*counts))
        T = max(counts)
        x = rows(seed, B, T, (G + 2) * H, D)
        q = mog.rope_store(c, None, pos, granted, x[:, :, : G * H], x[:, :, G * H:(G + 1) * H], x[:, :, (G + 1) * H:], r)
        return pos.clone(), q

    step(60, n, 0, 0)
    pool.assign(ints(0, 0, 0))
    pos, q = step(61, 1, 2, 0)
    step(62, 0, 0, 1)
    assert pool.status() == 0 and pool.lengths.tolist() == [n + 1, n + 2, n + 1]
    got = [torch.zeros((B, 64, H, D), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    mog.kv_load(c, None, ints(0, 0, 0), pool.lengths, *got)
    for i, (codes, scales) in enumerate(((K, ks), (V, vs))):
        rows64 = codes.double() * scales.double().repeat_interleave(block, -1)[..., None]
        model[i] = rows64[pool.block_table.clamp_min(0).long()].transpose(1, 2).flatten(2, 3)
    # the prompt's full blocks are the same rows in every sequence
    assert torch.equal(got[0][0, :32], got[0][1, :32]) and torch.equal(got[0][0, :32], got[0][2, :32])
    q = q[:, 0].contiguous()
    out = mog.dense_decode(c, None, pool.lengths, 64, q)
    for b, m in enumerate(pool.lengths.tolist()):
        for i in range(2):
            assert torch.equal(got[i][b, :m], model[i][b, :, :m].transpose(0, 1).float().bfloat16())
        if b == 2:
            continue  # (it had no query of its own in that step)
        for h in range(H):
            want, size = attended(q[b, h * G:(h + 1) * G], model[0][b, h, :m], model[1][b, h, :m])
            assert ((out[b, h * G:(h + 1) * G].double() - want).abs() <= 2.0 ** -14 * size).all()


def test_captured_and_on_another_stream():
    c = Cache8(70, 2, 2, 256, 64, 64)
    r = mog.Rope(128)
    q, k, v = rows(71, 2, 3, 4, D), rows(72, 2, 3, 2, D), rows(73, 2, 3, 2, D)
    pos, qo = ints(0, 70), torch.empty_like(q)
    out = [torch.zeros_like(k) for _ in range(2)]

    def call():
        mog.rope_store(c.cache, None, pos, None, q, k, v, r, q_out=qo)
        mog.kv_load(c.cache, None, pos, None, *out)

    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    c.store([0, 70], [3, 3], (mog.rope(k, pos, r), v))
    c.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for p in ([3, 73], [200, 0], [64, 255]):
        pos.copy_(torch.tensor(p, dtype=torch.int32))
        k.copy_(rows(74 + p[0], 2, 3, 2, D))
        graph.replay()
        torch.cuda.synchronize()
        c.store(p, [3, 3], (mog.rope(k, pos, r), v))
        c.check()
        assert torch.equal(qo, mog.rope(q, pos, r))


def test_rows_past_32_bit_offsets():
    """Rows of one head spread over more than 4 GiB, new rows as far apart, and their read-back."""
    n, stride = 40000, 128 * 1024
    big = torch.zeros(n * stride, dtype=torch.int8, device=DEV)
    K, V = (big[at:].as_strided((1, 1, n, D), (n * stride, n * stride, stride, 1)) for at in (0, 1024))
    s = torch.zeros((1, 1, n // 64), device=DEV)
    c = mog.KVI8(K, V, s, s.clone(), 64)
    x = rows(80, 1, 70, 1, D)
    mog.kv_store(c, None, ints(n - 70), None, x, x)
    out = [torch.zeros_like(x) for _ in range(2)]
    mog.kv_load(c, None, ints(n - 70), None, *out)
    step = s[0, 0, (n - 70) // 64:].max()
    assert ((out[0].double() - x.double()).abs() <= step.double() * 0.51 + BF * x.double().abs()).all()
    assert torch.equal(out[0], out[1])
