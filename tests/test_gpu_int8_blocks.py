"""int8 caches further: what adds up in a block whose scale rises again and again, blocks that hold a NaN, page moves, and the
differential step in 64 bits."""
import types

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import serving_mog_decode_gb300 as mog
from serving_mog_decode_gb300 import buildlib
from test_gpu_cache import check_diff, weights
from test_gpu_pages import Model, bits, same, tensors
from test_gpu_rows import Cache8, DEV, D, gen, ints, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    buildlib.build()


@pytest.mark.parametrize("block", [16, 128])
@pytest.mark.parametrize("grow", ["slow", "fast", "any", "down"])
def test_what_rises_of_the_scale_add_up_to(grow, block):
    """Rows stored one by one: a row is off by half a step of the scale that it was stored with, and of every scale that its
    block rose to since.  (fp32: two roundings of up to 127 steps each time, 2^-16 of a step.)"""
    H, n = 2, 128
    x = rows(1, 1, n, H, D, spread=0.0).float()
    x = x / x.abs().amax(-1, keepdim=True)
    t = torch.arange(n, device=DEV)[None, :, None, None]
    x = x * {"slow": 1.003 ** t, "fast": 2.0 ** (t / 8), "down": 0.97 ** t,
             "any": torch.exp2(3 * torch.randn((1, n, H, 1), generator=gen(2), device=DEV))}[grow]
    x = x.bfloat16()
    K, V = (torch.zeros((1, H, n, D), dtype=torch.int8, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros((1, H, n // block), device=DEV) for _ in range(2))
    c = mog.KVI8(K, V, ks, vs, block)
    bound = torch.zeros((H, n), dtype=torch.float64, device=DEV)
    for i in range(n):
        old = ks.clone()
        mog.kv_store(c, None, ints(i), None, x[:, i:i + 1], x[:, i:i + 1])
        b, s = i // block, ks[0, :, i // block].double()
        rose = (ks[0, :, b] > old[0, :, b]).double() * (i % block > 0)
        bound[:, b * block:i] += (rose * s * (0.5 + 2.0 ** -16))[:, None]
        bound[:, i] = s * (0.5 + 2.0 ** -16)
    got = K[0].double() * ks[0].double().repeat_interleave(block, -1)[..., None]
    off = (got - x[0].transpose(0, 1).double()).abs().amax(-1)
    assert (off <= bound).all(), (off / bound).max()
    assert torch.equal(K, V) and torch.equal(ks, vs)
    if grow == "down":  # (a scale that never rises: half a step)
        assert (off <= ks[0].double().repeat_interleave(block, -1) * (0.5 + 2.0 ** -16)).all()


def test_going_back_in_a_block_that_holds_a_nan():
    """The scale is all that a block has: it stays NaN behind the row that made it so, also when that row is given up, until the
    block's first row is written; its codes stay."""
    c = Cache8(3, 1, 2, 64, 32)
    k, v = rows(4, 1, 20, 2, D), rows(5, 1, 20, 2, D)
    k[0, 19, 1, 7] = float("nan")
    for pos, n in ((0, 19), (19, 1), (12, 3), (10, 1)):
        part = k[:, pos:pos + n].clone(), v[:, pos:pos + n].clone()
        mog.kv_store(c.cache, None, ints(pos), None, *part)
        c.store([pos], [n], part)
        c.check()
    assert torch.isnan(c.ks[0, 1, 0]) and torch.isfinite(c.ks[0, 0, 0]) and torch.isfinite(c.vs[0, :, 0]).all()
    before = c.K.clone()
    mog.kv_store(c.cache, None, ints(5), None, k[:, :2].contiguous(), v[:, :2].contiguous())
    assert torch.equal(c.K[0, 1], before[0, 1]) and torch.isnan(c.ks[0, 1, 0])
    fresh = rows(6, 1, 3, 2, D)
    mog.kv_store(c.cache, None, ints(0), None, fresh, fresh)
    assert torch.isfinite(c.ks[0, :, 0]).all()


@pytest.mark.parametrize("layers,heads_first,block", [(1, True, 16), (2, False, 16), (1, True, 32)])
def test_pages_move_with_their_scales(layers, heads_first, block):
    """Random forks, frees, growth and compaction of int8 pools, codes and scales bit for bit."""
    n_pages, R, batch, pps, H = 60, 32, 7, 12, 4
    g = gen(7)
    tail = (H, R) if heads_first else (R, H)
    small = (H, R // block) if heads_first else (R // block, H)
    K, V = ([torch.randint(-127, 128, (n_pages,) + tail + (D,), generator=g, device=DEV, dtype=torch.int8) for _ in range(layers)] for _ in range(2))
    ks, vs = ([torch.rand((n_pages,) + small, generator=g, device=DEV) for _ in range(layers)] for _ in range(2))
    pool, model = mog.PagePool(K, V, batch, pps, heads_first=heads_first, k_scale=ks, v_scale=vs), Model(n_pages, R, batch, pps)
    before = [bits(t) for t in tensors(pool)]
    rng = np.random.default_rng(layers)
    for step in range(30):
        what = step % 3 if step < 6 else rng.integers(0, 3)
        if what == 0:
            n = np.where(rng.random(batch) < 0.6, rng.integers(0, 2 * R, batch), 0).tolist()
            assert pool.grow(ints(*n))[1].tolist() == model.grow(n)[1]
        elif what == 1:
            src = np.where(rng.random(batch) < 0.6, np.arange(batch), rng.integers(-1, batch, batch)).tolist()
            pool.assign(ints(*src))
            model.assign(src)
        else:
            pool.compact()
            model.compact()
        same(pool, model, before)
    assert pool.status() in (0, 8)  # (growth may have found no room)
    assert pool.cache(layers - 1).block_rows == block


@pytest.mark.parametrize("G", [1, 4, 5, 8])
@pytest.mark.parametrize("lens,page,block", [((1, 0, 1000), 16, 16), ((300, 77), 64, 32), ((129, 5000), 0, 128)])
@pytest.mark.parametrize("out_type", [torch.float32, torch.bfloat16])
def test_diff_in_64_bits(G, lens, page, block, out_type):
    B, H, n_max = len(lens), 2, max(lens)
    cap = n_max if page == 0 else -(-n_max // page) * page
    c = Cache8(8, B, H, cap, block, page)
    for s in c.pools[2:] if page else (c.ks, c.vs):
        s.mul_(2.0 ** -12)  # scales of rows of size one
    codes, scales = c.state()
    rows64 = [x.double() * s.double().repeat_interleave(block, -1)[..., :cap, None] for x, s in zip(codes, scales)]
    q = rows(9, B, H * G, D, spread=0.0)
    lam, gamma = weights(10)
    out = torch.full(q.shape, float("nan"), dtype=out_type, device=DEV)
    mog.diff_decode(c.cache, None, ints(*lens), n_max, q, lam, 0.5, gamma=gamma, eps=1e-5, out=out)
    check_diff(types.SimpleNamespace(lens=lens, H=H, rows64=rows64), q, out, G, lam, 0.5, gamma, 1e-5)
