"""Host-side checks of rotary positions, int8 caches and their read-back: every refusal comes before any
device work, and the frequencies are those of their formulas."""
import ctypes as C
import math

import pytest

torch = pytest.importorskip("torch")

import serving_mog_decode_gb300 as mog
from serving_mog_decode_gb300 import buildlib

P = C.c_void_p(1 << 20)  # a 16-byte aligned address that no refused call reads
ODD = C.c_void_p((1 << 20) + 8)
OK, ARG, SHAPE, SMALL = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    buildlib.build()
    return mog.lib()


def cache(**kw):
    base = dict(type=3, n_cap=1 << 20, k=P.value, v=P.value, k_scale=P.value, v_scale=P.value, stride_b=8 << 27,
                stride_h=1 << 27, stride_n=128, scale_b=8 << 16, scale_h=1 << 16, scale_n=1, block_rows=64)
    base.update(kw)
    return mog.Cache(**base)


BAD_CACHES = [
    (dict(k=None), ARG), (dict(k_scale=None), ARG), (dict(v_scale=P.value + 2), ARG), (dict(stride_n=64), SHAPE),
    (dict(stride_n=136), SHAPE), (dict(block_rows=0), SHAPE), (dict(block_rows=8), SHAPE), (dict(block_rows=48), SHAPE),
    (dict(block_rows=256), SHAPE), (dict(block_rows=-64), SHAPE), (dict(type=2), ARG), (dict(type=4), ARG),
    (dict(block_table=P.value, page_rows=32, pages_per_seq=1 << 18, n_pages=64), SHAPE),
    (dict(block_table=P.value, page_rows=64, pages_per_seq=1 << 18, n_pages=0), SHAPE),
]
S3 = (C.c_int64 * 3)(1024, 1024, 128)
S_ODD = (C.c_int64 * 3)(1024, 1028, 128)


def rope_params(**kw):
    base = dict(turns=P.value, rot_dim=64, layout=0, factor=1.0)
    base.update(kw)
    return mog.RopeParams(**base)


BAD_ROPES = [(dict(turns=None), ARG), (dict(turns=P.value + 4), ARG), (dict(rot_dim=0), SHAPE), (dict(rot_dim=24), SHAPE),
             (dict(rot_dim=144), SHAPE), (dict(rot_dim=-16), SHAPE), (dict(layout=2), ARG),
             (dict(factor=float("nan")), ARG), (dict(factor=float("inf")), ARG)]


def test_store_load_and_decode_refuse_bad_int8_caches(lib):
    def store(c):
        return lib.mog_kv_store(C.byref(c), 2, 8, 128, 1, P, None, P, P, 1024, 1024, 128, None)

    def load(c):
        return lib.mog_kv_load(C.byref(c), 2, 8, 128, 1, P, None, P, P, 1024, 1024, 128, None)

    def dense(c):
        return lib.dense_decode8(C.byref(c), P, 1 << 20, 2, 8, 32, 128, P, P, 0, P, 1 << 40, None)

    def both(c):
        return lib.mog_rope_store(C.byref(c), C.byref(rope_params()), 2, 8, 32, 128, 1, P, None, P, S3, P, S3, P, P, S3, None)

    for kw, why in BAD_CACHES:
        for call in (store, load, dense, both):
            assert call(cache(**kw)) == why, (kw, call.__name__)


def test_load_refusals(lib):
    def load(batch=2, h_kv=8, d=128, t=1, pos=P, k=P, v=P, sb=1024, st=1024, sh=128):
        return lib.mog_kv_load(C.byref(cache()), batch, h_kv, d, t, pos, None, k, v, sb, st, sh, None)

    for kw, why in [(dict(batch=0), ARG), (dict(h_kv=0), ARG), (dict(t=0), ARG), (dict(d=64), SHAPE),
                    (dict(batch=65536), SHAPE), (dict(t=1 << 27), SHAPE), (dict(pos=None), ARG), (dict(k=None), ARG),
                    (dict(v=ODD), ARG), (dict(st=1028), SHAPE)]:
        assert load(**kw) == why, kw
    assert lib.mog_kv_load(None, 2, 8, 128, 1, P, None, P, P, 1024, 1024, 128, None) == ARG


def test_rope_refusals(lib):
    def apply(r=None, batch=2, heads=8, d=128, t=1, pos=P, x=P, xs=S3, out=P, os_=S3):
        return lib.mog_rope_apply(C.byref(r if r is not None else rope_params()), batch, heads, d, t, pos, 0, None, 0, x,
                                  xs, out, os_, None)

    def store(r=None, batch=2, h_kv=8, h_q=32, d=128, t=1, pos=P, q=P, qs=S3, qo=P, os_=S3, k=P, v=P, ks=S3):
        return lib.mog_rope_store(C.byref(cache()), C.byref(r if r is not None else rope_params()), batch, h_kv, h_q, d, t,
                                  pos, None, q, qs, qo, os_, k, v, ks, None)

    for kw, why in BAD_ROPES:
        assert apply(rope_params(**kw)) == why and store(rope_params(**kw)) == why, kw
    for kw, why in [(dict(batch=0), ARG), (dict(heads=0), ARG), (dict(t=0), ARG), (dict(d=64), SHAPE),
                    (dict(batch=65536), SHAPE), (dict(t=(1 << 27) + 1), SHAPE), (dict(pos=None), ARG), (dict(x=None), ARG),
                    (dict(x=ODD), ARG), (dict(out=None), ARG), (dict(xs=S_ODD), SHAPE), (dict(os_=S_ODD), SHAPE),
                    (dict(xs=None), ARG), (dict(os_=None), ARG)]:
        assert apply(**kw) == why, kw
    for kw, why in [(dict(batch=0), ARG), (dict(h_kv=0), ARG), (dict(h_q=0), ARG), (dict(t=0), ARG), (dict(d=64), SHAPE),
                    (dict(batch=65536), SHAPE), (dict(t=1 << 25), SHAPE), (dict(pos=None), ARG), (dict(q=None), ARG),
                    (dict(qo=ODD), ARG), (dict(k=ODD), ARG), (dict(v=None), ARG), (dict(qs=S_ODD), SHAPE),
                    (dict(os_=S_ODD), SHAPE), (dict(ks=S_ODD), SHAPE), (dict(ks=None), ARG)]:
        assert store(**kw) == why, kw
    assert lib.mog_rope_apply(None, 2, 8, 128, 1, P, 0, None, 0, P, S3, P, S3, None) == ARG
    assert lib.mog_rope_store(None, C.byref(rope_params()), 2, 8, 32, 128, 1, P, None, P, S3, P, S3, P, P, S3, None) == ARG


def test_frequencies():
    f, a = mog.rope_frequencies(64, 10000.0)
    assert a == 1.0 and len(f) == 32 and f[0] == 1.0 and abs(f[16] - 0.01) < 1e-15
    g, _ = mog.rope_frequencies(64, 10000.0, dict(type="linear", factor=4))
    assert all(x == y / 4 for x, y in zip(g, f))
    g, _ = mog.rope_frequencies(64, 10000.0, dict(type="ntk", factor=4))
    assert g[0] == 1.0 and abs(g[31] / (f[31] / 4) - 1) < 1e-12  # the slowest pair is interpolated in full
    yarn = dict(type="yarn", factor=8, original_len=4096)
    g, a = mog.rope_frequencies(128, 10000.0, yarn)
    f, _ = mog.rope_frequencies(128, 10000.0)
    assert abs(a - (0.1 * math.log(8) + 1)) < 1e-15
    turns = [4096 * x / (2 * math.pi) for x in f]
    for x, y, t in zip(g, f, turns):
        assert (x == y or t < 40) and (abs(x * 8 / y - 1) < 1e-12 or t > 0.8) and y / 8 <= x * (1 + 1e-12) and x <= y
    assert mog.rope_frequencies(128, 10000.0, dict(yarn, attention_factor=1.5))[1] == 1.5
    g, a = mog.rope_frequencies(128, 500000.0, dict(type="bands", factor=8, original_len=8192, low=1, high=4))
    f, _ = mog.rope_frequencies(128, 500000.0)
    assert a == 1.0
    for x, y in zip(g, f):
        t = 8192 * y / (2 * math.pi)
        k = min(max((t - 1) / 3, 0), 1)
        assert abs(x - (y * k + y / 8 * (1 - k))) < 1e-15
    for bad in (dict(type="cubic", factor=2), dict(type="linear", factor=0), dict(type="bands", factor=2, original_len=4, low=2, high=2)):
        with pytest.raises(ValueError):
            mog.rope_frequencies(64, 10000.0, bad)


def test_turns_are_exact_fractions():
    """The 64-bit fractions of a turn, against integer arithmetic of 2 pi to 30 digits."""
    two_pi = 6283185307179586476925286766559  # * 10^-30
    f = mog.rope_frequencies(128, 10000.0)[0] + [7.0, -0.5, 0.0]
    f = f[:61] + f[-3:]
    r = mog.Rope(128, inv_freq=f, device="cpu")
    assert r.turns.dtype == torch.int64 and r.turns.shape == (64,)
    for x, t in zip(f, r.turns.tolist()):
        num, den = float(x).as_integer_ratio()
        want = (num * 10 ** 30 << 64) // (den * two_pi)
        off = (t - want + (1 << 63)) % (1 << 64) - (1 << 63)
        assert abs(off) <= max(abs(want) >> 51, 4), (x, off)  # fp64 of x / 2 pi: two roundings


def test_rope_object_refusals():
    for kw in (dict(rot_dim=8), dict(rot_dim=40), dict(rot_dim=144), dict(rot_dim=64, inv_freq=[1.0] * 31),
               dict(inv_freq=[1.0] * 64, scaling=dict(type="linear", factor=2)), dict(factor=float("nan"))):
        with pytest.raises(ValueError):
            mog.Rope(device="cpu", **kw)
    r = mog.Rope(device="cpu")
    with pytest.raises(AttributeError, match="fixed"):
        r.factor = 2.0


def test_int8_cache_shapes_are_checked():
    """(Host tensors: the device check is the last word of each.)"""
    K = torch.zeros((2, 3, 100, 128), dtype=torch.int8)
    s = torch.ones((2, 3, 4))
    for rows, ks, vs, block in ((K.float(), s, s, 32), (K[..., ::2], s, s, 32)):
        with pytest.raises(ValueError):
            mog.KVI8(rows, rows, ks, vs, block)
    with pytest.raises(ValueError, match="CUDA int8"):
        mog.KVI8(K, K, s, s, 32)


def test_cross_refusals(lib):
    def cross(c=None, lengths=P, n_max=1 << 20, batch=2, h_kv=8, h_q=32, d=128, t=4, q=P, qs=S3, out=P, os_=S3, scratch=P,
              nbytes=1 << 40):
        c = c if c is not None else cache(type=0, k_scale=None, v_scale=None)
        return lib.mog_cross_attend(C.byref(c), lengths, n_max, batch, h_kv, h_q, d, t, None, q, qs, out, os_, scratch,
                                    nbytes, None)

    assert cross(cache()) == ARG and cross(cache(type=0)) == ARG
    for kw, why in [(dict(k=None), ARG), (dict(v=ODD.value), ARG), (dict(stride_n=64), SHAPE), (dict(n_cap=100), SHAPE),
                    (dict(stride_b=1 << 39), SHAPE), (dict(stride_h=1 << 39), SHAPE), (dict(stride_n=1 << 39), SHAPE),
                    (dict(block_table=P.value, page_rows=64, pages_per_seq=1 << 18, n_pages=4, stride_h=0), SHAPE),
                    (dict(block_table=P.value, page_rows=64, pages_per_seq=1 << 18, n_pages=4, stride_b=0), SHAPE),
                    (dict(block_table=P.value, page_rows=24, pages_per_seq=1 << 18, n_pages=4), SHAPE)]:
        assert cross(cache(**dict(dict(type=0, k_scale=None, v_scale=None), **kw))) == why, kw
    for kw, why in [(dict(lengths=None), ARG), (dict(n_max=0), ARG), (dict(n_max=(1 << 20) + 1), SHAPE),
                    (dict(n_max=(1 << 30) + 1), SHAPE), (dict(batch=0), ARG), (dict(h_kv=0), ARG), (dict(h_q=0), ARG),
                    (dict(h_q=33), SHAPE), (dict(h_kv=1, h_q=17), SHAPE), (dict(batch=8192), SHAPE), (dict(d=64), SHAPE),
                    (dict(t=0), ARG), (dict(t=1 << 26), SHAPE), (dict(q=None), ARG), (dict(q=ODD), ARG), (dict(out=ODD), ARG),
                    (dict(qs=S_ODD), SHAPE), (dict(os_=S_ODD), SHAPE), (dict(qs=None), ARG), (dict(scratch=None), ARG),
                    (dict(qs=(C.c_int64 * 3)(1024, 0, 128)), SHAPE), (dict(qs=(C.c_int64 * 3)(1024, 1024, 0)), SHAPE),
                    (dict(qs=(C.c_int64 * 3)(-1024, 1024, 128)), SHAPE), (dict(qs=(C.c_int64 * 3)(1 << 35, 1024, 128)), SHAPE),
                    (dict(batch=4096, n_max=1 << 19, t=1 << 13, h_q=8), SHAPE),
                    (dict(scratch=ODD), ARG), (dict(nbytes=16), SMALL)]:
        assert cross(**kw) == why, kw
    assert mog.cross_scratch_bytes(1, 2, 8, 20, 200) == 0 and mog.cross_scratch_bytes(1, 1, 1, 20, 1 << 20) > 0
