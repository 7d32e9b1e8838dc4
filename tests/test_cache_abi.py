"""Host-side checks of the cache, differential-decode and page calls: every refusal comes
before any device work, so these run without a GPU."""
import ctypes as C

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
    base = dict(type=1, n_cap=1 << 20, k=P.value, v=P.value, k_scale=P.value, v_scale=P.value, stride_b=8 << 27,
                stride_h=1 << 27, stride_n=128, scale_b=8 << 20, scale_h=1 << 20, scale_n=1)
    base.update(kw)
    return mog.Cache(**base)


BAD_CACHES = [
    (dict(k=None), ARG), (dict(v=None), ARG), (dict(k=ODD.value), ARG), (dict(type=2), ARG), (dict(type=-1), ARG),
    (dict(k_scale=None), ARG), (dict(v_scale=P.value + 2), ARG), (dict(stride_n=64), SHAPE), (dict(stride_n=136), SHAPE),
    (dict(stride_h=(1 << 27) + 8), SHAPE), (dict(stride_b=-16), SHAPE), (dict(n_cap=(1 << 20) - 1), SHAPE),
    (dict(block_table=P.value, page_rows=8, pages_per_seq=1 << 18, n_pages=64), SHAPE),
    (dict(block_table=P.value, page_rows=24, pages_per_seq=1 << 18, n_pages=64), SHAPE),
    (dict(block_table=P.value, page_rows=16, pages_per_seq=0, n_pages=64), SHAPE),
    (dict(block_table=P.value, page_rows=16, pages_per_seq=(1 << 16) - 1, n_pages=64), SHAPE),
    (dict(block_table=P.value, page_rows=16, pages_per_seq=1 << 16, n_pages=0), SHAPE),
]


def dense8(lib, c, n_max=1 << 20, batch=2, h_kv=8, h_q=32, d=128, q=P, out=P, out_type=0, scratch=P, nbytes=1 << 40,
           lengths=P):
    return lib.dense_decode8(C.byref(c) if c else None, lengths, n_max, batch, h_kv, h_q, d, q, out, out_type, scratch,
                             nbytes, None)


def diff(lib, c, n_max=1 << 20, batch=2, h_kv=8, h_q=32, d=128, q=P, out=P, out_type=0, scratch=P, nbytes=1 << 40,
         lengths=P, prm=None, **kw):
    base = dict(lam=P.value, gamma=P.value, lam_heads=1, lambda_init=0.5, eps=1e-5)
    base.update(kw)
    prm = mog.DiffParams(**base)
    return lib.mog_diff_decode(C.byref(c) if c else None, lengths, n_max, batch, h_kv, h_q, d, q, C.byref(prm), out,
                               out_type, scratch, nbytes, None)


@pytest.mark.parametrize("call", [dense8, diff])
def test_decode_refusals(lib, call):
    for kw, why in BAD_CACHES:
        assert call(lib, cache(**kw)) == why, kw
    assert call(lib, None) == ARG
    most = 16 if call is dense8 else 8
    for kw, why in [(dict(n_max=0), ARG), (dict(batch=0), ARG), (dict(h_kv=0), ARG), (dict(h_q=0), ARG),
                    (dict(d=64), SHAPE), (dict(h_q=33), SHAPE), (dict(h_kv=1, h_q=most + 1), SHAPE),
                    (dict(n_max=(1 << 20) + 1), SHAPE), (dict(n_max=(1 << 30) + 1), SHAPE), (dict(batch=1 << 28), SHAPE), (dict(q=None), ARG), (dict(q=ODD), ARG),
                    (dict(out=None), ARG), (dict(out=ODD), ARG), (dict(out_type=2), ARG), (dict(scratch=None), ARG),
                    (dict(scratch=ODD), ARG), (dict(lengths=None), ARG), (dict(nbytes=16), SMALL)]:
        assert call(lib, cache(), **kw) == why, kw
    assert dense8(lib, cache(type=0, k_scale=None, v_scale=None)) == ARG  # bf16 rows: dense_decode
    assert diff(lib, cache(type=0)) == ARG                                # bf16 rows have no scales


def test_diff_parameter_refusals(lib):
    for kw, why in [(dict(lam=None), ARG), (dict(lam=ODD.value), ARG), (dict(gamma=ODD.value), ARG),
                    (dict(lam_heads=8), SHAPE), (dict(lam_heads=0), SHAPE), (dict(eps=0.0), ARG),
                    (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG), (dict(lambda_init=float("inf")), ARG)]:
        assert diff(lib, cache(), **kw) == why, kw
    assert lib.mog_diff_decode(C.byref(cache()), P, 1 << 20, 2, 8, 32, 128, P, None, P, 0, P, 1 << 40, None) == ARG


def test_scratch_grows_with_the_heads_and_maps(lib):
    a, b = mog.dense8_scratch_bytes(2, 8, 8, 1 << 20), mog.dense8_scratch_bytes(2, 8, 16, 1 << 20)
    assert a > 0 and b == 2 * a and mog.diff_scratch_bytes(2, 8, 8, 1 << 20) == 2 * a
    assert mog.dense8_scratch_bytes(1, 1, 1, 64) == 0  # short: one launch without scratch
    with pytest.raises(mog.MogError, match="SHAPE"):
        mog.diff_scratch_bytes(1, 1, 9, 4096)


def test_store_refusals(lib):
    def store(c, batch=2, h_kv=8, d=128, t=1, pos=P, k=P, v=P, sb=1024, st=1024, sh=128):
        return lib.mog_kv_store(C.byref(c) if c else None, batch, h_kv, d, t, pos, None, k, v, sb, st, sh, None)

    for kw, why in BAD_CACHES:
        if "n_cap" not in kw and kw.get("pages_per_seq") != (1 << 16) - 1:  # (a store may have fewer positions)
            assert store(cache(**kw)) == why, kw
    for kw, why in [(dict(batch=0), ARG), (dict(h_kv=0), ARG), (dict(t=0), ARG), (dict(d=256), SHAPE),
                    (dict(batch=65536), SHAPE), (dict(t=(1 << 26) + 1), SHAPE), (dict(pos=None), ARG), (dict(k=None), ARG), (dict(v=ODD), ARG),
                    (dict(sb=4), SHAPE), (dict(st=4), SHAPE), (dict(sh=130), SHAPE)]:
        assert store(cache(), **kw) == why, kw
    assert store(None) == ARG


def test_page_refusals(lib):
    need = C.c_size_t()
    assert lib.mog_pages_work_bytes(64, 4, C.byref(need)) == OK and need.value >= 4 * 64 * 3
    assert lib.mog_pages_work_bytes(64, 4097, C.byref(need)) == SHAPE
    assert lib.mog_pages_work_bytes(0, 4, C.byref(need)) == ARG
    lib.mog_pages_work_bytes(64, 4, C.byref(need))

    def pages(pool=(1 << 20, 4096, 4096), **kw):
        desc = (mog.PagePoolDesc * 1)(mog.PagePoolDesc(*pool))
        base = dict(n_pages=64, page_rows=16, batch=4, pages_per_seq=16, block_table=P.value, lengths=P.value,
                    refs=P.value, work=P.value, work_bytes=need.value, pools=desc, n_pools=1)
        base.update(kw)
        return mog.Pages(**base)

    calls = [lambda p: lib.mog_pages_assign(p, P, None), lambda p: lib.mog_pages_grow(p, P, P, P, None),
             lambda p: lib.mog_pages_compact(p, None), lambda p: lib.mog_pages_status(p, None)]
    for kw, why in [(dict(n_pages=0), ARG), (dict(batch=0), ARG), (dict(batch=5000), SHAPE), (dict(page_rows=8), SHAPE),
                    (dict(page_rows=48), SHAPE), (dict(pages_per_seq=0), SHAPE), (dict(pages_per_seq=1 << 28), SHAPE),
                    (dict(block_table=None), ARG), (dict(lengths=None), ARG), (dict(refs=P.value + 2), ARG),
                    (dict(work=None), ARG), (dict(work_bytes=need.value - 4), SMALL), (dict(n_pools=-1), ARG), (dict(n_pools=0), ARG),
                    (dict(pools=None), ARG), (dict(pool=(None, 4096, 4096)), ARG),
                    (dict(pool=((1 << 20) + 4, 4096, 4096)), ARG), (dict(pool=(1 << 20, 4096, 4104)), SHAPE),
                    (dict(pool=(1 << 20, 4096, 8192)), SHAPE), (dict(pool=(1 << 20, 4096, 0)), SHAPE)]:
        for call in calls:
            assert call(C.byref(pages(**kw))) == why, kw
    for call in calls:
        assert call(None) == ARG
    good = pages()
    assert lib.mog_pages_assign(C.byref(good), None, None) == ARG
    assert lib.mog_pages_grow(C.byref(good), P, None, P, None) == ARG
    assert lib.mog_pages_grow(C.byref(good), None, P, P, None) == ARG
    assert lib.mog_pages_grow(C.byref(good), P, P, None, None) == ARG


def test_python_refuses_host_tensors_and_wrong_types():
    k = torch.zeros((2, 1, 16, 128), dtype=torch.float8_e4m3fn)
    s = torch.ones((2, 1, 16))
    t = torch.zeros((1, 2), dtype=torch.int32)
    with pytest.raises(ValueError):
        mog.KV8(k, k, s, s)
    with pytest.raises(ValueError):
        mog.PagedKV8(k, k, s, s, t, 16)
    with pytest.raises(ValueError):
        mog.PagePool(k.bfloat16(), k.bfloat16(), 1, 2)
    with pytest.raises(ValueError):
        mog.kv_store(k.bfloat16(), k.bfloat16(), t[0], None, k, k)
