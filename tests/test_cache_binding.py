"""What the binding refuses before any device work: pools, streams and attributes that the cache and page
calls cannot take.  Host tensors stand in for device ones, as far as a check looks."""
import types

import pytest

torch = pytest.importorskip("torch")

import serving_mog_decode_gb300 as mog


def paged(**kw):
    """A PagedKV over host tensors, with attributes set anew."""
    p = object.__new__(mog.PagedKV)
    pool = torch.zeros((8, 2, 16, 128), dtype=torch.bfloat16)
    base = dict(K=pool, V=pool.clone(), block_table=torch.zeros((3, 2), dtype=torch.int32), page_rows=16,
                heads_first=True, h_kv=2, device=pool.device, _cache=None, _checked=(None, None))
    for name, value in {**base, **kw}.items():
        setattr(p, name, value)
    return p


SHORT = torch.zeros((7, 2, 16, 128), dtype=torch.bfloat16)
WIDE = torch.zeros((8, 2, 32, 128), dtype=torch.bfloat16)[:, :, :16]
HALF = torch.zeros((8, 2, 16, 128), dtype=torch.float16)


@pytest.mark.parametrize("kw", [dict(V=SHORT), dict(V=WIDE), dict(V=HALF), dict(K=HALF, V=HALF),
                                dict(K=WIDE[..., ::2], V=WIDE[..., ::2])])
def test_a_paged_cache_set_anew_to_pools_that_do_not_match_is_refused(kw):
    assert mog._cache(paged(), None)[1:4] == (3, 2, 32)
    for read in (lambda p: mog._cache(p, None), lambda p: p.struct()):
        with pytest.raises(ValueError, match="pools"):
            read(paged(**kw))
        p = paged()
        read(p)
        for name, value in kw.items():
            setattr(p, name, value)
        with pytest.raises(ValueError, match="pools"):
            read(p)


def test_a_paged_cache_whose_tensors_take_another_shape_in_place_is_read_anew():
    big = torch.zeros((8, 2, 16, 128), dtype=torch.bfloat16)
    p = paged(K=big[:], V=big[:])
    c, batch, h_kv, positions, _ = mog._cache(p, None)
    assert (c.n_pages, c.stride_b, batch, positions) == (8, 4096, 3, 32)
    p.K.data, p.V.data = big[::2], big[::2]  # (the same addresses)
    c = mog._cache(p, None)[0]
    assert (c.n_pages, c.stride_b) == (4, 8192)
    p.K.data = big  # K alone
    with pytest.raises(ValueError, match="pools"):
        mog._cache(p, None)
    p.K.data, p.block_table.data = big[::2], torch.zeros((5, 1), dtype=torch.int32)
    assert mog._cache(p, None)[1:4] == (5, 2, 16)


def test_pools_whose_pages_overlap_are_refused():
    """An expanded pool has one page of memory: strides taken for more would lead out of it."""
    pool = torch.zeros((8, 2, 16, 128), dtype=torch.bfloat16)
    d = mog._pool_desc(pool)
    assert (d.base, d.page_stride, d.page_bytes) == (pool.data_ptr(), 8192, 8192)
    d = mog._pool_desc(pool[1::2])
    assert (d.page_stride, d.page_bytes) == (16384, 8192)
    d = mog._pool_desc(pool[2:3].as_strided((1, 2, 16, 128), (1, 2048, 128, 1)))  # (the stride of one page counts for nothing)
    assert (d.page_stride, d.page_bytes) == (8192, 8192)
    for bad in (pool[:1].expand(8, -1, -1, -1), pool.view(-1).as_strided((8, 2, 16, 128), (2048, 2048, 128, 1)), pool[:0]):
        with pytest.raises(ValueError, match="overlap"):
            mog._pool_desc(bad)


def test_what_a_descriptor_was_made_of_cannot_be_set_anew():
    for cls in (mog.KV8, mog.PagedKV8, mog.PagePool):
        x = object.__new__(cls)
        x.K, x._made = 1, True
        for name in ("K", "block_table"):
            with pytest.raises(AttributeError, match="fixed"):
                setattr(x, name, 2)
        assert x.K == 1


def test_a_stream_of_another_device_is_refused():
    """Taken as it is, the work would go to the current stream of the cache's device instead."""
    stream = types.SimpleNamespace(device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        mog._there(torch.device("cuda", 0), stream)
