"""PagePool over state that the caller has broken, or set anew: reported or refused, and other sequences'
rows stay theirs."""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import serving_mog_decode_gb300 as mog
from serving_mog_decode_gb300 import buildlib
from test_gpu_pages import DEV, bits, ints, make, tensors

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    buildlib.build()
    mog.lib()


def row_bytes(pool, b):
    """The bytes of sequence b's pages in every pool, in the sequence's order."""
    used = -(-int(pool.lengths[b]) // pool.page_rows)
    pages = pool.block_table[b, :used].long()
    return [bits(t)[pages] for t in tensors(pool)]


@pytest.mark.parametrize("grown", [False, True])  # (an earlier call's list in the work buffer)
@pytest.mark.parametrize("slot", [0, 5])          # a page in front of the moved ones, one behind
def test_compaction_reports_a_held_page_that_refs_count_as_free(slot, grown):
    R, n = 16, 6 * 16
    pool = make(64, R, 4, 8)
    if grown:
        pool.grow(ints([n] * 4))
    else:  # the same state, in a work buffer that no call has written
        pool.block_table[:, :6] = torch.arange(24, device=DEV, dtype=torch.int32).view(4, 6)
        pool.lengths.fill_(n)
        pool.refs[:24] = 1
    pool.assign(ints([-1, 1, 2, 3]))  # pages 0 .. 5 come free, 18 pages live
    page = 3 * 6 + slot if slot else 6
    b, at = (3, slot) if slot else (1, 0)
    assert int(pool.block_table[b, at]) == page and pool.status() == 0
    pool.refs[page] = 0
    others = [x for x in range(1, 4) if x != b]
    keep = {x: row_bytes(pool, x) for x in others}
    pool.compact()
    assert pool.status() == 5
    assert int(pool.block_table[b, at]) == page
    for x in others:
        assert all(torch.equal(got, want) for got, want in zip(row_bytes(pool, x), keep[x]))
    table = pool.block_table.clone()
    table[b, at] = -1
    held = torch.bincount(table[table >= 0].long(), minlength=64).int()
    assert torch.equal(held, pool.refs)  # every other entry and its count moved together


def test_pools_whose_pages_overlap_are_refused():
    K = torch.zeros((8, 2, 16, 128), dtype=torch.bfloat16, device=DEV)
    for bad in (K[:1].expand(8, -1, -1, -1), K[:0]):
        with pytest.raises(ValueError):
            mog.PagePool(bad, bad, 2, 4)


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_pool_and_its_caches_keep_their_tensors(e4m3):
    """A state tensor set anew would be read by cache() and not by grow, assign and compact."""
    pool = make(8, 16, 2, 4, e4m3=e4m3)
    for name in ("block_table", "lengths", "refs", "K", "pos"):
        with pytest.raises(AttributeError, match="fixed"):
            setattr(pool, name, getattr(pool, name))
    want = pool.cache()
    pool.K[0] = torch.zeros_like(pool.K[0])  # (the list is the caller's to change, the pool's tensors are not)
    got = pool.cache()
    assert got.K is want.K and got.V is want.V and got.block_table is pool.block_table
    if e4m3:
        for c in (got, mog.KV8(want.K, want.V, want.k_scale, want.v_scale)):
            for name in ("K", "k_scale", "batch"):
                with pytest.raises(AttributeError, match="fixed"):
                    setattr(c, name, getattr(c, name))


def test_calls_on_a_stream_of_the_cache_s_device():
    pool = make(16, 16, 2, 4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    pos, granted = pool.grow(ints([20, 3]), stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert pos.tolist() == [0, 0] and granted.tolist() == [20, 3] and pool.status(stream=s) == 0


@pytest.mark.parametrize("name", ["pos", "granted", "lengths"])
def test_grow_by_what_an_earlier_growth_returned(name):
    """n_new in the tensors that grow writes."""
    pool = make(40, 16, 3, 12)
    pool.grow(ints([5, 0, 20]))
    pool.grow(ints([1, 2, 3]))
    n, before = getattr(pool, name).tolist(), pool.lengths.tolist()
    pos, granted = pool.grow(getattr(pool, name))
    assert granted.tolist() == n and pos.tolist() == before
    assert pool.lengths.tolist() == [x + y for x, y in zip(before, n)] and pool.status() == 0
