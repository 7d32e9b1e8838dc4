"""Cross attention on a stream of the caller's, beside work of the current one."""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import serving_mog_decode_gb300 as mog
from serving_mog_decode_gb300 import buildlib
from test_gpu_cross import D, Made, ints, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    buildlib.build()


@pytest.mark.parametrize("T", [1, 6, 300])
def test_on_another_stream(T):
    """The result of a call on another stream, read after that stream, is that of the current one, while the current one
    works on another call of the same inputs."""
    m = Made(70, (5000, 3000), 2, 64)
    q, count = randn(71, 2, T, 8, D), ints(T, max(T - 2, 1))
    want = torch.full_like(q, 2.0)
    assert mog.cross_attend(*m.cache, m.lengths, m.n_max, q, count=count, out=want) is want
    m.check(q, want, 4, count.tolist(), fill=2.0)
    s, other, mine = torch.cuda.Stream(), torch.full_like(q, 2.0), torch.full_like(q, 2.0)
    for own_scratch in (False, True):
        other.fill_(2.0)
        torch.cuda.synchronize()
        n = mog.cross_scratch_bytes(2, 2, 8, T, m.n_max)
        scratch = torch.empty(max(n, 16), dtype=torch.uint8, device=q.device) if own_scratch else None
        s.wait_stream(torch.cuda.current_stream())
        got = mog.cross_attend(*m.cache, m.lengths, m.n_max, q, count=count, out=other, scratch=scratch, stream=s)
        mog.cross_attend(*m.cache, m.lengths, m.n_max, q, count=count, out=mine)
        s.synchronize()
        assert got is other and other is not want
        assert torch.equal(other, want)
        torch.cuda.current_stream().synchronize()
        assert torch.equal(mine, want)
