"""Decode attention over contiguous int8 caches whose sequences, heads, rows or scales lie further apart than 32 bits count:
the same bits as over compact ones."""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import serving_mog_decode_gb300 as mog
from serving_mog_decode_gb300 import buildlib

pytestmark = pytest.mark.gpu
DEV, D = "cuda", 128


@pytest.fixture(scope="module", autouse=True)
def built():
    buildlib.build()


def spread(x, strides):
    """x in memory of its own with the given strides (what lies between is not written)."""
    at = sum((n - 1) * s for n, s in zip(x.shape, strides)) + 1
    y = torch.empty(at, dtype=x.dtype, device=DEV).as_strided(x.shape, strides)
    y.copy_(x)
    return y


@pytest.mark.parametrize("G", [1, 12])
@pytest.mark.parametrize("rows,scales", [((1 << 31, 700 * D, D, 1), (1 << 31, 22, 1)),           # sequences
                                         ((1 << 13, (1 << 31) + 256, D, 1), (11, 1 << 31, 2)),    # heads
                                         ((1 << 33, 1024, 1 << 23, 1), (1 << 20, 1 << 19, 1 << 10))])  # rows 8 MiB apart
def test_far_apart(rows, scales, G):
    B, H, n, block = (1 if rows[0] < rows[1] else 2), 2, 700, 32
    g = torch.Generator(device=DEV).manual_seed(G)
    codes = [torch.randint(-127, 128, (B, H, n, D), generator=g, device=DEV, dtype=torch.int8) for _ in range(2)]
    s = [torch.rand((B, H, -(-n // block)), generator=g, device=DEV) / 64 for _ in range(2)]
    q = torch.randn((B, H * G, D), generator=g, device=DEV).bfloat16()
    lengths = torch.tensor([n, 333][:B], dtype=torch.int32, device=DEV)
    want = mog.dense_decode(mog.KVI8(*codes, *s, block), None, lengths, n, q)
    far = mog.KVI8(*(spread(x, rows) for x in codes), *(spread(x, scales) for x in s), block)
    assert torch.equal(mog.dense_decode(far, None, lengths, n, q), want)
    # (the compact answer itself, in 64 bits)
    K, V = (x[0, 1].double() * e[0, 1].double().repeat_interleave(block)[:n, None] for x, e in zip(codes, s))
    p = torch.softmax(q[0, G:].double() @ K.T / D ** 0.5, -1)
    assert ((want[0, G:].double() - p @ V).abs() <= 2.0 ** -14 * (p @ V.abs())).all()
