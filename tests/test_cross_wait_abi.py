"""Host-side refusals of the self-check of cross attention's waits: its own, and those of the call that it stands for."""
import ctypes as C

import pytest

import serving_mog_decode_gb300 as mog
from serving_mog_decode_gb300 import buildlib

P = C.c_void_p(1 << 20)
ARG, SHAPE, SMALL = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    buildlib.build()
    return mog.lib()


def test_refusals(lib):
    s3 = (C.c_int64 * 3)(1024, 1024, 128)

    def check(polls=5, t=4, n_max=1 << 20, d=128, h_q=32, q=P, nbytes=1 << 40, **kw):
        c = mog.Cache(**dict(dict(type=0, n_cap=1 << 20, k=P.value, v=P.value, stride_b=8 << 27, stride_h=1 << 27, stride_n=128), **kw))
        return lib.mog_check_cross_wait(C.byref(c), P, n_max, 2, 8, h_q, d, t, None, q, s3, P, s3, P, nbytes, polls, None)

    for kw, why in [(dict(polls=-1), ARG), (dict(t=1), ARG), (dict(t=0), ARG), (dict(n_max=0), ARG), (dict(d=64), SHAPE),
                    (dict(h_q=33), SHAPE), (dict(q=None), ARG), (dict(nbytes=16), SMALL), (dict(type=3), ARG), (dict(stride_n=64), SHAPE)]:
        assert check(**kw) == why, kw
