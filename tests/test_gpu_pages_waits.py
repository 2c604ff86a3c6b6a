"""The paged attention's give-up path, on the GPU, without a fault or a hang:
the test build's poll limits set to 0 make every barrier wait of the tile
kernel give up at once.  It sets the error bit and returns; with the limits
back the same call gives the reference's results and sets no bit."""
import ctypes
import os

import pytest

from tests.test_gpu_pages import Setup

pytestmark = pytest.mark.gpu

ERR_BARRIER = 2


@pytest.fixture()
def waitlib(monkeypatch):
    from kv_cache_bit_b200 import build, kvq
    assert os.path.exists(build.TEST_LIB), "the test build libkvq_waittest.so is missing (run the build)"
    product = kvq.LIB_PATH
    kvq.LIB_PATH = build.TEST_LIB
    try:
        L = kvq._load()
    finally:
        kvq.LIB_PATH = product
    L.kvq_test_set_pages_wait_scale.restype = ctypes.c_int
    L.kvq_test_set_pages_wait_scale.argtypes = [ctypes.c_uint32]
    monkeypatch.setattr(kvq, "lib", L)
    kvq.kvq_pages_read_errors(clear=True)
    yield L
    L.kvq_test_set_pages_wait_scale(1)


@pytest.mark.parametrize("d,rotated", [(128, True), (64, False)])
def test_paged_attention_gives_up_and_recovers(waitlib, d, rotated):
    from kv_cache_bit_b200 import kvq
    s = Setup([(300, 200), (150, 1)], d=d, H=2, page=32, rotated=rotated)
    q = s.tensor(8, "fp16")
    assert waitlib.kvq_test_set_pages_wait_scale(0) == kvq.KVQ_OK
    s.attend(q)
    assert kvq.kvq_pages_read_errors(clear=True) == ERR_BARRIER
    assert waitlib.kvq_test_set_pages_wait_scale(1) == kvq.KVQ_OK
    s.check(q, *s.attend(q), "fp16", only={0, 1, 77, 199, 200})
