"""The error words are read once the GPU is done with all streams, also those
that do not wait for the default stream."""
import numpy as np
import pytest

from tests.test_gpu_pages import Setup

pytestmark = pytest.mark.gpu


def busy(stream):
    """Some tens of milliseconds of ordinary work on a stream."""
    import torch
    with torch.cuda.stream(stream):
        x = torch.ones(8192, 8192, dtype=torch.bfloat16, device="cuda")
        for _ in range(40):
            y = x @ x
        return x, y


def test_pages_errors_of_a_call_that_is_still_to_run():
    import torch
    s = Setup([(200, 1), (90, 1)], page=16)
    bad = s.batch.table.clone()
    bad[0, 3] = s.n_pages
    batch = s.kvq.Batch(s.batch.start, s.batch.length, bad[:, :s.b.table.shape[1]], max_rows=1)
    q = s.tensor(4, "fp16")
    out = torch.zeros_like(q)
    ws = torch.empty(s.kvq.kvq_pages_attention_workspace_bytes(s.cfg, s.pages, batch, s.rows, 4), dtype=torch.uint8,
                     device="cuda")
    side = torch.cuda.Stream()
    busy(side)  # the library's first use is not what is waited for
    torch.cuda.synchronize()
    assert s.kvq.kvq_pages_read_errors() == 0
    keep = busy(side)
    s.kvq.kvq_pages_attention(s.cfg, s.pages, batch, q, out, ws=ws, stream=side)
    assert s.kvq.kvq_pages_read_errors(clear=False) == 4
    assert s.kvq.kvq_pages_read_errors(clear=True) == 4
    assert s.kvq.kvq_pages_read_errors() == 0
    del keep
    assert np.isfinite(out.float().cpu().numpy()).all()


@pytest.fixture()
def waitlib(monkeypatch):
    import ctypes
    from kv_cache_bit_b200 import build, kvq
    product = kvq.LIB_PATH
    kvq.LIB_PATH = build.TEST_LIB
    try:
        L = kvq._load()
    finally:
        kvq.LIB_PATH = product
    L.kvq_test_set_wait_scale.argtypes = [ctypes.c_uint32]
    monkeypatch.setattr(kvq, "lib", L)
    yield L
    L.kvq_test_set_wait_scale(1)


def test_block_cache_errors_of_a_call_that_is_still_to_run(waitlib):
    """The test build's waits give up at once: the quantizer's error bit."""
    import torch
    from kv_cache_bit_b200 import kvq
    cfg = kvq.Config(128, 4, kvq.NORM_SEP | kvq.PER_CHANNEL)
    cache = kvq.KVCache.allocate(cfg, 1, 2, 256)
    x = torch.randn(1, 2, 256, 128, device="cuda").half().view(torch.int16)
    side = torch.cuda.Stream()
    busy(side)
    torch.cuda.synchronize()
    assert kvq.kvq_read_device_errors(clear=True) == 0
    assert waitlib.kvq_test_set_wait_scale(0) == kvq.KVQ_OK
    keep = busy(side)
    kvq.kvq_quantize_block(cfg, cache, x, x, 0, 256, stream=side.cuda_stream)
    assert kvq.kvq_read_device_errors(clear=True) & 1
    assert kvq.kvq_read_device_errors() == 0
    del keep
