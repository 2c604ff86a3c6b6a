"""Paged cache on the GPU: tensors that are slices of one buffer."""
import pytest

from tests.test_gpu_pages import Setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [3, 90])
def test_attention_into_another_slice_of_the_queries_buffer(rows):
    import torch
    s = Setup([(200, rows), (90, 1)], page=16)
    q = s.tensor(4, "fp16")
    want, _ = s.attend(q)
    ws = torch.empty(s.kvq.kvq_pages_attention_workspace_bytes(s.cfg, s.pages, s.batch, s.rows, 4), dtype=torch.uint8,
                     device="cuda")
    wide, deep = (torch.full(shape, 7.0, dtype=torch.float16, device="cuda")
                  for shape in ((s.rows, 8, 128), (s.rows, 4, 2, 128)))
    for x, y in ((wide[:, :4], wide[:, 4:]), (deep[:, :, 1], deep[:, :, 0])):
        x.copy_(q)
        s.kvq.kvq_pages_attention(s.cfg, s.pages, s.batch, x, y, ws=ws)
        assert torch.equal(y, want) and torch.equal(x, q)
    with pytest.raises(s.kvq.KvqError):
        s.kvq.kvq_pages_attention(s.cfg, s.pages, s.batch, wide[:, :4], wide[:, 3:7], ws=ws)
