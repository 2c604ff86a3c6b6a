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


@pytest.mark.parametrize("first,last", [(0, 150), (37, 210), (130, 131), (200, 333)])
@pytest.mark.parametrize("hint", [0, 200])
def test_a_part_of_a_batchs_rows(first, last, hint):
    """Tensors that hold rows first .. last - 1 of a batch: start[] moved down by
    `first`, so that sequences begin before the tensors or end behind them."""
    import numpy as np
    import torch
    from tests import pages_ref as ref
    from tests.test_gpu_pages import host
    s = Setup([(180, 130), (70, 3), (300, 200)], page=16, H=2)
    s.b.start = s.b.start - np.int32(first)
    s.batch = s.kvq.Batch(torch.from_numpy(s.b.start).cuda(), s.batch.length, s.batch.table, max_rows=hint)
    s.rows = last - first
    q = s.tensor(8, "fp16")
    s.check(q, *s.attend(q), "fp16", only=set(range(s.rows)))
    s.check(q, *s.attend(q, window=50), "fp16", only=set(range(0, s.rows, 3)), window=50)
    k, v = s.tensor(2, "fp16"), s.tensor(2, "fp16")
    s.kvq.kvq_pages_write(s.cfg, s.pages, s.batch, k, v)
    out = torch.full_like(k, 7.0)
    s.kvq.kvq_pages_read(s.cfg, s.pages, s.batch, out, None)
    assert s.kvq.kvq_pages_read_errors() == 0
    for i, x in enumerate((k, v)):
        c, t = ref.pack(host(x), s.signs)
        for r, seq, pos in s.b.rows():
            if 0 <= r < s.rows:
                p, o = s.b.slot(seq, pos, 16, s.n_pages)
                s.codes[i][p, :, o], s.tok[i][p, :, o] = c[r], t[r]
        assert np.array_equal(s.pages.codes[i].cpu().numpy(), s.codes[i])
        assert np.array_equal(s.pages.tok[i].cpu().numpy().view(np.uint16), s.tok[i].view(np.uint16))
    want = (ref.codes_of(ref.pack(host(k), s.signs)[0]) * ref.pack(host(k), s.signs)[1].astype(np.float64)[..., None]) \
        @ ref.matrix(128, s.signs)
    assert (np.abs(host(out) - want) <= (2.0 ** -11 + 3 * 2.0 ** -24) * np.abs(want) + 2.0 ** -25).all()


@pytest.mark.parametrize("hint", [0, 1, 500])
def test_rows_that_belong_to_nobody(hint):
    """A batch whose sequences have no rows leaves all tensors as they are."""
    import torch
    s = Setup([(100, 0), (0, 0), (33, 0)], lead=5, tail=7, max_rows=hint)
    q, k = s.tensor(4, "fp16"), s.tensor(2, "fp16")
    out, lse = s.attend(q)
    assert bool((out == 7).all()) and bool((lse == 7).all())
    before = [x.clone() for x in (*s.pages.codes, *(t.view(torch.int16) for t in s.pages.tok))]
    s.kvq.kvq_pages_write(s.cfg, s.pages, s.batch, k, k)
    kept = torch.full_like(k, 7.0)
    s.kvq.kvq_pages_read(s.cfg, s.pages, s.batch, kept, None)
    assert bool((kept == 7).all())
    assert all(torch.equal(a, b) for a, b in zip(before, (*s.pages.codes, *(t.view(torch.int16) for t in s.pages.tok))))


@pytest.mark.parametrize("d,G", [(128, 81), (128, 256), (64, 80), (64, 256), (128, 32), (128, 48)])
@pytest.mark.parametrize("hint", [0, 3])
def test_many_query_heads_a_kv_head(d, G, hint):
    """Up to the 256 that are allowed, and at the bounds between the kernels."""
    s = Setup([(150, 1), (40, 3), (0, 1), (300, 2)], H=1, d=d, page=32, max_rows=hint)
    q = s.tensor(G, "bf16")
    s.check(q, *s.attend(q), "bf16")
