"""Paged cache: what the sources and the host checks have to keep to (CPU only;
every library call made here with placeholder addresses fails a host check or
has nothing to do)."""
import ctypes
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "kv_cache_bit_b200", "csrc")


def test_register_split_is_one_instruction_a_warpgroup():
    """PTX: all warps of a warpgroup execute the same setmaxnreg.  The many-row
    kernel's warps 12, 13 and 14, 15 have different roles and are one
    warpgroup, so the instruction stands ahead of the roles, once for each
    direction, under a condition on whole warpgroups."""
    with open(os.path.join(CSRC, "kvq_pages_tile.cuh")) as f:
        text = f.read()
    assert re.findall(r"setmaxnreg\.(inc|dec)", text) == ["inc", "dec"]
    split = re.search(r"if \(works\) \{\s*if \(warp < (\d+)\) asm volatile\(\"setmaxnreg\.inc[^;]*;\" ::\"n\"\(kSoftmaxRegs\)\);"
                      r"\s*else asm volatile\(\"setmaxnreg\.dec[^;]*;\" ::\"n\"\(kProducerRegs\)\);\s*\}", text)
    assert split and int(split.group(1)) % 4 == 0
    assert split.end() < text.index("warp >= 14")


A = 1 << 20  # placeholder address, 16-byte aligned, never dereferenced
P2 = ctypes.c_void_p * 2


@pytest.fixture(scope="module")
def kvq():
    from kv_cache_bit_b200 import build
    build.build()
    from kv_cache_bit_b200 import kvq as mod
    return mod


class Call:
    """Arguments of the paged calls: with `n_seqs` 0 write and read pass all
    checks and do nothing, attention without a workspace ends at that check."""

    def __init__(self, kvq, d=128, heads=2, page=16, pages=4, n_seqs=0):
        self.kvq, self.L, self.heads = kvq, kvq.lib, heads
        self.cfg = kvq.kvq_config(d, 4, 0, 0, None)
        self.pool = kvq.kvq_pages(10, heads, d, page, P2(A, A), P2(A, A))
        self.batch = kvq.kvq_batch(n_seqs, pages, pages, 0, A, A, A)

    def x(self, rs, hs, data=A, dt=0):
        return self.kvq.kvq_rows(data, rs, hs, dt, 0)

    def write(self, k, v, rows):
        return self.L.kvq_pages_write(self.cfg, self.pool, self.batch, k, v, rows, None)

    def read(self, k, v, rows):
        return self.L.kvq_pages_read(self.cfg, self.pool, self.batch, k, v, rows, None)

    def attend(self, q, out, rows, heads=None):
        return self.L.kvq_pages_attention(self.cfg, self.pool, self.batch, q, heads or self.heads, rows, 0.0, 1, 0,
                                          out, None, None, 0, None)


@pytest.mark.parametrize("heads", [1, 3, 8, 28])
def test_row_limits_are_the_documented_ones(kvq, heads):
    """rows * kv_heads < 2^29 of a write and a read, rows * q_heads < 2^31 and
    80 * n_seqs * q_heads < 2^31 of an attention call; both sides of each."""
    OK, UNS, WS = kvq.KVQ_OK, kvq.KVQ_ERR_UNSUPPORTED, kvq.KVQ_ERR_WORKSPACE
    c = Call(kvq, heads=heads)
    x, y = c.x(heads * 128, 128), c.x(heads * 128, 128, data=A + (1 << 44))
    last = (2 ** 29 - 1) // heads
    assert (c.write(x, y, last), c.write(x, y, last + 1)) == (OK, UNS)
    assert (c.read(x, y, last), c.read(x, y, last + 1)) == (OK, UNS)
    last = (2 ** 31 - 1) // heads
    assert (c.attend(x, y, last), c.attend(x, y, last + 1)) == (OK, UNS)
    last = (2 ** 31 - 1) // (80 * heads)
    assert (Call(kvq, heads=heads, n_seqs=last).attend(x, y, 8), Call(kvq, heads=heads, n_seqs=last + 1).attend(x, y, 8)) == (WS, UNS)
    assert c.write(x, y, 1 << 62) == UNS and c.attend(x, y, 1 << 62) == UNS


def test_strides_are_limited_by_where_they_reach(kvq):
    """A head-major tensor of 2^20 rows and more is an ordinary one; from 2^42
    bytes between its first and its last element on a tensor is refused."""
    OK, INV = kvq.KVQ_OK, kvq.KVQ_ERR_INVALID_ARG
    c = Call(kvq, heads=8)
    for rows in (1 << 20, (1 << 20) + 1, 1 << 25):
        x, y = c.x(128, rows * 128), c.x(128, rows * 128, data=A + (1 << 44))
        assert (c.write(x, y, rows), c.read(x, y, rows), c.attend(x, y, rows)) == (OK, OK, OK), rows
    most = 1 << 41  # elements of 2 bytes
    for rs, hs, rows, over in (((most - 128) // 8, 0, 9, 0), ((most - 128 + 64) // 8, 0, 9, 1), (0, (most - 128) // 56 * 8, 5, 0),
                               (0, (most - 128) // 56 * 8 + 8, 5, 1), (-((most - 128) // 8), 0, 9, 0), (1 << 62, 0, 2, 1),
                               (-(1 << 62), 0, 2, 1), (0, 1 << 62, 2, 1), (1 << 40, 0, (1 << 29) // 8 - 1, 1),
                               (1 << 62, 128, 1, 0), (most // 2, most // 14 // 8 * 8, 2, 1)):
        x = c.x(rs // 8 * 8, hs)
        assert c.write(x, x, rows) == (INV if over else OK), (rs, hs, rows)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_a_table_leaves_room_to_round_its_last_token_up(kvq, page):
    """Tokens are counted in 32 bits and rounded up to whole units of 32 or 64:
    a table may not reach the last of them."""
    UNS, WS = kvq.KVQ_ERR_UNSUPPORTED, kvq.KVQ_ERR_WORKSPACE
    most = (2 ** 31 - 256) // page
    for pages, want in ((most, WS), (most + 1, UNS), ((2 ** 31 - 1) // page, UNS)):
        c = Call(kvq, page=page, pages=pages, n_seqs=2)
        x, y = c.x(256, 128), c.x(256, 128, data=A + (1 << 30))
        assert c.attend(x, y, 8) == want, pages
        if want == UNS:
            assert c.write(x, y, 8) == UNS and c.read(x, y, 8) == UNS
    assert (most * page + 63) < 2 ** 31


def test_queries_and_outputs_may_be_slices_of_one_buffer(kvq):
    """Refused are outputs that share an element with the queries, by counting
    all elements of small tensors; interleaved slices are not."""
    INV, WS = kvq.KVQ_ERR_INVALID_ARG, kvq.KVQ_ERR_WORKSPACE
    d, seen = 64, set()
    for heads in (1, 2, 3):
        c = Call(kvq, d=d, heads=heads, n_seqs=2)
        for rows in (1, 2, 4):
            wide = heads * d
            for rs, hs in ((wide, d), (2 * wide, d), (2 * wide, 2 * d), (2 * wide + 64, d), (d, rows * d), (2 * d, 2 * rows * d),
                           (d, 2 * rows * d), (3 * wide, 3 * d)):
                for off in [8 * k * s for k in (1, 3, 7, 8, 9, 16, 24, 40) for s in (1, -1)] + [wide, -wide, rows * d, 2 * wide + 56]:
                    if off % 8:
                        continue
                    other = {r * rs + h * hs + off + e for r in range(rows) for h in range(heads) for e in range(0, d, 8)}
                    full = {r * rs + h * hs + e for r in range(rows) for h in range(heads) for e in range(0, d, 8)}
                    got = c.attend(c.x(rs, hs), c.x(rs, hs, data=A + 2 * off), rows)
                    assert got == (INV if other & full else WS), (heads, rows, rs, hs, off)
                    seen.add((got, rows > 1 and heads > 1))
    assert len(seen) == 4
    c = Call(kvq, d=d, heads=2, n_seqs=2)
    assert c.attend(c.x(128, 64), c.x(256, 64, data=A + 128), 8) == INV   # other strides: by extent
    assert c.attend(c.x(0, 64), c.x(128, 64, data=A + (1 << 20)), 8) == WS


def test_read_outputs_that_share_elements_are_refused(kvq):
    """A K output that begins inside the V output: what it holds afterwards
    would be a race."""
    INV = kvq.KVQ_ERR_INVALID_ARG
    c = Call(kvq, d=64, heads=2, n_seqs=2)
    for rs, hs, off in ((128, 64, 64), (128, 64, -8 * 64), (256, 64, 64), (256, 128, 128), (64, 8 * 64, 8 * 64 - 64)):
        assert c.read(c.x(rs, hs), c.x(rs, hs, data=A + 2 * off), 8) == INV, (rs, hs, off)


def test_binding_refuses_missing_tensors_and_caches_on_the_host(kvq):
    import torch
    c = kvq.Config(64, 4, 0, None, device="cpu")
    p = kvq.PagedCache.allocate(c, 5, 2, 32, device="cpu")
    i = lambda *x: torch.zeros(x, dtype=torch.int32)  # noqa: E731
    b = kvq.Batch(i(3), i(2), i(2, 4))
    x, ws = torch.zeros(6, 2, 64, dtype=torch.float16), torch.zeros(64, dtype=torch.uint8)
    for call in (lambda: kvq.kvq_pages_write(c, p, b, None, None), lambda: kvq.kvq_pages_write(c, p, b, x, None),
                 lambda: kvq.kvq_pages_read(c, p, b, None, None), lambda: kvq.kvq_pages_attention(c, p, b, None, x, ws=ws),
                 lambda: kvq.kvq_pages_attention(c, p, b, x, None, ws=ws), lambda: kvq.kvq_pages_write(c, p, b, x, x),
                 lambda: kvq.kvq_pages_read(c, p, b, x, None),
                 lambda: kvq.kvq_pages_attention(c, p, b, x, x.clone(), ws=ws)):
        with pytest.raises(kvq.KvqError) as e:
            call()
        assert e.value.status == kvq.KVQ_ERR_INVALID_ARG


def test_one_source_is_one_program():
    """nvcc's split compilation shares registers out by chance: the same source
    built twice had kernels of 138 and 168 registers."""
    from kv_cache_bit_b200 import build
    assert not any("split-compile" in flag for flag in build._FLAGS)
