"""Paged cache: what the host refuses, the plain reference's own checks, and
the binding's objects on host tensors (CPU only; every library call made here
with placeholder addresses fails a host check or has nothing to do)."""
import ctypes
import math

import numpy as np
import pytest

import oracle
from tests import pages_ref as ref

A = 1 << 20  # placeholder address, 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def kvq():
    from kv_cache_bit_b200 import build
    build.build()
    from kv_cache_bit_b200 import kvq as mod
    return mod


P2 = ctypes.c_void_p * 2


def cfg(kvq, d=128, bits=4, flags=0, reserved=0, signs=None):
    return kvq.kvq_config(d, bits, flags, reserved, signs)


def pool(kvq, n=10, h=2, d=128, t=16, codes=(A, A), tok=(A, A)):
    return kvq.kvq_pages(n, h, d, t, P2(*codes), P2(*tok))


def batch(kvq, n=2, pages=4, stride=4, rows=0, start=A, length=A, table=A):
    return kvq.kvq_batch(n, pages, stride, rows, start, length, table)


def rows(kvq, data=A, rs=256, hs=128, dt=0, reserved=0):
    return kvq.kvq_rows(data, rs, hs, dt, reserved)


def calls(kvq, c=None, p=None, b=None, x=None, n=8):
    """The statuses of write, read and attention for one set of arguments."""
    c, p, b = c or cfg(kvq), p or pool(kvq), b or batch(kvq)
    x = x or rows(kvq)
    o = kvq.kvq_rows((x.data or 0) + (1 << 30) if x.data else x.data, x.row_stride, x.head_stride, x.dtype, x.reserved)
    L = kvq.lib
    return (L.kvq_pages_write(c, p, b, x, o, n, None), L.kvq_pages_read(c, p, b, x, o, n, None),
            L.kvq_pages_attention(c, p, b, x, p.kv_heads, n, 0.0, 1, 0, o, None, None, 0, None))


def test_paged_refusals(kvq):
    INV, UNS, WS = kvq.KVQ_ERR_INVALID_ARG, kvq.KVQ_ERR_UNSUPPORTED, kvq.KVQ_ERR_WORKSPACE
    bad = [
        (dict(c=cfg(kvq, reserved=1)), INV), (dict(c=cfg(kvq, signs=A + 8)), INV),
        (dict(c=cfg(kvq, d=96)), UNS), (dict(c=cfg(kvq, bits=3)), UNS), (dict(c=cfg(kvq, bits=2)), UNS),
        (dict(c=cfg(kvq, flags=3)), UNS), (dict(c=cfg(kvq, flags=9)), UNS), (dict(c=cfg(kvq, flags=32)), UNS),
        (dict(p=pool(kvq, n=0)), INV), (dict(p=pool(kvq, h=0)), INV), (dict(p=pool(kvq, d=64)), INV),
        (dict(p=pool(kvq, t=8)), UNS), (dict(p=pool(kvq, t=48)), UNS), (dict(p=pool(kvq, t=256)), UNS),
        (dict(p=pool(kvq, codes=(A, None))), INV), (dict(p=pool(kvq, codes=(A + 8, A))), INV),
        (dict(p=pool(kvq, tok=(None, A))), INV), (dict(p=pool(kvq, tok=(A, A + 2))), INV),
        (dict(p=pool(kvq, n=1 << 24, h=8, t=16)), UNS),      # 2^31 slots
        (dict(b=batch(kvq, n=-1)), INV), (dict(b=batch(kvq, rows=-1)), INV), (dict(b=batch(kvq, pages=0)), INV),
        (dict(b=batch(kvq, pages=5, stride=4)), INV), (dict(b=batch(kvq, start=None)), INV),
        (dict(b=batch(kvq, length=A + 1)), INV), (dict(b=batch(kvq, table=None)), INV),
        (dict(b=batch(kvq, pages=1 << 27, stride=1 << 27)), UNS),
        (dict(x=rows(kvq, data=None)), INV), (dict(x=rows(kvq, data=A + 2)), INV), (dict(x=rows(kvq, reserved=1)), INV),
        (dict(x=rows(kvq, rs=260)), INV), (dict(x=rows(kvq, hs=132)), INV), (dict(x=rows(kvq, dt=3)), UNS),
        (dict(x=rows(kvq, rs=1 << 40)), INV), (dict(n=-1), INV), (dict(n=1 << 40), UNS),
    ]
    for kw, want in bad:
        assert calls(kvq, **kw) == (want,) * 3, kw
    L, c, p, b, x = kvq.lib, cfg(kvq), pool(kvq), batch(kvq), rows(kvq)
    far = rows(kvq, data=A + (1 << 30))
    for args in ((None, p, b), (c, None, b), (c, p, None)):
        assert L.kvq_pages_write(*args, x, x, 8, None) == INV
    assert L.kvq_pages_write(c, p, b, None, x, 8, None) == INV
    assert L.kvq_pages_write(c, p, b, x, rows(kvq, dt=1), 8, None) == INV            # K and V of two types
    assert L.kvq_pages_write(c, p, b, rows(kvq, dt=2), rows(kvq, dt=2), 8, None) == UNS  # fp32 inputs
    # outputs: at least one, of one type, no two elements in one place
    assert L.kvq_pages_read(c, p, b, None, None, 8, None) == INV
    assert L.kvq_pages_read(c, p, b, x, rows(kvq, data=A + (1 << 30), dt=2), 8, None) == INV
    assert L.kvq_pages_read(c, p, b, x, x, 8, None) == INV
    for rs, hs in ((0, 128), (256, 0), (-256, 128), (256, -128), (128, 128), (64, 1024)):
        assert L.kvq_pages_read(c, p, b, rows(kvq, rs=rs, hs=hs), None, 8, None) == INV, (rs, hs)
    # attention
    at = lambda q=x, heads=2, n=8, scale=0.0, causal=1, window=0, out=far, lse=None, ws=None, size=0: \
        L.kvq_pages_attention(c, p, b, q, heads, n, scale, causal, window, out, lse, ws, size, None)  # noqa: E731
    assert at() == WS
    assert at(heads=3) == INV and at(heads=1) == INV and at(heads=0) == INV
    assert at(heads=2 * 257, q=rows(kvq, rs=2 * 257 * 128), out=rows(kvq, A + (1 << 30), rs=2 * 257 * 128)) == UNS
    assert at(window=-1) == INV and at(causal=0, window=5) == INV
    assert at(scale=float("inf")) == INV and at(scale=float("nan")) == INV
    assert at(out=rows(kvq, A + (1 << 30), dt=1)) == INV and at(q=rows(kvq, dt=2), out=rows(kvq, A + (1 << 30), dt=2)) == UNS
    assert at(out=x) == INV and at(out=rows(kvq, A + 16)) == INV                      # overlaps the queries
    assert at(lse=A + 2) == INV
    need = L.kvq_pages_attention_workspace_bytes(c, p, b, 8, 2)
    assert need > 0 and at(ws=A + 4, size=need) == WS and at(ws=A, size=need - 1) == WS
    assert L.kvq_pages_attention_workspace_bytes(c, p, b, 8, 3) == 0
    assert L.kvq_pages_attention_workspace_bytes(cfg(kvq, bits=3), p, b, 8, 2) == 0
    assert L.kvq_pages_read_errors(None, 0) == INV


def test_paged_calls_without_rows_or_sequences_do_nothing(kvq):
    assert calls(kvq, n=0) == (0, 0, 0)
    assert calls(kvq, b=batch(kvq, n=0, pages=0, stride=0, start=None, length=None, table=None)) == (0, 0, 0)


def test_binding_objects_on_host_tensors(kvq):
    import torch
    c = kvq.Config(64, 4, kvq.HADAMARD, None, device="cpu")
    p = kvq.PagedCache.allocate(c, 5, 2, 32, device="cpu")
    assert p.nbytes() == 2 * 5 * 2 * 32 * (32 + 2)
    for t in (*p.codes, *p.tok):
        t.copy_(torch.randint(0, 100, t.shape).to(t.dtype))
    snap = p.snapshot()
    o = kvq.PagedCache.allocate(c, 5, 2, 32, device="cpu")
    o.restore(snap)
    assert all(torch.equal(a, b) for a, b in zip((*p.codes, *p.tok), (*o.codes, *o.tok)))
    for other in (kvq.PagedCache.allocate(c, 4, 2, 32, device="cpu"), kvq.PagedCache.allocate(c, 5, 2, 16, device="cpu")):
        with pytest.raises(kvq.KvqError):
            other.restore(snap)
    for args in ((c, 5, 2, 24), (kvq.Config(64, 3, 0, None, device="cpu"), 5, 2, 32),
                 (kvq.Config(96, 4, 0, None, device="cpu"), 5, 2, 32)):
        with pytest.raises(kvq.KvqError):
            kvq.PagedCache.allocate(*args, device="cpu")
    with pytest.raises(kvq.KvqError):
        kvq.PagedCache.wrap(c, p.codes, [p.tok[0], p.tok[1][:4]])
    with pytest.raises(kvq.KvqError):
        kvq.PagedCache.wrap(c, [p.codes[0], p.codes[1].transpose(0, 1)], p.tok)
    i = lambda *x: torch.zeros(x, dtype=torch.int32)  # noqa: E731
    b = kvq.Batch(i(4), i(3), i(3, 20)[:, :7], max_rows=2)
    assert (b.c.n_seqs, b.c.max_pages, b.c.table_stride, b.c.max_rows) == (3, 7, 20, 2)
    for args in ((i(3), i(3), i(3, 7)), (i(4), i(3), i(2, 7)), (i(4), i(3), i(7, 3).t()), (i(4).long(), i(3), i(3, 7))):
        with pytest.raises(kvq.KvqError):
            kvq.Batch(*args)
    x = torch.zeros(6, 2, 64, dtype=torch.float16)
    for k in (x[:, :1], x[..., :32], torch.zeros(6, 2, 128, dtype=torch.float16)[..., ::2], x[0], x[:5]):
        with pytest.raises(kvq.KvqError):
            kvq.kvq_pages_write(c, p, b, k, x)
    with pytest.raises(kvq.KvqError):
        kvq.kvq_pages_attention(c, p, b, x, x.clone(), torch.zeros(6, 2, dtype=torch.float64), ws=x)
    with pytest.raises(kvq.KvqError):
        kvq.kvq_pages_attention(c, p, b, x, x[:, :1], ws=x)


# ------------------------------------------------------------ the reference

@pytest.mark.parametrize("d", [64, 128])
def test_reference_rotation_is_orthogonal_and_agrees_with_the_butterflies(d):
    signs = oracle.make_signs(3, d)
    R = ref.matrix(d, signs)
    assert np.allclose(R @ R.T, np.eye(d), atol=1e-13)
    x = np.random.default_rng(0).standard_normal((5, d))
    assert np.allclose(ref.butterflies(x * signs) / math.sqrt(d), x @ R.T, atol=1e-13)


@pytest.mark.parametrize("rotated", [False, True])
def test_reference_codes_lie_on_the_nearest_grid_point(rotated):
    d = 128
    signs = oracle.make_signs(5, d) if rotated else None
    x = np.random.default_rng(1).standard_normal((40, d)).astype(np.float16).astype(np.float32)
    x[3] = 0
    codes, sigma = ref.pack(x, signs)
    back = (ref.codes_of(codes) * sigma.astype(np.float64)[:, None]) @ ref.matrix(d, signs)
    # half a step of the grid in each rotated channel, and the scale's own rounding at the ends
    bound = sigma.astype(np.float64) * (0.5 + 7 * 2.0 ** -11) + 1e-5
    assert (np.abs((back - x) @ ref.matrix(d, signs).T).max(-1) <= bound).all()
    assert (codes[3] == 0x88).all() and sigma[3] == 0


def test_reference_codes_agree_with_the_naive_mode_of_the_oracle():
    d = 128
    x = np.random.default_rng(2).standard_normal((1, 1, 128, d)).astype(np.float16)
    c = oracle.quantize(oracle.Cfg(d=d, bits=4, flags=0, signs=None), x.view(np.uint16))
    codes, sigma = ref.pack(x[0, 0].astype(np.float32), None)
    assert np.array_equal(c["codes"][0, 0], codes)
    assert np.array_equal(c["tok"].reshape(-1), sigma.view(np.uint16))


def test_reference_attention_agrees_with_the_oracle_on_one_sequence():
    d, H, G, n = 64, 2, 3, 41
    r = np.random.default_rng(3)
    K, V = (r.standard_normal((n, H, d)).astype(np.float32) for _ in range(2))
    q = r.standard_normal((1, H * G, d)).astype(np.float16)
    k, v = ref.pack(K, None), ref.pack(V, None)
    pages = [(c.reshape(n, H, 1, -1).astype(np.uint8), t.reshape(n, H, 1)) for c, t in (k, v)]
    b = ref.Seqs(np.array([0, 1]), np.array([n]), np.arange(n)[None])
    out, lse, _, _ = ref.attention(*pages, b, q.astype(np.float64), None, 0.0, True, 0, 0.0)[0]
    kh, vh = (np.ascontiguousarray((ref.codes_of(c) * t.astype(np.float64)[..., None]).transpose(1, 0, 2), np.float32)
              for c, t in (k, v))
    want = oracle.attention(q.view(np.uint16), kh[None], vh[None])
    assert np.abs(out - np.asarray(want).reshape(H * G, d)).max() < 1e-5
