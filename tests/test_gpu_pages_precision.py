"""Paged attention on the GPU to within the averages that its roundings leave
(tests/pages_precision.py): long ranges of tokens, equal weights, ordinary
batches of few and of many rows."""
import numpy as np
import pytest

from tests import pages_precision as prec
from tests import pages_ref as ref
from tests.test_gpu_pages import Setup, host

pytestmark = pytest.mark.gpu


def shared(n_seqs, tokens, G, d, rotated, page, sharp, ragged=False):
    """One stored sequence that all sequences of a batch share, a query row each:
    (setup, q, out, lse, exact out, exact lse)."""
    import torch
    s = Setup([(tokens, 1)], d=d, H=1, page=page, rotated=rotated)
    k, v = prec.stored(s, 0, tokens)
    length = np.full(n_seqs, tokens, np.int32)
    if ragged:
        length = s.rng.integers(1, tokens + 1, n_seqs).astype(np.int32)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    s.batch = s.kvq.Batch(dev(np.arange(n_seqs + 1, dtype=np.int32)), dev(length),
                          s.batch.table.repeat(n_seqs, 1).contiguous(), max_rows=1)
    s.rows = n_seqs
    q = s.tensor(G, "fp16", scale=sharp)
    out, lse = s.attend(q)
    assert s.kvq.kvq_pages_read_errors() == 0
    return s, q, out, lse, prec.exact(q, k, v, s.signs, length.astype(np.int64) - 1, length.astype(np.int64))


@pytest.mark.parametrize("d,G,rotated,page", [(128, 4, True, 16), (128, 8, False, 64), (128, 12, True, 32),
                                              (64, 2, True, 128), (64, 16, False, 16)])
def test_nearly_equal_weights_over_thousands_of_tokens_a_warp(d, G, rotated, page):
    """1040 sequences of 8192 tokens and one kv head are some 4800 tokens a warp
    of the generation-step kernel, in one sum: what the sum rounds must not grow
    with its length, in any channel."""
    s, q, out, lse, (want, want_lse) = shared(1040, 8192, G, d, rotated, page, 0.1)
    assert not prec.faults(out, lse, want, want_lse, "fp16")
    # All rows have nearly the same output, the values' mean, so that a channel's may be far from the rms of all.
    # Of the two roundings the weights' is 2^-11 / sqrt 3 of the rms of all channels (values of one size), the
    # output's 2^-11 / sqrt 3 of the channel's own: together 2^-11 sqrt((rms^2 + rms_c^2) / 3); / 2 is allowed,
    # which is the limit of all channels where rms_c = rms.
    err, size = (out.double() - want).square().mean((0, 1)), want.square().mean((0, 1))
    assert bool((err.sqrt() <= prec.LIMITS["fp16"][0] * ((size.mean() + size) / 2).sqrt()).all())


@pytest.mark.parametrize("d,G,rotated,page", [(128, 4, True, 16), (64, 8, False, 32), (128, 16, False, 128)])
def test_many_units_a_warp_of_ragged_sequences(d, G, rotated, page):
    """Segments of more than 32 units, whose pages a warp looks up 32 at a time,
    beginning anywhere in a sequence."""
    s, q, out, lse, want = shared(900, 6000, G, d, rotated, page, 1.0, ragged=True)
    assert not prec.faults(out, lse, *want, "fp16")


@pytest.mark.parametrize("d,G,dtype,rotated", [(128, 4, "fp16", True), (128, 4, "bf16", True), (128, 7, "fp16", False),
                                               (64, 1, "fp16", True), (64, 8, "bf16", False)])
@pytest.mark.parametrize("rows", [1, 5, 300])
def test_ordinary_batches(d, G, dtype, rotated, rows):
    import torch
    H = 2
    s = Setup([(2300, rows), (700, rows), (1111, rows)], d=d, H=H, page=16, rotated=rotated)
    q = s.tensor(H * G, dtype, scale=1.5)
    out, lse = s.attend(q)
    assert s.kvq.kvq_pages_read_errors() == 0
    want, want_lse = torch.empty(q.shape, dtype=torch.float64, device="cuda"), \
        torch.empty(q.shape[:2], dtype=torch.float64, device="cuda")
    for i, (n, m) in enumerate(s.counts):
        at = slice(int(s.b.start[i]), int(s.b.start[i + 1]))
        want[at], want_lse[at] = prec.exact(q[at], *prec.stored(s, i, n), s.signs, np.arange(n - m, n), np.full(m, n))
    assert not prec.faults(out, lse, want, want_lse, dtype)

@pytest.mark.parametrize("d,G,rotated,dtype", [(128, 16, True, "fp16"), (64, 16, False, "fp16"), (128, 33, False, "bf16")])
def test_nearly_equal_weights_of_many_rows_over_thousands_of_tokens(d, G, rotated, dtype):
    """The same for the many-row kernel: 160 sequences of 10 rows are more than
    8192 tokens a CTA."""
    import torch
    n, m, tokens = 160, 10, 8192
    s = Setup([(tokens, 1)], d=d, H=1, page=64, rotated=rotated)
    k, v = prec.stored(s, 0, tokens)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    s.batch = s.kvq.Batch(dev(np.arange(n + 1, dtype=np.int32) * m), dev(np.full(n, tokens, np.int32)),
                          s.batch.table.repeat(n, 1).contiguous(), max_rows=m)
    s.rows = n * m
    q = s.tensor(G, dtype, scale=0.1)
    out, lse = s.attend(q)
    assert s.kvq.kvq_pages_read_errors() == 0
    want = prec.exact(q, k, v, s.signs, np.tile(np.arange(tokens - m, tokens), n), np.full(n * m, tokens))
    assert not prec.faults(out, lse, *want, dtype)


@pytest.mark.parametrize("n,H,tokens", [(64, 2, 500), (65, 2, 500), (200, 1, 512), (222, 2, 100), (400, 1, 33)])
def test_many_short_sequences(n, H, tokens):
    """Caches that CTAs take whole, for so many sequences that a block finds its
    own by a search; some of them empty."""
    import torch
    counts = [((i * 37) % (tokens + 1), 1) for i in range(n - 1)] + [(tokens, 1)]
    s = Setup(counts, H=H, d=64, page=16, max_rows=1)
    q = s.tensor(2 * H, "fp16")
    out, lse = s.attend(q)
    rows = {0, 1, n // 2, n - 2, n - 1} | {int(r) for r in s.rng.integers(0, n, 40)}
    s.check(q, out, lse, "fp16", only=rows)
    empty = torch.tensor([c == 0 for c, _ in counts], device="cuda")
    assert not out[empty].any() and bool(torch.isneginf(lse[empty]).all()) and bool(torch.isfinite(lse[~empty]).all())


def values_of(s, mags, keep=None):
    """New stored values of the setup's only sequence, of magnitudes mags
    [tokens]; `keep`: tokens whose values stay."""
    import torch
    n = len(mags)
    x = (s.rng.standard_normal((n, s.H, s.d)) * mags[:, None, None]).astype(np.float32)
    c, t = ref.pack(x, s.signs)
    for k in range(n):
        if keep is None or k >= keep:
            p, o = s.b.slot(0, k, s.page, s.n_pages)
            s.codes[1][p, :, o], s.tok[1][p, :, o] = c[k], t[k]
    s.pages.codes[1].copy_(torch.from_numpy(s.codes[1]))
    s.pages.tok[1].copy_(torch.from_numpy(s.tok[1]))


@pytest.mark.parametrize("rotated", [False, True])
@pytest.mark.parametrize("silent", [1e-3, 1e-4, 1e-5])
@pytest.mark.parametrize("d,G,window", [(128, 4, 0), (64, 8, 0), (128, 1, 20)])
def test_loud_values_that_a_row_does_not_see(d, G, window, silent, rotated):
    """A prompt whose first tokens of every 64 have small values and whose later
    ones have huge ones: rows that see only small ones are as exact as rows
    without the huge ones behind them."""
    n = 300
    s = Setup([(n, n)], d=d, H=1, page=16, rotated=rotated)
    mags = np.where(np.arange(n) % 64 < 40, silent, 2e4)
    values_of(s, mags)
    q = s.tensor(G, "fp16")
    quiet = {r for r in range(n) if mags[max(0, r - window + 1) if window else 0:r + 1].max() == silent}
    assert len(quiet) >= 40
    out, lse = s.attend(q, window=window)
    s.check(q, out, lse, "fp16", window=window, many=True)
    k, v = prec.stored(s, 0, n)
    want, _ = prec.exact(q, k, v, s.signs, np.arange(n), np.full(n, n), window=window)
    rows = sorted(quiet)
    # the weights' rounding, the output's, and half a step of fp16's smallest numbers
    off = (out.double() - want)[rows].square().mean(-1).sqrt()
    assert bool((off <= prec.LIMITS["fp16"][1] * want[rows].square().mean(-1).sqrt() + 2.0 ** -25).all())


@pytest.mark.parametrize("d,G,rotated", [(128, 4, True), (64, 8, False), (128, 1, False)])
def test_a_row_does_not_depend_on_later_tokens(d, G, rotated):
    """The same bits for the first rows of a prompt whatever K and V the tokens
    behind them have."""
    import torch
    n, first = 300, 75
    s = Setup([(n, n)], d=d, H=1, page=16, rotated=rotated)
    q = s.tensor(G, "fp16")
    got = []
    for loud in (1.0, 1e-4, 3e4):
        values_of(s, np.full(n, loud), keep=first)
        for k in range(first, n):
            p, o = s.b.slot(0, k, s.page, s.n_pages)
            s.codes[0][p, :, o] = s.rng.integers(16, 256, (s.H, d // 2))
            s.tok[0][p, :, o] = np.float16(loud)
        s.pages.codes[0].copy_(torch.from_numpy(s.codes[0]))
        s.pages.tok[0].copy_(torch.from_numpy(s.tok[0]))
        got.append(s.attend(q))
    for out, lse in got[1:]:
        assert torch.equal(out[:first], got[0][0][:first]) and torch.equal(lse[:first], got[0][1][:first])
