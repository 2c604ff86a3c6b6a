"""Paged 4-bit cache on the GPU against the plain numpy reference: stored bits
exactly, values read back and attention within the bounds that their
roundings allow (tests/pages_ref.py)."""
import numpy as np
import pytest

from tests import pages_ref as ref

pytestmark = pytest.mark.gpu

HALF = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


def tt(name):
    import torch
    return {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}[name]


def host(x):
    return x.float().cpu().numpy()


class Setup:
    """A pool, ragged sequences in shuffled pages and their batch.  counts:
    (tokens, rows) of each sequence; lead and tail rows belong to nobody."""

    def __init__(self, counts, H=2, d=128, page=16, rotated=True, signs="random", lead=0, tail=0, seed=0, spare=2,
                 stride=3, max_rows=0, fill=True):
        import torch
        from kv_cache_bit_b200 import kvq
        self.kvq, self.rng = kvq, np.random.default_rng(seed)
        self.H, self.d, self.page, self.counts = H, d, page, counts
        self.signs = None
        if rotated:
            self.signs = kvq.kvq_make_signs(seed + 9, d) if signs == "random" else np.ones(d, np.int8)
        self.cfg = kvq.Config(d, 4, kvq.HADAMARD if rotated else 0,
                              self.signs if rotated and signs == "random" else None)
        n = len(counts)
        need = [-(-max(c, 0) // page) for c, _ in counts]
        self.n_pages = max(sum(need) + spare, 1)
        order = self.rng.permutation(self.n_pages)
        wide = max(need + [1])
        table = np.full((n, wide), 2 ** 31 - 1, np.int32)  # entries no token reaches may hold anything
        at = 0
        for s, m in enumerate(need):
            table[s, :m] = order[at:at + m]
            at += m
        start = lead + np.concatenate(([0], np.cumsum([r for _, r in counts]))).astype(np.int32)
        self.rows = int(start[-1]) + tail
        self.b = ref.Seqs(start, np.array([c for c, _ in counts], np.int32), table)
        self.codes = [self.rng.integers(0, 256, (self.n_pages, H, page, d // 2), np.uint8) for _ in range(2)]
        self.tok = [self.rng.integers(0, 65536, (self.n_pages, H, page)).astype(np.uint16).view(np.float16)
                    for _ in range(2)]  # slots that hold nothing: any bits, NaN and infinities among them
        if fill:
            for i in range(2):
                x = (self.rng.standard_normal((sum(c for c, _ in counts if c > 0), H, d)) *
                     np.exp(0.5 * self.rng.standard_normal((1, H, 1)))).astype(np.float32)
                c, t = ref.pack(x.astype(np.float16).astype(np.float32), self.signs)
                k = 0
                for s, (m, _) in enumerate(counts):
                    for tk in range(max(m, 0)):
                        p, o = self.b.slot(s, tk, page, self.n_pages)
                        self.codes[i][p, :, o], self.tok[i][p, :, o] = c[k], t[k]
                        k += 1
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.pages = kvq.PagedCache.wrap(self.cfg, [dev(c) for c in self.codes], [dev(t) for t in self.tok])
        wide_table = torch.full((n, wide + stride), -7, dtype=torch.int32, device="cuda")
        wide_table[:, :wide] = dev(table)
        self.batch = kvq.Batch(dev(start), dev(self.b.length), wide_table[:, :wide], max_rows=max_rows)

    def tensor(self, heads, dtype, fused=0, scale=1.0):
        """Random [rows, heads, d] values; fused > 0: a slice of a wider row."""
        import torch
        x = torch.from_numpy((scale * self.rng.standard_normal((self.rows, heads + fused, self.d))).astype(np.float32))
        return x.cuda().to(tt(dtype))[:, fused:]

    def attend(self, q, lse=True, **kw):
        """(out, lse) with rows of nobody preset to 7."""
        import torch
        kvq = self.kvq
        out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
        l = torch.full(q.shape[:2], 7.0, dtype=torch.float32, device="cuda") if lse else None
        need = kvq.kvq_pages_attention_workspace_bytes(self.cfg, self.pages, self.batch, q.shape[0], q.shape[1])
        ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # NaN wherever it is read unwritten
        kvq.kvq_pages_attention(self.cfg, self.pages, self.batch, q, out, l, ws=ws, **kw)
        torch.cuda.synchronize()
        return out, l

    def check(self, q, out, lse, dtype, scale=0.0, causal=True, window=0, only=None, many=False):
        want = ref.attention((self.codes[0], self.tok[0]), (self.codes[1], self.tok[1]), self.b, host(q), self.signs,
                             scale, causal, window, HALF[dtype], only, many)
        out, l = host(out), None if lse is None else lse.cpu().numpy()
        assert np.isfinite(out).all()
        for r in range(q.shape[0]) if only is None else sorted(only):
            if r not in want:
                assert (out[r] == 7).all() and (l is None or (l[r] == 7).all()), f"row {r} belongs to nobody"
                continue
            o, ls, tol, ltol = want[r]
            bad = np.abs(out[r] - o) > tol
            assert not bad.any(), (r, float(np.abs(out[r] - o).max()), float((np.abs(out[r] - o) / tol).max()))
            if l is not None:
                empty = np.isneginf(ls)
                assert (np.isneginf(l[r]) == empty).all(), r
                off = np.abs(np.where(empty, 0.0, l[r]) - np.where(empty, 0.0, ls))
                assert (off <= ltol).all(), (r, off.max(), ltol.max())
        assert self.kvq.kvq_pages_read_errors() == 0


RAGGED = [(37, 37), (0, 0), (1, 1), (130, 5), (16, 16), (33, 0), (64, 64), (3, 9), (0, 2), (129, 1)]


# ------------------------------------------------------------------ write

@pytest.mark.parametrize("rotated,signs", [(False, ""), (True, "random"), (True, "ones")])
@pytest.mark.parametrize("d,H,page,dtype", [(128, 2, 16, "fp16"), (128, 3, 64, "bf16"), (64, 1, 32, "bf16"),
                                            (64, 8, 128, "fp16")])
def test_write_stores_the_defined_bits_and_nothing_else(d, H, page, dtype, rotated, signs):
    import torch
    s = Setup(RAGGED, H=H, d=d, page=page, rotated=rotated, signs=signs, lead=2, tail=3, fill=False)
    k, v = s.tensor(H, dtype, fused=2, scale=3.0), s.tensor(H, dtype)
    k[1:9, :, 5] *= 60.0
    s.kvq.kvq_pages_write(s.cfg, s.pages, s.batch, k, v)
    torch.cuda.synchronize()
    for i, x in enumerate((k, v)):
        c, t = ref.pack(host(x), s.signs)
        for r, q, pos in s.b.rows():
            if pos >= 0:
                p, o = s.b.slot(q, pos, page, s.n_pages)
                s.codes[i][p, :, o], s.tok[i][p, :, o] = c[r], t[r]
        assert np.array_equal(s.pages.codes[i].cpu().numpy(), s.codes[i])
        assert np.array_equal(s.pages.tok[i].cpu().numpy().view(np.uint16), s.tok[i].view(np.uint16))
    assert s.kvq.kvq_pages_read_errors() == 0


@pytest.mark.parametrize("rotated", [False, True])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_write_of_extreme_rows(dtype, rotated):
    """NaN, infinities, magnitudes past fp16's, zeros, the smallest numbers."""
    import torch
    d, H = 128, 1
    s = Setup([(24, 24)], H=H, d=d, page=16, rotated=rotated, fill=False)
    x = s.tensor(H, dtype)
    x[0] = 0
    x[1, 0, 3] = float("nan")
    x[2, 0, 9] = float("inf")
    x[3, 0, 10] = -float("inf")
    x[4] = float("nan")
    x[5] = float("inf")
    x[6] = 65504.0
    x[7] = torch.where(torch.arange(d, device="cuda") % 3 == 0, 6e-8, 0.0).to(x.dtype)
    x[8] = x[8] * 1e-6
    x[9] = x[9] * 2e-7
    x[10] = 0
    x[10, 0, 127] = -1.0
    if dtype == "bf16":
        x[11] = 3e38
        x[12, 0, 0] = 1e30
        x[13] = 1e-39
        x[14, 0, 5] = -70000.0
    s.kvq.kvq_pages_write(s.cfg, s.pages, s.batch, x, -x)
    torch.cuda.synchronize()
    for i, y in enumerate((host(x), host(-x))):
        c, t = ref.pack(y, s.signs)
        assert np.isfinite(t.astype(np.float32)).all()
        for r, q, pos in s.b.rows():
            p, o = s.b.slot(q, pos, 16, s.n_pages)
            assert np.array_equal(s.pages.tok[i][p, :, o].cpu().numpy(), t[r]), (i, r)
            assert np.array_equal(s.pages.codes[i][p, :, o].cpu().numpy(), c[r]), (i, r)


def test_write_agrees_with_the_block_cache_in_naive_mode():
    import torch
    from kv_cache_bit_b200 import kvq
    d, H, n = 128, 2, 128
    s = Setup([(n, n)], H=H, d=d, page=128, rotated=False, fill=False)
    k, v = s.tensor(H, "fp16"), s.tensor(H, "fp16")
    s.kvq.kvq_pages_write(s.cfg, s.pages, s.batch, k, v)
    cfg = kvq.Config(d, 4, 0)
    c = kvq.KVCache.allocate(cfg, 1, H, n)
    heads_first = lambda x: x.transpose(0, 1).contiguous()[None].view(torch.int16)  # noqa: E731
    kvq.kvq_quantize_block(cfg, c, heads_first(k), heads_first(v), 0, n)
    page = int(s.b.table[0, 0])
    assert torch.equal(s.pages.codes[0][page], c.codes[0][0])
    for i in range(2):
        assert torch.equal(s.pages.tok[i][page].view(torch.int16), c.tok[i][0, :, :, 0])


# ------------------------------------------------------------------ read

@pytest.mark.parametrize("rotated", [False, True])
@pytest.mark.parametrize("d,H,page,dtype", [(128, 2, 16, "fp16"), (128, 3, 32, "bf16"), (64, 1, 64, "fp32"),
                                            (64, 4, 128, "fp16"), (128, 1, 128, "fp32")])
def test_read_rebuilds_the_rows(d, H, page, dtype, rotated):
    import torch
    s = Setup(RAGGED, H=H, d=d, page=page, rotated=rotated, lead=1, tail=2)
    R = ref.matrix(d, s.signs)
    for which in ((0, 1), (0,), (1,)):
        wide = torch.full((s.rows, 2, H, d + 8), 7.0, dtype=tt(dtype), device="cuda")
        outs = [wide[:, i, :, :d] if i in which else None for i in range(2)]
        s.kvq.kvq_pages_read(s.cfg, s.pages, s.batch, *outs)
        torch.cuda.synchronize()
        got = wide.double().cpu().numpy()
        assert (got[..., d:] == 7).all()
        owned = {r: (q, pos) for r, q, pos in s.b.rows()}
        for i in range(2):
            for r in range(s.rows):
                x = got[r, i, :, :d]
                if i not in which or r not in owned:
                    assert (x == 7).all()
                elif owned[r][1] < 0:
                    assert (x == 0).all()
                else:
                    p, o = s.b.slot(*owned[r], page, s.n_pages)
                    want = (ref.codes_of(s.codes[i][p, :, o]) * s.tok[i][p, :, o].astype(np.float64)[:, None]) @ R
                    # sigma / sqrt(d) and the product, then the result; 2^-25: half a step of fp16's smallest
                    assert (np.abs(x - want) <= (HALF[dtype] + 3 * 2.0 ** -24) * np.abs(want) + 2.0 ** -25
                            + 1e-13).all(), (i, r)
    assert s.kvq.kvq_pages_read_errors() == 0


def test_read_saturates_in_fp16():
    import torch
    s = Setup([(3, 3)], H=1, rotated=False, fill=False)
    x = torch.full((3, 1, 128), 65504.0, dtype=torch.float16, device="cuda")
    x[1] = -x[1]
    s.kvq.kvq_pages_write(s.cfg, s.pages, s.batch, x, x)
    k, v = torch.empty_like(x), torch.empty_like(x)
    s.kvq.kvq_pages_read(s.cfg, s.pages, s.batch, k, v)
    # sigma = fp16(65504 / 7) = 9360, 7 sigma = 65520
    assert torch.equal(k, x) and torch.equal(v, x)


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("rotated,signs", [(False, ""), (True, "random"), (True, "ones")])
@pytest.mark.parametrize("d,H,G,page,dtype", [(128, 2, 4, 16, "fp16"), (128, 1, 7, 64, "bf16"), (64, 3, 1, 32, "fp16"),
                                              (64, 2, 8, 128, "bf16"), (128, 2, 1, 128, "bf16"), (64, 1, 16, 16, "fp16"),
                                              (128, 1, 33, 32, "fp16")])
def test_attention_of_ragged_batches(d, H, G, page, dtype, rotated, signs):
    s = Setup(RAGGED, H=H, d=d, page=page, rotated=rotated, signs=signs, lead=1, tail=2)
    q = s.tensor(H * G, dtype, fused=1, scale=1.5)
    s.check(q, *s.attend(q), dtype)


@pytest.mark.parametrize("d,G,dtype", [(128, 4, "fp16"), (128, 7, "bf16"), (64, 1, "fp16"), (64, 6, "bf16")])
@pytest.mark.parametrize("causal,window", [(True, 1), (True, 2), (True, 40), (True, 1000), (False, 0)])
def test_attention_masks(d, G, dtype, causal, window):
    s = Setup([(1, 1), (200, 70), (65, 65), (7, 12), (0, 3), (300, 1), (64, 2)], d=d, H=2, page=32)
    q = s.tensor(2 * G, dtype)
    s.check(q, *s.attend(q, causal=causal, window=window, scale=0.2), dtype, causal=causal, window=window, scale=0.2)


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 8, 9, 16, 17, 31, 40])
@pytest.mark.parametrize("d,G", [(128, 4), (128, 1), (64, 7)])
def test_attention_of_few_rows_over_longer_sequences(rows, d, G):
    s = Setup([(1100, rows), (777, rows), (64 * 7, rows)], d=d, H=1, page=64, max_rows=rows)
    q = s.tensor(G, "fp16")
    s.check(q, *s.attend(q), "fp16")


@pytest.mark.parametrize("d,G,dtype,rotated", [(128, 2, "fp16", True), (128, 3, "bf16", False), (64, 1, "bf16", True)])
def test_attention_of_prompts(d, G, dtype, rotated):
    s = Setup([(261, 261), (130, 130), (1, 1), (520, 200)], d=d, H=1, page=16, rotated=rotated, tail=1)
    q = s.tensor(G, dtype)
    s.check(q, *s.attend(q), dtype)
    s.check(q, *s.attend(q, window=77), dtype, window=77)


@pytest.mark.parametrize("d,G,dtype,rotated", [(128, 4, "fp16", True), (128, 2, "bf16", False), (64, 4, "bf16", True),
                                               (64, 1, "fp16", False)])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 700), (False, 0)])
def test_attention_of_long_prompts(d, G, dtype, rotated, causal, window):
    """Enough rows that one CTA takes many tiles and several items; a sample of the rows."""
    s = Setup([(2300, 2300), (1500, 700), (90, 90), (1700, 1)], d=d, H=2, page=32, rotated=rotated)
    q = s.tensor(2 * G, dtype, scale=1.3)
    only = {int(r) for r in s.rng.integers(0, s.rows, 60)} | {0, 63, 64, 65, 2299, 2300, 2999, 3000, 3089, 3090}
    s.check(q, *s.attend(q, causal=causal, window=window), dtype, causal=causal, window=window, only=only)


@pytest.mark.parametrize("causal", [True, False])
def test_attention_of_many_rows_over_few_tokens(causal):
    """Empty sequences and paddings with as many rows as a prompt."""
    s = Setup([(0, 100), (5, 90), (1, 64), (64, 300), (128, 128), (-3, 70)], page=16)
    q = s.tensor(4, "fp16")
    s.check(q, *s.attend(q, causal=causal), "fp16", causal=causal)


def test_the_first_call_of_a_process_may_be_captured():
    import subprocess
    import sys
    code = '''
import torch
from tests.test_gpu_pages import Setup
s = Setup([(300, 150), (90, 1)], page=16)
q = s.tensor(8, "fp16")
out, ws = torch.zeros_like(q), torch.empty(
    s.kvq.kvq_pages_attention_workspace_bytes(s.cfg, s.pages, s.batch, s.rows, 8), dtype=torch.uint8, device="cuda")
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    s.kvq.kvq_pages_attention(s.cfg, s.pages, s.batch, q, out, ws=ws)
g.replay()
torch.cuda.synchronize()
s.check(q, out, None, "fp16", only={0, 80, 149, 150})
print("captured")
'''
    done = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=240)
    assert done.returncode == 0 and "captured" in done.stdout, done.stderr[-2000:]


def test_attention_with_a_wrong_row_hint_and_without_lse():
    for hint in (0, 1, 7, 10 ** 6):
        s = Setup([(150, 40), (20, 1), (90, 90)], max_rows=hint)
        q = s.tensor(4, "fp16")
        out, _ = s.attend(q, lse=False)
        s.check(q, out, None, "fp16")


@pytest.mark.parametrize("rows", [3, 50])
def test_attention_of_loud_and_silent_values(rows):
    """Scales over fp16's whole range: tokens of huge and tiny values in one
    sequence, zero rows, queries that single out one token or none."""
    d, H, G = 128, 1, 4
    s = Setup([(300, rows)], d=d, H=H, page=16, rotated=False, fill=False)
    r = s.rng
    mags = np.exp(r.uniform(np.log(1e-6), np.log(3e4), (300, 1, 1))).astype(np.float32)
    x = [(r.standard_normal((300, H, d)) * (1 if i == 0 else mags)).astype(np.float32) for i in range(2)]
    x[1][10:40] = 0
    x[0][50:60] = 0
    for i in range(2):
        c, t = ref.pack(x[i], None)
        for k in range(300):
            p, o = s.b.slot(0, k, 16, s.n_pages)
            s.codes[i][p, :, o], s.tok[i][p, :, o] = c[k], t[k]
    import torch
    for i in range(2):
        s.pages.codes[i].copy_(torch.from_numpy(s.codes[i]))
        s.pages.tok[i].copy_(torch.from_numpy(s.tok[i]))
    for scale in (0.0, 1e-4, 4.0):
        q = s.tensor(G, "bf16", scale=2.0)
        q[0] = 0
        s.check(q, *s.attend(q, scale=scale), "bf16", scale=scale, many=rows == 50)


@pytest.mark.parametrize("rows", [6, 40])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("rotated", [False, True])
def test_attention_of_extreme_queries(dtype, rotated, rows):
    s = Setup([(100, rows)], rotated=rotated)
    q = s.tensor(4, dtype)
    q[0] *= 1e-6
    q[1] *= 2e3
    q[2, :, 1] = 6e4
    if dtype == "bf16":
        q[3] *= 1e-36
        q[4] *= 1e-3
    s.check(q, *s.attend(q, scale=0.003), dtype, scale=0.003)


@pytest.mark.parametrize("rows", [4, 90])
def test_a_query_that_is_not_a_number_stays_in_its_row(rows):
    s = Setup([(100, rows), (50, 1)])
    q = s.tensor(4, "fp16")
    q[1, 2, 5] = float("nan")
    q[2, 1, 7] = float("inf")
    import torch
    out, lse = s.attend(q)
    bad = torch.isnan(out).any(-1)
    want = torch.zeros_like(bad)
    want[1, 2] = want[2, 1] = True
    assert torch.equal(bad, want)
    q2, keep = q.clone(), ~want
    q2[~keep] = 0
    out2, lse2 = s.attend(q2)
    assert torch.equal(out[keep], out2[keep]) and torch.equal(lse[keep], lse2[keep])


def test_a_row_does_not_depend_on_its_neighbours():
    """The same bits for rows of a sequence whatever the other rows' queries are."""
    import torch
    s = Setup([(700, 300), (300, 40)], page=32)
    q = s.tensor(4, "bf16")
    q2 = s.tensor(4, "bf16", scale=30.0)
    q2[::3] = q[::3]
    (a, la), (b, lb) = s.attend(q), s.attend(q2)
    assert torch.equal(a[::3], b[::3]) and torch.equal(la[::3], lb[::3])
    s.check(q2, b, lb, "bf16", only=set(range(0, s.rows, 17)))


# ------------------------------------------------------------------ bad pages

@pytest.mark.parametrize("rows", [1, 30])
def test_pages_outside_the_pool_are_left_out(rows):
    import torch
    s = Setup([(200, rows), (90, rows), (130, rows)], page=16, H=2)
    for bad in (-1, s.n_pages, 2 ** 31 - 1, -2 ** 31):
        table = s.b.table.copy()
        table[0, 3] = table[1, 0] = bad
        table[1, 5] = bad  # the page of sequence 1's last rows
        keep, s.b.table = s.b.table, table
        wide = s.batch.table.clone()
        wide[:, :table.shape[1]] = torch.from_numpy(table).cuda()
        batch, s.batch = s.batch, s.kvq.Batch(s.batch.start, s.batch.length, wide[:, :table.shape[1]])
        q = s.tensor(8, "fp16")
        out, lse = s.attend(q)
        assert s.kvq.kvq_pages_read_errors() == 4
        s.check(q, out, lse, "fp16")
        before = [c.clone() for c in s.pages.codes]
        x = s.tensor(2, "fp16")
        ko, vo = torch.full_like(x, 7.0), torch.full_like(x, 7.0)
        s.kvq.kvq_pages_read(s.cfg, s.pages, s.batch, ko, vo)
        assert s.kvq.kvq_pages_read_errors() == 4
        for r, q_, pos in s.b.rows():
            if s.b.slot(q_, pos, 16, s.n_pages) is None:
                assert not ko[r].any() and not vo[r].any()
            else:
                assert ko[r].any()
        s.kvq.kvq_pages_write(s.cfg, s.pages, s.batch, x, x)
        assert s.kvq.kvq_pages_read_errors() == 4
        touched = {s.b.slot(q_, pos, 16, s.n_pages) for r, q_, pos in s.b.rows()}
        for i in range(2):
            diff = (before[i] != s.pages.codes[i]).any(-1).any(1).cpu().numpy()
            assert {(int(a), int(b)) for a, b in zip(*np.nonzero(diff))} <= touched
            s.pages.codes[i].copy_(torch.from_numpy(s.codes[i]))
            s.pages.tok[i].copy_(torch.from_numpy(s.tok[i]))
        s.b.table, s.batch = keep, batch


def test_tokens_past_the_table_are_left_out():
    import torch
    s = Setup([(100, 3), (60, 60)], page=16)
    short = s.kvq.Batch(s.batch.start, s.batch.length, s.batch.table[:, :4])
    s.b.table, s.batch = s.b.table[:, :4], short
    q = s.tensor(4, "fp16")
    out, lse = s.attend(q)
    assert s.kvq.kvq_pages_read_errors() == 4
    s.check(q, out, lse, "fp16")
    x = s.tensor(2, "fp16")
    s.kvq.kvq_pages_write(s.cfg, s.pages, s.batch, x, x)
    assert s.kvq.kvq_pages_read_errors() == 4
    out = torch.full_like(x, 7.0)
    s.kvq.kvq_pages_read(s.cfg, s.pages, s.batch, out, None)
    assert s.kvq.kvq_pages_read_errors() == 4
    assert not out[:3].any() and out[3:].any(-1).all()


# ------------------------------------------------------------------ shapes of use

def test_many_sequences():
    """More sequences than a block keeps start[] of in shared memory."""
    counts = [(i % 7, min(i % 7, 1 + i % 2)) for i in range(1500)]
    import torch
    s = Setup(counts, H=1, d=64, page=16, spare=5)
    q = s.tensor(2, "fp16")
    s.check(q, *s.attend(q), "fp16")
    x = s.tensor(1, "fp16")
    s.kvq.kvq_pages_write(s.cfg, s.pages, s.batch, x, x)
    k = torch.empty_like(x)
    s.kvq.kvq_pages_read(s.cfg, s.pages, s.batch, k, None)
    c, t = ref.pack(host(x), s.signs)
    want = (ref.codes_of(c) * t.astype(np.float64)[..., None]) @ ref.matrix(64, s.signs)
    own = [r for r, _, pos in s.b.rows()]
    assert np.abs(host(k)[own] - want[own]).max() <= 2.0 ** -10 * np.abs(want).max()


def test_sequences_may_share_pages():
    """Two sequences with one prefix: their tables name the same pages."""
    import torch
    s = Setup([(96, 1), (96, 1)], page=16, H=2)
    s.b.table[1, :3] = s.b.table[0, :3]
    s.batch.table.copy_(torch.from_numpy(s.b.table))
    q = s.tensor(4, "fp16")
    s.check(q, *s.attend(q), "fp16")


def test_head_major_tensors_and_broadcast_inputs():
    """Tensors whose heads are the outer dimension, and inputs of stride 0."""
    import torch
    s = Setup([(40, 40), (9, 2)], H=2, page=16)
    q = s.tensor(4, "fp16")
    flipped = q.transpose(0, 1).contiguous().transpose(0, 1)
    out, lse = s.attend(q)
    other = torch.full((4, s.rows, 128), 7.0, dtype=torch.float16, device="cuda").transpose(0, 1)
    ws = torch.empty(s.kvq.kvq_pages_attention_workspace_bytes(s.cfg, s.pages, s.batch, s.rows, 4),
                     dtype=torch.uint8, device="cuda")
    s.kvq.kvq_pages_attention(s.cfg, s.pages, s.batch, flipped, other, None, ws=ws)
    assert torch.equal(out, other)
    one = q[:1, :1].expand(s.rows, 2, 128)
    s.kvq.kvq_pages_write(s.cfg, s.pages, s.batch, one, one)
    k, v = (torch.empty(2, s.rows, 128, dtype=torch.float16, device="cuda").transpose(0, 1) for _ in range(2))
    s.kvq.kvq_pages_read(s.cfg, s.pages, s.batch, k, v)
    assert torch.equal(k, k[:1, :1].expand_as(k)) and torch.equal(k, v) and k[0, 0].any()


def test_other_streams_and_two_calls_at_once():
    """Two calls on two streams with workspaces of their own, and the same
    results as one after the other."""
    import torch
    s = Setup([(900, 1), (400, 20), (1300, 1), (600, 150)], page=64)
    q = [s.tensor(8, "fp16"), s.tensor(8, "fp16")]
    want = [s.attend(x) for x in q]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    need = s.kvq.kvq_pages_attention_workspace_bytes(s.cfg, s.pages, s.batch, s.rows, 8)
    bufs = [(torch.full_like(x, 7.0), torch.full(x.shape[:2], 7.0, device="cuda"),
             torch.empty(need, dtype=torch.uint8, device="cuda")) for x in q]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, x, (o, l, ws) in zip(streams, q, bufs):
            s.kvq.kvq_pages_attention(s.cfg, s.pages, s.batch, x, o, l, ws=ws, stream=st)
    torch.cuda.synchronize()
    for (o, l, _), (wo, wl) in zip(bufs, want):
        assert torch.equal(o, wo) and torch.equal(l, wl)


@pytest.mark.parametrize("hint", [0, 1])
def test_captured_steps_follow_the_batch_contents(hint):
    """write + attention + read in a graph, replayed while lengths, rows and
    tables change in place; a second graph shares the workspace (in order)."""
    import torch
    s = Setup([(60, 1), (200, 1), (31, 1)], page=16, H=2, spare=12, max_rows=hint)
    kvq = s.kvq
    used = {int(p) for q_, n in enumerate((60, 200, 31)) for p in s.b.table[q_, :-(-n // 16)]}
    s.b.table[2, 2] = next(p for p in range(s.n_pages) if p not in used)  # where sequence 2 grows to
    s.batch.table.copy_(torch.from_numpy(s.b.table))
    need = kvq.kvq_pages_attention_workspace_bytes(s.cfg, s.pages, s.batch, s.rows, 8)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    k, v, q = s.tensor(2, "fp16"), s.tensor(2, "fp16"), s.tensor(8, "fp16")
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    k_out, v_out = torch.empty_like(k), torch.empty_like(v)

    def step():
        kvq.kvq_pages_write(s.cfg, s.pages, s.batch, k, v)
        kvq.kvq_pages_attention(s.cfg, s.pages, s.batch, q, out, lse, ws=ws)
        kvq.kvq_pages_read(s.cfg, s.pages, s.batch, k_out, v_out)

    step()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append(g)
    for i in range(4):
        s.b.length = s.b.length + np.array([1, 0, 1], np.int32)
        if i == 2:
            s.b.length[1] = 0
        s.batch.length.copy_(torch.from_numpy(s.b.length))
        for x, heads in ((k, 2), (v, 2), (q, 8)):
            x.copy_(s.tensor(heads, "fp16"))
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        for j in range(2):
            s.codes[j], s.tok[j] = s.pages.codes[j].cpu().numpy(), s.pages.tok[j].cpu().numpy()
        s.check(q, out, lse, "fp16")
        c, t = ref.pack(host(k), s.signs)
        for r, seq, pos in s.b.rows():
            if pos >= 0:
                p, o = s.b.slot(seq, pos, 16, s.n_pages)
                assert np.array_equal(s.codes[0][p, :, o], c[r]) and np.array_equal(s.tok[0][p, :, o], t[r])
                got = host(k_out)[r]
                want = (ref.codes_of(c[r]) * t[r].astype(np.float64)[:, None]) @ ref.matrix(128, s.signs)
                assert np.abs(got - want).max() <= 2.0 ** -10 * np.abs(want).max()


def test_repeated_calls_give_the_same_bits():
    import torch
    s = Setup([(1500, 1), (700, 33), (2100, 2)], page=64, H=2)
    q = s.tensor(8, "fp16")
    a = s.attend(q)
    for _ in range(3):
        b = s.attend(q)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_offsets_past_32_bits():
    """Pages at the end of a pool of more than 2^32 bytes of codes a tensor."""
    import torch
    from kv_cache_bit_b200 import kvq
    H, d, page = 4, 128, 64
    n_pages = (1 << 32) // (H * page * d // 2) + 600
    cfg = kvq.Config(d, 4, kvq.HADAMARD, kvq.kvq_make_signs(1, d))
    codes = [torch.empty((n_pages, H, page, d // 2), dtype=torch.uint8, device="cuda") for _ in range(2)]
    tok = [torch.empty((n_pages, H, page), dtype=torch.float16, device="cuda") for _ in range(2)]
    pages = kvq.PagedCache.wrap(cfg, codes, tok)
    s = Setup([(700, 700), (33, 33)], H=H, d=d, page=page, rotated=True, fill=False)
    s.cfg, s.signs = cfg, kvq.kvq_make_signs(1, d)
    far = (s.batch.table % s.n_pages) + (n_pages - s.n_pages)
    batch = kvq.Batch(s.batch.start, s.batch.length, far.to(torch.int32))
    k, v, q = s.tensor(H, "fp16"), s.tensor(H, "fp16"), s.tensor(2 * H, "fp16")
    kvq.kvq_pages_write(cfg, pages, batch, k, v)
    small = kvq.PagedCache.wrap(cfg, [c[-s.n_pages:].clone() for c in codes], [t[-s.n_pages:].clone() for t in tok])
    near = kvq.Batch(s.batch.start, s.batch.length, (s.batch.table % s.n_pages).to(torch.int32))
    got = []
    for p, b in ((pages, batch), (small, near)):
        out, ko = torch.empty_like(q), torch.empty_like(k)
        ws = torch.empty(kvq.kvq_pages_attention_workspace_bytes(cfg, p, b, s.rows, 2 * H), dtype=torch.uint8,
                         device="cuda")
        kvq.kvq_pages_attention(cfg, p, b, q, out, ws=ws)
        kvq.kvq_pages_read(cfg, p, b, ko, None)
        got.append((out, ko))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    s.pages, s.batch, s.b.table = small, near, s.b.table % s.n_pages
    for i in range(2):
        s.codes[i], s.tok[i] = small.codes[i].cpu().numpy(), small.tok[i].cpu().numpy()
    sub = [0, 350, 699, 700, 732]
    want = ref.attention((s.codes[0], s.tok[0]), (s.codes[1], s.tok[1]), s.b, host(q), s.signs, 0.0, True, 0, 2.0 ** -11)
    for r in sub:
        assert (np.abs(host(got[0][0])[r] - want[r][0]) <= want[r][2]).all()


def test_a_prompt_and_generation_steps_together():
    """The calls as they are used: a prompt in two chunks, then steps in a
    batch with another sequence, against 64 bits at every step."""
    import torch
    from kv_cache_bit_b200 import kvq
    H, G, d, page = 2, 4, 128, 16
    s = Setup([(90, 90), (45, 45)], H=H, d=d, page=page, spare=30, fill=False)
    cfg, pages = s.cfg, s.pages
    table = torch.from_numpy(np.pad(s.b.table % s.n_pages, ((0, 0), (0, 4)))).cuda()
    free = [p for p in range(s.n_pages) if p not in set(s.b.table[0]) | set(s.b.table[1][:3])]
    table[1, 3:] = torch.tensor(free[:table.shape[1] - 3], dtype=torch.int32)
    table[0, 6:] = torch.tensor(free[10:10 + table.shape[1] - 6], dtype=torch.int32)
    plan = [[(50, 50), (45, 45)], [(90, 40), (46, 1)]] + [[(90 + i, 1), (46 + i, 1)] for i in range(1, 5)]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for counts in plan:
        start = np.concatenate(([0], np.cumsum([r for _, r in counts]))).astype(np.int32)
        b = kvq.Batch(i32(start.tolist()), i32([c for c, _ in counts]), table, max_rows=max(r for _, r in counts))
        s.rows, s.batch = int(start[-1]), b
        s.b = ref.Seqs(start, np.array([c for c, _ in counts], np.int32), table.cpu().numpy())
        k, v, q = s.tensor(H, "bf16"), s.tensor(H, "bf16"), s.tensor(H * G, "bf16")
        kvq.kvq_pages_write(cfg, pages, b, k, v)
        out, lse = s.attend(q)
        for j in range(2):
            s.codes[j], s.tok[j] = pages.codes[j].cpu().numpy(), pages.tok[j].cpu().numpy()
        s.check(q, out, lse, "bf16")
