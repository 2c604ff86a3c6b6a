"""What is measured of the paged 4-bit cache: writing tokens into it, reading
them back, and attention over it, as plain torch operations and as calls of
the library.

A cache is a pool of pages.  For K and for V it holds packed 4-bit codes
[n_pages][kv_heads][page][head_dim / 2] and one fp16 scale a token and head
[n_pages][kv_heads][page].  A batch says which rows of a tensor belong to
which sequence: rows start[s] .. start[s + 1] - 1 are the last tokens of
sequence s, whose token count is length[s] and whose pages are table[s].

  write      y = x, or R x with R = H diag(signs) / sqrt(d); sigma = fp16(max|y| / 7);
             q = rint(y r) in -7 .. 7 with r = 1 / sigma in 32 bits; stored are
             q + 8 and sigma
  read       sigma q, or R^T (sigma q)
  attention  softmax(scale q . k_hat) v_hat over the tokens a row sees: all up
             to its own (causal) or all of the sequence, of these the last
             `window` where a window is given; also the log of the sum
"""
import math
import random

import torch

own = False

# ------------------------------------------------------------------ cases


def _case(name, op, lens, rows, hq, hkv, d, page, dtype, rotate, causal=True, window=0):
    """lens: "n x low .. high" token counts, ragged where low < high; rows: new
    rows of each sequence, "all" (every token) or "mixed:r" (r rows for the
    first eighth of the sequences, one for the others)."""
    return {"name": name, "op": op, "lens": lens, "rows": rows, "hq": hq, "hkv": hkv, "d": d, "page": page,
            "dtype": dtype, "rotate": rotate, "causal": causal, "window": window}


def listed():
    return [
        # one token for each of a few sequences: a generation step's write and its read-back
        _case("write step 8", "write", "8 x 700 .. 1500", "1", 32, 8, 128, 16, "fp16", True),
        # ragged prompts of a 4-head model, bf16, no rotation
        _case("write prompts 28-4", "write", "12 x 37 .. 4093", "all", 28, 4, 128, 64, "bf16", False),
        # a whole prefill of a large batch
        _case("write prefill 32x4096", "write", "32 x 4096 .. 4096", "all", 32, 8, 128, 64, "fp16", True),
        # a small head dim, ragged, read back whole
        _case("read ragged d64", "read", "16 x 1 .. 1023", "all", 8, 8, 64, 16, "fp16", True),
        # a long prefix rebuilt in 16 bits for another consumer
        _case("read prefix 4x32768", "read", "4 x 32768 .. 32768", "all", 32, 8, 128, 128, "bf16", True),
        # the smallest attention call: one sequence, one token, a short cache
        _case("attend 1x256 d64", "attend", "1 x 256 .. 256", "1", 8, 8, 64, 16, "fp16", False),
        # a generation step of a grouped-query model, 7 query heads a kv head
        _case("attend 8x4096 28-4", "attend", "8 x 2049 .. 4095", "1", 28, 4, 128, 16, "bf16", True),
        # the largest generation step: 64 ragged sequences
        _case("attend 64x8192 32-8", "attend", "64 x 500 .. 8192", "1", 32, 8, 128, 64, "fp16", True),
        # few sequences with long contexts
        _case("attend 4x32768 32-8", "attend", "4 x 32000 .. 32768", "1", 32, 8, 128, 64, "fp16", True),
        # a few drafted tokens a sequence, checked at once
        _case("attend draft 16x5", "attend", "16 x 300 .. 3001", "5", 28, 4, 128, 32, "bf16", False),
        # generation steps and two prompt chunks in one batch, sliding window
        _case("attend mixed 16", "attend", "16 x 1000 .. 4096", "mixed:500", 32, 8, 128, 64, "fp16", True, True, 2048),
        # a whole prompt attending to itself
        _case("attend prompt 8192", "attend", "1 x 8192 .. 8192", "all", 32, 8, 128, 128, "bf16", True),
    ]


def draw(rng):
    """One more case of the ranges of listed()."""
    op = rng.choice(["write", "read", "attend", "attend", "attend"])
    hq, hkv = rng.choice([(8, 8), (28, 4), (32, 8), (32, 32), (16, 1), (12, 4)])
    d, page = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    spread = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    window, causal = 0, True
    if op != "attend":
        n = spread(1, 48)
        high = spread(1, min(32768, 32 * 4096 * 8 // (n * max(hkv, 8))))
        low = rng.choice([1, high // 3 + 1, high])
        rows = rng.choice(["1", "all", "all", str(rng.randint(2, 200))])
    else:
        n = spread(1, 64)
        high = spread(1, min(32768, 64 * 8192 * 8 // (n * max(hkv, 8))))
        low = rng.choice([1, high // 2 + 1, high])
        room = 8192 * 4096 * 32 // (n * high * hq)  # rows a sequence at the largest listed case's scores
        rows = rng.choice(["1", "1", str(rng.randint(2, 9)), str(spread(9, 900)), "all", "mixed:%d" % spread(2, 600)])
        most = high if rows == "all" else int(rows.split(":")[-1])
        if most > max(1, room):
            rows = str(max(1, min(room, 16)))
        causal = rng.random() < 0.8
        if causal and rng.random() < 0.3:
            window = spread(1, 4096)
    return {"op": op, "lens": "%d x %d .. %d" % (n, low, high), "rows": rows, "hq": hq, "hkv": hkv, "d": d,
            "page": page, "dtype": rng.choice(["fp16", "bf16"]), "rotate": rng.random() < 0.6, "causal": causal,
            "window": window}


def _counts(case):
    """(token counts, row counts) of the sequences, from the case alone."""
    n, rest = case["lens"].split(" x ")
    n, (low, high) = int(n), (int(x) for x in rest.split(" .. "))
    r = random.Random("%s %s" % (case["lens"], case["page"]))
    lens = [r.randint(low, high) for _ in range(n)]
    lens[n // 2] = high
    if case["rows"] == "all":
        rows = list(lens)
    elif case["rows"].startswith("mixed:"):
        many = int(case["rows"][6:])
        rows = [many if i < (n + 7) // 8 else 1 for i in range(n)]
    else:
        rows = [int(case["rows"])] * n
    return lens, [min(a, b) for a, b in zip(rows, lens)]


def _pairs(case):
    """How many (row, token) pairs the attention of one head covers, and how
    many tokens of the cache some row sees."""
    pairs = seen = 0
    for n, m in zip(*_counts(case)):
        w = case["window"] or n
        if case["causal"]:
            pairs += sum(min(p + 1, w) for p in range(n - m, n))
            seen += min(n, m + w - 1)
        else:
            pairs += n * m
            seen += n
    return pairs, seen


def work(case):
    """Each input read once, each output written once; the page table and the
    sequence lengths are left out (a few bytes a page)."""
    lens, rows = _counts(case)
    d, hkv, hq, m = case["d"], case["hkv"], case["hq"], sum(rows)
    packed = 2 * hkv * (d // 2 + 2)  # K and V of one token
    plain = 2 * hkv * d * 2
    turn = int(math.log2(d)) * d if case["rotate"] else 0
    if case["op"] == "write":  # 16-bit rows in, codes out, codes in, 16-bit rows out
        return {"bytes": 2 * m * (plain + packed), "flops": 2 * m * 2 * hkv * (6 * d + turn)}
    if case["op"] == "read":
        return {"bytes": m * (plain + packed), "flops": m * 2 * hkv * (2 * d + turn)}
    pairs, seen = _pairs(case)
    return {"bytes": seen * packed + m * hq * (2 * d * 2 + 4), "flops": 4 * pairs * d * hq}


# ------------------------------------------------------------------ plain forms


def _stage(x, s):
    """One stage of the Walsh-Hadamard transform: a + b and a - b of the
    elements s apart."""
    y = x.unflatten(-1, (-1, 2, s))
    a, b = y[..., 0, :], y[..., 1, :]
    return torch.stack((a + b, a - b), -2).flatten(-3)


def _hadamard(x):
    y = _stage(_stage(_stage(_stage(_stage(_stage(x, 1), 2), 4), 8), 16), 32)
    return _stage(y, 64) if x.shape[-1] == 128 else y


def _turn(x, signs):
    """R x; signs None: x."""
    return x if signs is None else _hadamard(x * signs) * (1.0 / math.sqrt(x.shape[-1]))


def _turn_back(x, signs):
    return x if signs is None else _hadamard(x) * (1.0 / math.sqrt(x.shape[-1])) * signs


def _pack(x, signs):
    """Codes (uint8, two a byte) and fp16 scales of rows x."""
    y = _turn(x.float().nan_to_num(0.0, 65504.0, -65504.0).clamp(-65504.0, 65504.0), signs)
    sigma = (y.abs().amax(-1) / 7.0).clamp(max=65504.0).half()
    inverse = torch.where(sigma > 0, 1.0 / sigma.float(), 0.0)
    # the product of two 24-bit numbers is exact in 64 bits, so the only rounding is to the code
    q = (y.double() * inverse.double().unsqueeze(-1)).round().clamp(-7, 7)
    e = (q + 8).to(torch.uint8).unflatten(-1, (-1, 2))
    return e[..., 0] | (e[..., 1] << 4), sigma


def _values(codes, sigma):
    """sigma q in 32 bits, in the stored (rotated) domain."""
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float() - 8.0
    return q * sigma.float().unsqueeze(-1)


def _places(s):
    """(page, slot) of every row's token."""
    step = torch.arange(s["rows"], device="cuda") - s["start"][:-1].long()[s["owner"]]
    pos = s["first"][s["owner"]] + step
    return s["table"].long()[s["owner"], pos // s["page"]], pos % s["page"]


def _plain_write(s):
    page, slot = _places(s)
    for_k, k_scale = _pack(s["k"], s["signs_f"])
    for_v, v_scale = _pack(s["v"], s["signs_f"])
    s["codes"][0][page, :, slot] = for_k
    s["codes"][1][page, :, slot] = for_v
    s["tok"][0][page, :, slot] = k_scale
    s["tok"][1][page, :, slot] = v_scale


def _plain_read(s):
    page, slot = _places(s)
    k = _values(s["codes"][0][page, :, slot], s["tok"][0][page, :, slot])
    v = _values(s["codes"][1][page, :, slot], s["tok"][1][page, :, slot])
    top = torch.finfo(s["type"]).max
    return tuple(_turn_back(x, s["signs_f"]).clamp(-top, top).to(s["type"]) for x in (k, v))


def _plain_attend(s):
    n, hkv, d, page = s["n"], s["hkv"], s["d"], s["page"]
    group, most = s["hq"] // hkv, s["most_rows"]
    table = s["table"].long()[:, :-(-s["most_len"] // page)]
    whole = lambda x: x[table].transpose(1, 2).flatten(2, 3)  # noqa: E731   [n, hkv, tokens, ...]
    k = _values(whole(s["codes"][0]), whole(s["tok"][0]))
    v = _values(whole(s["codes"][1]), whole(s["tok"][1]))
    step = torch.arange(most, device="cuda")
    counts = (s["start"][1:] - s["start"][:-1]).long()
    valid = step < counts[:, None]
    at = (s["start"][:-1].long()[:, None] + step).clamp(max=s["rows"] - 1)
    q = _turn(s["q"][at].float(), s["signs_f"]) * (1.0 / math.sqrt(d))
    q = q.unflatten(2, (hkv, group)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [n, hkv, group * most, d]
    token = torch.arange(k.shape[2], device="cuda")
    pos = s["first"][:, None] + step
    sees = (token < s["length"].long()[:, None, None]).expand(n, most, -1)
    if s["causal"]:
        sees = sees & (token <= pos[..., None])
    if s["window"]:
        sees = sees & (token > pos[..., None] - s["window"])
    score = (q @ k.transpose(-1, -2)).unflatten(2, (group, most))
    score = score.masked_fill(~sees[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = p.flatten(2, 3) @ v
    o = o.unflatten(2, (group, most)) / torch.where(total > 0, total, 1.0)
    limit = torch.finfo(s["type"]).max
    o = _turn_back(o, s["signs_f"]).clamp(-limit, limit).permute(0, 3, 1, 2, 4).flatten(2, 3)
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 3, 1, 2).flatten(2, 3)
    return o[valid].to(s["type"]), lse[valid]


# ------------------------------------------------------------------ inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    lens, rows = _counts(case)
    n, hkv, hq, d, page = len(lens), case["hkv"], case["hq"], case["d"], case["page"]
    kind = {"fp16": torch.float16, "bf16": torch.bfloat16}[case["dtype"]]
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)  # noqa: E731
    need = [-(-x // page) for x in lens]
    pool = sum(need) + 3  # pages lie in no order, and some belong to nobody
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    ends = ints(need).cumsum(0)
    column = torch.arange(max(need), device="cuda")
    table = order[(column + (ends - ints(need))[:, None]).clamp(max=pool - 1)].contiguous()
    signs = torch.where(torch.rand(d, generator=g, device="cuda") < 0.5, -1, 1).to(torch.int8) if case["rotate"] else None
    signs_f = None if signs is None else signs.float()
    loud = torch.ones(d, device="cuda")
    loud[torch.randperm(d, generator=g, device="cuda")[:4]] = 8.0  # a few channels of K are larger than the rest

    def keys(*shape):
        return randn(*shape, d) * loud * torch.exp(0.4 * randn(*shape, 1))

    def values(*shape):
        return randn(*shape, d) * torch.exp(0.4 * randn(*shape, 1))

    total = sum(rows)
    s = {"op": case["op"], "n": n, "hkv": hkv, "hq": hq, "d": d, "page": page, "type": kind, "rows": total,
         "causal": case["causal"], "window": case["window"], "most_len": max(lens), "most_rows": max(rows),
         "signs": signs, "signs_f": signs_f, "table": table, "length": ints(lens),
         "start": torch.cat((ints([0]), ints(rows).cumsum(0).to(torch.int32))),
         "first": ints(lens).long() - ints(rows).long(),
         "owner": torch.repeat_interleave(torch.arange(n, device="cuda"), ints(rows).long())}
    codes = [torch.full((pool, hkv, page, d // 2), 0x88, dtype=torch.uint8, device="cuda") for _ in range(2)]
    tok = [torch.zeros((pool, hkv, page), dtype=torch.float16, device="cuda") for _ in range(2)]
    s["codes"], s["tok"] = codes, tok
    if case["op"] == "write":
        s["k"], s["v"] = keys(total, hkv).to(kind), values(total, hkv).to(kind)
    else:  # a cache that is already full
        part = max(1, (1 << 26) // (hkv * page * d))
        for at in range(0, pool, part):
            m = min(part, pool - at)
            for i, make in enumerate((keys, values)):
                codes[i][at:at + m], tok[i][at:at + m] = _pack(make(m, hkv, page).to(kind), signs_f)
    if case["op"] == "attend":
        s["q"] = randn(total, hq, d).to(kind)
        s["out"] = torch.zeros((total, hq, d), dtype=kind, device="cuda")
        s["lse"] = torch.zeros((total, hq), dtype=torch.float32, device="cuda")
    else:
        s["k_out"] = torch.zeros((total, hkv, d), dtype=kind, device="cuda")
        s["v_out"] = torch.zeros_like(s["k_out"])
    return s


# ------------------------------------------------------------------ one pass


def _handles(s):
    """What a program makes once and keeps: the configuration, the pool's and
    the batch's descriptions and the attention's workspace."""
    from kv_cache_bit_b200 import kvq

    cfg = kvq.Config(s["d"], 4, 0 if s["signs"] is None else kvq.HADAMARD, s["signs"])
    pages = kvq.PagedCache.wrap(cfg, s["codes"], s["tok"])
    batch = kvq.Batch(s["start"], s["length"], s["table"], max_rows=s["most_rows"])
    ws = None
    if s["op"] == "attend":
        need = kvq.kvq_pages_attention_workspace_bytes(cfg, pages, batch, s["rows"], s["hq"])
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    return kvq, cfg, pages, batch, ws


def run(s):
    if not own:
        if s["op"] == "attend":
            return _plain_attend(s)
        if s["op"] == "write":
            _plain_write(s)
        return _plain_read(s)
    if "handles" not in s:
        s["handles"] = _handles(s)
    kvq, cfg, pages, batch, ws = s["handles"]
    if s["op"] == "attend":
        kvq.kvq_pages_attention(cfg, pages, batch, s["q"], s["out"], s["lse"], causal=s["causal"], window=s["window"], ws=ws)
        return s["out"], s["lse"]
    if s["op"] == "write":
        kvq.kvq_pages_write(cfg, pages, batch, s["k"], s["v"])
    kvq.kvq_pages_read(cfg, pages, batch, s["k_out"], s["v_out"])
    return s["k_out"], s["v_out"]


# ------------------------------------------------------------------ 64 bits


def _matrix(d, signs):
    """R in 64 bits: Sylvester's matrix, H[i][j] = (-1)^popcount(i & j)."""
    if signs is None:
        return torch.eye(d, dtype=torch.float64, device="cuda")
    h = torch.ones((1, 1), dtype=torch.float64, device="cuda")
    while h.shape[0] < d:
        h = torch.cat((torch.cat((h, h), 1), torch.cat((h, -h), 1)), 0)
    return h * signs.double() / math.sqrt(d)


def exact(case, seed):
    s = prepare(case, seed)
    d, hkv, hq, page = s["d"], s["hkv"], s["hq"], s["page"]
    turn = _matrix(d, s["signs"])
    lens, rows = _counts(case)
    if case["op"] == "write":
        found = []
        for x in (s["k"], s["v"]):
            out = torch.empty(x.shape, dtype=torch.float64, device="cuda")
            for at in range(0, x.shape[0], 4096):
                y = x[at:at + 4096].double() @ turn.T
                sigma = (y.abs().amax(-1, keepdim=True) / 7).half().double()
                r = (1.0 / torch.where(sigma > 0, sigma, torch.inf).float()).double()
                q = torch.round(y * r).clamp(-7, 7)
                out[at:at + 4096] = (sigma * q) @ turn
            found.append(out)
        return tuple(found)

    def stored(i, seq, begin, end):
        """Rows [hkv, tokens, d] of a sequence in the stored domain."""
        pages = s["table"][seq, begin // page:-(-end // page)].long()
        c = s["codes"][i][pages].transpose(0, 1).reshape(hkv, -1, d // 2).to(torch.int64)
        t = s["tok"][i][pages].transpose(0, 1).reshape(hkv, -1, 1).double()
        x = torch.empty((*c.shape[:2], d), dtype=torch.float64, device="cuda")
        x[..., 0::2], x[..., 1::2] = (c % 16 - 8).double(), (c // 16 - 8).double()
        skip = begin - begin // page * page
        return (x * t)[:, skip:skip + end - begin]

    if case["op"] == "read":
        out = [torch.empty((s["rows"], hkv, d), dtype=torch.float64, device="cuda") for _ in range(2)]
        at = 0
        for seq, (n, m) in enumerate(zip(lens, rows)):
            for i in range(2):
                out[i][at:at + m] = (stored(i, seq, n - m, n) @ turn).transpose(0, 1)
            at += m
        return tuple(out)

    out = torch.empty((s["rows"], hq, d), dtype=torch.float64, device="cuda")
    lse = torch.empty((s["rows"], hq), dtype=torch.float64, device="cuda")
    group, at = hq // hkv, 0
    for seq, (n, m) in enumerate(zip(lens, rows)):
        k, v = stored(0, seq, 0, n), stored(1, seq, 0, n)
        for r in range(0, m, 256):
            c = min(256, m - r)
            q = s["q"][at + r:at + r + c].double() @ turn.T
            pos = torch.arange(n - m + r, n - m + r + c, device="cuda")[:, None]
            token = torch.arange(n, device="cuda")
            hidden = torch.zeros((c, n), dtype=torch.bool, device="cuda")
            if case["causal"]:
                hidden |= token > pos
            if case["window"]:
                hidden |= token <= pos - case["window"]
            for h in range(hq):
                x = (q[:, h] @ k[h // group].T / math.sqrt(d)).masked_fill(hidden, float("-inf"))
                lse[at + r:at + r + c, h] = torch.logsumexp(x, -1)
                out[at + r:at + r + c, h] = torch.softmax(x, -1) @ v[h // group] @ turn
        at += m
    return out, lse
