"""The paged 4-bit cache in plain numpy: the stored bits from the definition
(fp32 butterflies in the stated order, every other step exact or rounded as
stated), reading back and attention in 64 bits, and the error bounds that the
kernels' roundings allow."""
from __future__ import annotations

import math
from dataclasses import dataclass

import numpy as np


def bf16_to_f32(bits: np.ndarray) -> np.ndarray:
    return (bits.astype(np.uint32) << 16).view(np.float32)


def butterflies(x: np.ndarray) -> np.ndarray:
    """Unnormalized Walsh-Hadamard transform of the last axis in x's own type,
    strides 1, 2, .., d / 2."""
    d, h = x.shape[-1], 1
    while h < d:
        y = x.reshape(*x.shape[:-1], d // (2 * h), 2, h)
        x = np.stack((y[..., 0, :] + y[..., 1, :], y[..., 0, :] - y[..., 1, :]), -2).reshape(x.shape)
        h *= 2
    return x


def matrix(d: int, signs) -> np.ndarray:
    """R in 64 bits (the identity for signs None)."""
    if signs is None:
        return np.eye(d)
    i = np.arange(d)
    pop = np.array([bin(v).count("1") for v in range(d)])
    return (1.0 - 2.0 * (pop[i[:, None] & i] & 1)) * np.asarray(signs, np.float64) / math.sqrt(d)


def pack(x: np.ndarray, signs):
    """(codes uint8 [.., d / 2], scales float16 [..]) of rows x (float32)."""
    with np.errstate(invalid="ignore"):
        x = np.where(np.isnan(x), np.float32(0), np.clip(x, np.float32(-65504), np.float32(65504))).astype(np.float32)
    d = x.shape[-1]
    if signs is not None:
        x = butterflies(x * np.asarray(signs, np.float32)) * np.float32(1.0 / math.sqrt(d))
    assert x.dtype == np.float32
    m = np.abs(x).max(-1)
    sigma = np.minimum(m / np.float32(7), np.float32(65504)).astype(np.float16)
    with np.errstate(divide="ignore"):
        r = np.where(sigma > 0, np.float32(1) / sigma.astype(np.float32), np.float32(0))
    q = np.clip(np.rint(x.astype(np.float64) * r.astype(np.float64)[..., None]), -7, 7)
    e = (q + 8).astype(np.uint8)
    return e[..., 0::2] | (e[..., 1::2] << 4), sigma


def codes_of(packed: np.ndarray) -> np.ndarray:
    q = np.empty((*packed.shape[:-1], packed.shape[-1] * 2), np.float64)
    q[..., 0::2], q[..., 1::2] = packed & 15, packed >> 4
    return q - 8


@dataclass
class Seqs:
    """A batch on the host."""
    start: np.ndarray    # [n + 1]
    length: np.ndarray   # [n]
    table: np.ndarray    # [n, max_pages]

    def rows(self):
        """(row, sequence, token) of every row that belongs to a sequence."""
        for s in range(len(self.length)):
            lo, hi = int(self.start[s]), int(self.start[s + 1])
            for r in range(lo, hi):
                yield r, s, int(self.length[s]) - (hi - lo) + (r - lo)

    def slot(self, s, tok, page_tokens, n_pages):
        """(page, slot), or None where the page is refused."""
        col = tok // page_tokens
        if col >= self.table.shape[1]:
            return None
        page = int(self.table[s, col])
        return (page, tok % page_tokens) if 0 <= page < n_pages else None


def gather(codes, tok, b: Seqs, s: int, n: int):
    """Stored codes (64 bits) and scales [H, n, d], [H, n] of tokens 0 .. n - 1
    of a sequence, and which of them are there."""
    n_pages, H, T, half = codes.shape
    q, sc, there = np.zeros((H, n, 2 * half)), np.zeros((H, n)), np.zeros(n, bool)
    for t in range(n):
        at = b.slot(s, t, T, n_pages)
        if at is not None:
            q[:, t], sc[:, t], there[t] = codes_of(codes[at[0], :, at[1]]), tok[at[0], :, at[1]], True
    return q, sc, there


def attention(k, v, b: Seqs, q: np.ndarray, signs, scale, causal, window, half_step, only=None,
              many=False):
    """Attention in 64 bits over k, v = (codes, tok), and the bounds of the
    kernels' errors: {row: (out [Hq, d], lse [Hq], out bound, lse bound)}, of
    all rows or of those in `only`.

    Roundings of the kernels, each relative to what it rounds:
      scores  the query keeps 22 bits, the products with codes (exact, 15 is
              counted for their magnitude) are summed in the tensor core
              within 2^-19 of the sum of their magnitudes, or in fp32 (128
              terms: 2^-17 at worst); the scaling and exp2's argument add
              three fp32 roundings of the score.
              delta = 2^-17 sum |q~| 15 sigma scale + 4 2^-24 |score|
      p       exp(score - reference): e^(2 delta) - 1 against the others, the
              exponential itself 2^-21; p sigma_v is rounded to fp16, 2^-12
              (2^-11 is counted)
      values  sum of p sigma_v e, |e| <= 15, again 2^-17 of its magnitudes
      result  half a step of its type
    With `many` (sequences of many rows, whose p sigma_v is scaled by the
    largest score and the largest sigma_v) it is also off by 2^-25 below
    2^-14, of 2^6 or more for those largest: by 2^-31 of the largest sigma_v.
    The rotation back is orthogonal: each element's error is at most the
    2-norm of the errors before it."""
    H, d, Hq = k[0].shape[1], q.shape[2], q.shape[1]
    R, G = matrix(d, signs), Hq // H
    scale = scale if scale > 0 else 1.0 / math.sqrt(d)
    res, cache = {}, {}
    for r, s, pos in b.rows():
        if only is not None and r not in only:
            continue
        n = max(int(b.length[s]), 0)
        if s not in cache:
            cache[s] = (gather(*k, b, s, n), gather(*v, b, s, n))
        (kq, ks, sees), (vq, vs, _) = cache[s]
        if causal:
            t = np.arange(n)
            sees = sees & (t <= pos)
            if window:
                sees &= t > pos - window
        out, lse = np.zeros((Hq, d)), np.full(Hq, -np.inf)
        tol, ltol = np.zeros((Hq, d)), np.zeros(Hq)
        if sees.any():
            qr = q[r].astype(np.float64) @ R.T
            for j in range(Hq):
                g = j // G
                x = scale * ks[g, sees] * (kq[g, sees] @ qr[j])
                mag = scale * 15 * ks[g, sees] * np.abs(qr[j]).sum()
                delta = float(np.max(2.0 ** -17 * mag + 2.0 ** -22 * np.abs(x)))
                m = x.max()
                p = np.exp(x - m)
                l = p.sum()
                o = (p * vs[g, sees]) @ vq[g, sees] / l
                lse[j] = m + math.log(l)
                rel = 2 * delta + 2.0 ** -20 + 2.0 ** -11
                err = rel * ((p * vs[g, sees]) @ np.abs(vq[g, sees])) / l \
                    + 2.0 ** -17 * 15 * float((p * vs[g, sees]).sum()) / l
                if many:
                    err = err + 2.0 ** -31 * vs[g, sees].max() * np.abs(vq[g, sees]).sum(0) / l
                out[j] = o @ R if signs is not None else o
                e2 = np.linalg.norm(err) if signs is not None else err
                tol[j] = e2 + half_step * (np.abs(out[j]) + e2) + 2.0 ** -25
                ltol[j] = delta + 2.0 ** -20 + 2.0 ** -22 * abs(lse[j])
        res[r] = (out, lse, tol, ltol)
    return res
