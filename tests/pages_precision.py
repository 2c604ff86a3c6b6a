"""How exact the paged attention has to be on ordinary inputs: errors against
64 bits as root mean squares, which shrink as rounding errors do when they are
averaged (the worst-case bounds of tests/pages_ref.py do not), and their limits.

What the kernels round, and what a number rounded to within half a step h
(relative) is off by on average, at most h / sqrt 3:
  a token's probability times its value scale, to fp16: 2^-11 / sqrt 3 of each
      term of the sum over tokens; the errors are independent, and the sum of
      zero-mean values has the root mean square of its terms' squares' sum too,
      so this is 2^-11 / sqrt 3 of the output's root mean square
  the output, to its type: h / sqrt 3 of it
  the scores: the rotated query keeps 22 bits, sums are fp32
Limits: both together are sqrt 2 2^-11 / sqrt 3 = 2^-11.3 for fp16 outputs:
2^-11 over all rows, and 2^-9 for one row's d channels (four times as much: a
row's values may cancel); bf16 outputs round 2^-8 / sqrt 3 = 2^-8.8: 2^-8 and
2^-7.  The logarithm of the sum, of magnitude 16 at most here, is itself rounded
to 2^-21 at worst, is made of two approximate functions of 2^-22 each and
of scores of magnitude 32 at most in log2, three fp32 roundings of 2^-20 each of
random sign over the tokens: 2^-19 over all rows, 2^-17 for any one."""
from __future__ import annotations

import math

import numpy as np
import torch

from tests import pages_ref as ref

LIMITS = {"fp16": (2.0 ** -11, 2.0 ** -9), "bf16": (2.0 ** -8, 2.0 ** -7)}
LSE_LIMITS = (2.0 ** -19, 2.0 ** -17)


def stored(s, seq, n):
    """K and V [H, n, d] of a sequence of a test's Setup as they are stored (in
    the rotated domain), 64 bits."""
    out = []
    for i in range(2):
        q, sc, there = ref.gather(s.codes[i], s.tok[i], s.b, seq, n)
        assert there.all()
        out.append(torch.from_numpy(q * sc[..., None]))
    return out


def exact(q, k, v, signs, pos, length, causal=True, window=0, scale=0.0):
    """(out [rows, Hq, d], lse [rows, Hq]) in 64 bits on q's device.  k, v: [H,
    n, d], stored; pos: the rows' tokens; length: the tokens each row's
    sequence has (of the n)."""
    d, H, n = q.shape[2], k.shape[0], k.shape[1]
    dev, G = q.device, q.shape[1] // H
    R = torch.from_numpy(ref.matrix(d, signs)).to(dev)
    k, v = k.to(dev), v.to(dev)
    pos, length = (torch.as_tensor(x, device=dev)[:, None] for x in (pos, length))
    t = torch.arange(n, device=dev)
    sees = (t < length) & ((t <= pos) if causal else (t >= 0))
    if window:
        sees &= t > pos - window
    qr = q.double() @ R.T * (scale if scale > 0 else 1.0 / math.sqrt(d))
    out = torch.empty(q.shape, dtype=torch.float64, device=dev)
    lse = torch.empty(q.shape[:2], dtype=torch.float64, device=dev)
    for j in range(q.shape[1]):
        x = (qr[:, j] @ k[j // G].T).masked_fill(~sees, -math.inf)
        lse[:, j] = torch.logsumexp(x, -1)
        out[:, j] = torch.softmax(x, -1) @ v[j // G] @ R
    return out, lse


def faults(out, lse, want, want_lse, dtype):
    """What is off by more than the limits, in words; empty where all is well."""
    every, row = LIMITS[dtype]
    err, size = (out.double() - want).square(), want.square()
    found = []
    total = float((err.mean() / size.mean()).sqrt())
    if not total <= every:
        found.append(f"outputs: {total:.3g} of their rms, {every:.3g} allowed")
    worst = float((err.mean(-1) / size.mean(-1)).sqrt().max())
    if not worst <= row:
        found.append(f"a row's outputs: {worst:.3g} of their rms, {row:.3g} allowed")
    off = (lse.double() - want_lse).abs()
    if not float(off.square().mean().sqrt()) <= LSE_LIMITS[0]:
        found.append(f"lse: rms {float(off.square().mean().sqrt()):.3g}")
    if not float(off.max()) <= LSE_LIMITS[1]:
        found.append(f"lse: {float(off.max()):.3g}")
    return found


def modelled(q, k, v, signs, pos, dtype, query_bits=22, drop=(), silent=()):
    """The kernels' roundings in a few lines, or a faulty kernel's: the rotated
    query cut to query_bits, weights rounded to fp16, tokens `drop` left out of
    the sums, values of tokens `silent` taken as zero.  One head, causal."""
    d, n = q.shape[2], k.shape[1]
    R = ref.matrix(d, signs)
    x = q[:, 0].double().numpy() @ R.T
    step = 2.0 ** (np.floor(np.log2(np.abs(x).max(-1, keepdims=True))) + 1 - query_bits)
    x = np.rint(x / step) * step / math.sqrt(d)
    t = np.arange(n)
    score = np.where(t <= np.asarray(pos)[:, None], x @ k[0].numpy().T, -np.inf)
    score[:, list(drop)] = -np.inf
    top = score.max(-1, keepdims=True)
    p = np.exp(score - top)
    total = p.sum(-1)
    sigma = np.abs(v[0].numpy()).max(-1) / 7
    w = (p * sigma * 256).astype(np.float16).astype(np.float64) / 256
    w[:, list(silent)] = 0
    out = w @ (v[0].numpy() / sigma[:, None]) / total[:, None] @ R
    kind = {"fp16": torch.float16, "bf16": torch.bfloat16}[dtype]
    return torch.from_numpy(out)[:, None].to(kind), torch.from_numpy(top[:, 0] + np.log(total))[:, None].float()
