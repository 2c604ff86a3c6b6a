"""The limits of tests/pages_precision.py tell a right kernel from a wrong one
(CPU only: both are modelled)."""
import numpy as np
import pytest
import torch

import oracle
from tests import pages_precision as prec
from tests import pages_ref as ref


@pytest.fixture(scope="module", params=[(128, 2300), (128, 300), (64, 1100)])
def case(request):
    d, n = request.param
    r = np.random.default_rng(d + n)
    signs = oracle.make_signs(4, d)
    k, v = (ref.pack(r.standard_normal((1, n, d)).astype(np.float32), signs) for _ in range(2))
    k, v = (torch.from_numpy(ref.codes_of(c) * t.astype(np.float64)[..., None]) for c, t in (k, v))
    pos = np.arange(n - 64, n)
    q = torch.from_numpy((1.5 * r.standard_normal((64, 1, d))).astype(np.float16))
    return q, k, v, signs, pos, prec.exact(q, k, v, signs, pos, np.full(64, n))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_the_kernels_roundings_pass(case, dtype):
    q, k, v, signs, pos, want = case
    assert not prec.faults(*prec.modelled(q, k, v, signs, pos, dtype), *want, dtype)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_lost_tokens_values_and_query_bits_do_not(case, dtype):
    q, k, v, signs, pos, want = case
    n = k.shape[1]
    half_page = range(96, 112)
    for wrong in (dict(drop=half_page), dict(silent=half_page), dict(drop=[n - 80]), dict(query_bits=11)):
        assert prec.faults(*prec.modelled(q, k, v, signs, pos, dtype, **wrong), *want, dtype), wrong
    assert not prec.faults(want[0].half(), want[1], *want, "fp16")
