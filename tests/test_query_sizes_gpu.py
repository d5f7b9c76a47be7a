"""Queries of any bf16 magnitude over INT4 keys and over prefixes in FP8: the kernels
put each row into f16 by a power of two, so a power of two on the queries and its
inverse on the factor of the scores change no bit of the result."""
import numpy as np
import pytest
import torch

from tests.test_int4_gpu import _run
from tests.test_shared_gpu import make, paged_fp8, ragged_fp8, to_fp8
from workloads import make_small, to_int4

pytestmark = pytest.mark.gpu


def scaled(f, log2):
    q = (f["q"].double() * 2.0 ** log2).to(torch.bfloat16)
    assert torch.equal(q.double(), f["q"].double() * 2.0 ** log2)
    return dict(f, q=q, scale=f["scale"] * 2.0 ** -log2)


@pytest.mark.parametrize("log2", [118, 60, -60, -105])
@pytest.mark.parametrize("hq", [4, 32])   # the column form and the row form
def test_int4_queries_of_any_size(cuda_device, hq, log2):
    f = to_int4(make_small(2, hq, 4, 128, [300, 20], seed=hq))
    want, got = _run(f, cuda_device), _run(scaled(f, log2), cuda_device)
    assert torch.isfinite(want[0]).all()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("log2", [118, 60, -60, -105])
def test_shared_fp8_queries_of_any_size(cuda_device, log2):
    f = to_fp8(make(8, 2, [3, 2], [300, 200], np.full(5, 4)))
    f["sk"] *= 64   # the factor of the scores stays a normal number
    for run in (ragged_fp8, lambda x: paged_fp8(x, 16)):
        want, got = run(f), run(scaled(f, log2))
        assert torch.isfinite(want[0]).all() and got[2] == 0
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
