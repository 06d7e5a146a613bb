"""The relative bias's gradient on the GPU: sums of the groups of a workgroup."""

import pytest
import torch

import distributed_sgd_gradient_amd as A
from conftest import flush_print
from test_layers_gpu import DTYPES, F16, F32, ids

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("queries,keys", [(64, 300), (64, 64), (80, 400), (100, 100), (160, 40)])
def test_groups_are_joined_in_fp64(gpu, queries, keys, dtype):
    """2^25 in a diagonal's first rows and a one for each other group of lanes: the
    workgroup's sum is rounded once, and every other value is zero."""
    flush_print(f"groups of {queries}x{keys} {dtype}")
    large, one = (2.0 ** 15, 2.0 ** -10) if dtype == F16 else (2.0 ** 25, 1.0)
    ds = torch.zeros(1, 1, queries, keys, dtype=dtype, device="cuda")
    ds[0, 0, 2, 2] = large
    ones = 0
    for i in range(16, min(queries, keys), 16):
        ds[0, 0, i, i] = one
        ones += 1
    got = A.relative_bias_grad(ds, 32, dtype=F32)
    want = torch.zeros(32, 1)
    want[0] = torch.tensor(large + ones * one, dtype=torch.float64).float()
    assert ones >= 2 and torch.equal(got.cpu(), want)
