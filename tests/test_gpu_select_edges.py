"""select at the borders of its keys, on the GPU: zeros of both signs among subnormals, where
neighbouring keys are not neighbouring scores (tests/test_select_keys.py has the arithmetic).

Indices are whole numbers and weights are copies: both are equal."""
import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import routing_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def R():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from exact_budget_soft_b200 import routing
    return routing


@pytest.mark.parametrize("kind", ref.ABOUT_ZERO)
@pytest.mark.parametrize("n,k", [(60, 20), (1000, 400), (1500, 20), (1500, 900), (6000, 5000), (20_000, 150), (20_000, 15_000),
                                 (40_000, 38_400), (40_000, 100), (100_000, 60_000), (33_000, 32_999), (1_000_003, 400_000)])
def test_select_about_zero(R, n, k, kind):
    r = np.stack([ref.about_zero(kind, n, k, seed) for seed in (1, 2)])
    p = torch.rand(2, n, device="cuda")
    idx, w = R.select(torch.from_numpy(r).cuda(), k, p)
    assert np.array_equal(idx.cpu().numpy(), ref.select(r, k))
    assert torch.equal(w, p.gather(1, idx.long()))


@pytest.mark.parametrize("value", [float("nan"), float("-inf"), float("inf"), -0.0, -2.0 ** -149, -3.4028235e38])
@pytest.mark.parametrize("n,ks", [(1, [1]), (50, [1, 9, 50]), (1000, [3, 500]), (1500, [9, 700]), (6000, [30, 6000]),
                                  (16_000, [100, 5000]), (20_000, [150, 15_000]), (40_000, [1, 30, 20_000, 40_000])])
def test_select_rows_of_one_value(R, n, ks, value):
    # a row that a mask leaves empty, one that it leaves a score or a few, and an ordinary one
    g = np.random.default_rng(n)
    r = np.full((4, n), value, np.float32)
    r[1, g.integers(0, n)] = 1.0
    r[2, g.integers(0, n, 1 + n // 100)] = 1.0
    r[3] = g.standard_normal(n)
    p = torch.rand(4, n, device="cuda")
    for k in ks:
        idx, w = R.select(torch.from_numpy(r).cuda(), k, p)
        assert np.array_equal(idx.cpu().numpy(), ref.select(r, k)), k
        assert torch.equal(w, p.gather(1, idx.long()))
