"""select_backward on rows that hold a NaN: both sums of lambda are then NaN, and so is every
value of the row's gradient; other rows stay as they are.  (lapsum_backward does the same for
rows of up to 32768 scores; in longer ones a NaN score marks its own value alone.)"""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def R():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from exact_budget_soft_b200 import routing
    return routing


@pytest.mark.parametrize("n", [1, 40, 129, 1000, 1025, 1500, 3001, 6000, 9001, 20_003, 32_768, 40_001])
@pytest.mark.parametrize("where", ["threshold", "first score", "last score", "middle score", "a selected score", "all scores"])
def test_a_nan_makes_its_row_nan(R, n, where):
    import exact_budget_soft_b200 as L
    torch.manual_seed(n)
    rows, k, t = 5, max(1, n // 50), 0.1
    r = torch.randn(rows, n, device="cuda")
    idx, _ = R.select(r, k)
    dw = torch.randn(rows, k, device="cuda")
    b = torch.full((rows,), 0.7, dtype=torch.float64, device="cuda")
    good = R.select_backward(r, b, idx, dw, t)
    assert torch.isfinite(good).all()
    for row in (1, 4):
        if where == "threshold":
            b[row] = float("nan")
        elif where == "a selected score":
            r[row, idx[row, k // 2].long()] = float("nan")
        else:
            at = {"first score": slice(0, 1), "last score": slice(n - 1, n), "middle score": slice(n // 2, n // 2 + 1),
                  "all scores": slice(0, n)}[where]
            r[row, at] = float("nan")
    got = R.select_backward(r, b, idx, dw, t)
    dense = torch.zeros_like(r).scatter_(1, idx.long(), dw)
    want = torch.isnan(L.backward(r, b, dense, t))
    assert (want[[1, 4]].all() if n <= 32768 else want[[1, 4]].any()) and not want[[0, 2, 3]].any()
    assert torch.isnan(got[[1, 4]]).all(), int(torch.isnan(got).sum())
    assert torch.equal(got[[0, 2, 3]], good[[0, 2, 3]])


@pytest.mark.parametrize("n", [40, 1000, 1500, 20_003, 40_001])
def test_infinite_scores_weigh_nothing(R, n):
    torch.manual_seed(n)
    r = torch.randn(3, n, device="cuda")
    r[1, ::3] = float("-inf")
    r[2, 1::7] = float("inf")
    idx, _ = R.select(torch.randn(3, n, device="cuda"), 9)
    dw = torch.randn(3, 9, device="cuda")
    b = torch.full((3,), 0.7, dtype=torch.float64, device="cuda")
    got = R.select_backward(r, b, idx, dw, 0.1)
    assert torch.isfinite(got).all() and not got[1, ::3].any() and not got[2, 1::7].any()
