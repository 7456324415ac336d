"""What the routing kernels do when a bounded wait gives up.  The checked build has waits say
so from a block's second row on, although the copies have landed (lapsum_selftest_give_up);
rows are then read from memory, with the same results, or marked, and none is stale.

Each case runs in a child process, as the checked build is loaded instead of the other."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

HEAD = """
import torch
import exact_budget_soft_b200 as L
from exact_budget_soft_b200 import routing as R
assert L.CHECKED
READ, WRITE = 0, 1
torch.manual_seed(1)

def given_up(wait, row, call):
    want = call()
    torch.cuda.synchronize()
    L.selftest_give_up(wait, row)
    got = call()
    torch.cuda.synchronize()
    L.selftest_give_up(wait, None)
    again = call()
    assert all(torch.equal(a, b) for a, b in zip(again, want))
    return want, got
"""


def child(code, *values):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    r = subprocess.run([sys.executable, "-c", HEAD + code.format(*values) + "\nprint('as expected')\n"], cwd=ROOT,
                       env=dict(os.environ, LAPSUM_CHECKED="1", PYTHONPATH=ROOT), capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "as expected" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]


SELECTION = """
rows, n, k, row = {}, {}, {}, {}
r = torch.randn(rows, n, device="cuda")
p = torch.rand(rows, n, device="cuda")
want, got = given_up(READ, row, lambda: R.select(r, k, p))
assert torch.equal(want[0].long(), torch.topk(r, k).indices.sort(dim=1).values)
assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
"""


@pytest.mark.parametrize("rows,n,k", [(9000, 1501, 9), (100, 3000, 30), (3000, 7000, 40), (1500, 12_003, 100), (700, 30_001, 200),
                                      (700, 32_768, 1100), (400, 20_000, 1500)])
@pytest.mark.parametrize("row", [0, 1])
def test_the_selection_goes_on_from_memory(rows, n, k, row):
    child(SELECTION, rows, n, k, row)


WRITING = """
rows, n, k, row = {}, {}, {}, {}
r = torch.randn(rows, n, device="cuda")
p = torch.rand(rows, n, device="cuda")
idx, w = torch.empty(rows, k, dtype=torch.int32, device="cuda"), torch.empty(rows, k, device="cuda")

def call():
    idx.fill_(7)
    w.fill_(0.5)
    R.select(r, k, p, idx_out=idx, w_out=w)
    return idx.clone(), w.clone()

want, got = given_up(WRITE, row, call)
marked = (got[0] == -1).any(dim=1)
blocks = torch.cuda.get_device_properties(0).multi_processor_count
turn = torch.arange(rows, device="cuda") // blocks
assert torch.equal(marked, (turn == row) | (turn == row + 1))      # the rows that had been handed over
assert (got[0][marked] == -1).all() and torch.isnan(got[1][marked]).all()
assert torch.equal(got[0][~marked], want[0][~marked]) and torch.equal(got[1][~marked], want[1][~marked])
"""


@pytest.mark.parametrize("rows,n,k,row", [(700, 30_001, 200, 1), (700, 20_000, 1, 0), (150, 32_768, 256, 0)])
def test_rows_that_nobody_writes_are_marked(rows, n, k, row):
    child(WRITING, rows, n, k, row)


GRADIENT = """
rows, n, k, row = {}, {}, {}, {}
r = torch.randn(rows, n, device="cuda")
idx, _ = R.select(r, k)
dw = torch.randn(rows, k, device="cuda")
b = torch.full((rows,), 1.3, dtype=torch.float64, device="cuda")
want, got = given_up(READ, row, lambda: (R.select_backward(r, b, idx, dw, 0.1),))
off = (want[0] != got[0]).any(dim=1).nonzero().flatten().tolist()
assert not off, (len(off), off[:5])
"""


@pytest.mark.parametrize("rows,n,k", [(9000, 1501, 30), (5000, 4000, 200), (2500, 8190, 3), (1000, 12_003, 600), (600, 30_001, 99)])
@pytest.mark.parametrize("row", [0, 1])
def test_the_gradient_goes_on_from_memory(rows, n, k, row):
    child(GRADIENT, rows, n, k, row)
