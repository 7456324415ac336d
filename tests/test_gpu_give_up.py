"""What the routing kernels do when a bounded wait gives up.  The checked build has waits say
so from a block's first or second row on, although the copies have landed
(lapsum_selftest_give_up); rows are then read from memory, with the same results, or marked,
and none is stale.

Each test is one child process, as the checked build is loaded instead of the other."""
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
READ, WRITE, AGAIN = 0, 1, 2
blocks = torch.cuda.get_device_properties(0).multi_processor_count
torch.manual_seed(1)

def given_up(wait, row, call):
    want = [v.clone() for v in call()]
    torch.cuda.synchronize()
    L.selftest_give_up(wait, row)
    got = [v.clone() for v in call()]
    torch.cuda.synchronize()
    L.selftest_give_up(wait, None)
    again = call()
    assert all(torch.equal(a, b) for a, b in zip(again, want))
    return want, got

def selection(rows, n, k, wait, row):
    r, p = torch.randn(rows, n, device="cuda"), torch.rand(rows, n, device="cuda")
    idx, w = torch.empty(rows, k, dtype=torch.int32, device="cuda"), torch.empty(rows, k, device="cuda")
    def call():
        idx.fill_(7)
        w.fill_(0.5)
        return R.select(r, k, p, idx_out=idx, w_out=w)
    want, got = given_up(wait, row, call)
    assert torch.equal(want[0].long(), torch.topk(r, k).indices.sort(dim=1).values)
    marked = (got[0] == -1).any(dim=1)
    assert (got[0][marked] == -1).all() and torch.isnan(got[1][marked]).all()
    assert torch.equal(got[0][~marked], want[0][~marked]) and torch.equal(got[1][~marked], want[1][~marked])
    return marked
"""


def child(code, timeout=300):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    r = subprocess.run([sys.executable, "-c", HEAD + code + "\nprint('as expected')\n"], cwd=ROOT,
                       env=dict(os.environ, LAPSUM_CHECKED="1", PYTHONPATH=ROOT), capture_output=True, text=True, timeout=timeout)
    assert r.returncode == 0 and "as expected" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]


def test_the_selection_goes_on_from_memory():
    child("""
for rows, n, k in ((9000, 1501, 9), (100, 3000, 30), (3000, 7000, 40), (1500, 12003, 100), (700, 30001, 200), (700, 32768, 1100),
                   (9000, 1501, 500), (3000, 7000, 3500), (1500, 12003, 6000), (400, 30001, 15000)):
    for row in (0, 1):
        assert not selection(rows, n, k, READ, row).any(), (n, k, row)
""")


def test_held_rows_whose_copy_is_late_are_marked():
    child("""
for rows, n, k in ((9000, 1501, 500), (3000, 7000, 3500), (1500, 12003, 6000), (400, 30001, 15000)):
    for row in (0, 1):
        L.selftest_give_up(AGAIN, 0)
        marked = selection(rows, n, k, READ, row)
        L.selftest_give_up(AGAIN, None)
        first = int(marked.nonzero()[0])              # the blocks' row-th rows start here
        assert marked[first:].all() and (first > 0) == (row > 0), (n, row, first)
""")


def test_rows_that_nobody_writes_are_marked():
    child("""
for rows, n, k, row in ((700, 30001, 200, 1), (700, 20000, 1, 0), (150, 32768, 256, 0)):
    turn = torch.arange(rows, device="cuda") // blocks
    marked = selection(rows, n, k, WRITE, row)
    assert torch.equal(marked, (turn == row) | (turn == row + 1)), (n, row)      # the rows that had been handed over
""")


def test_the_gradient_goes_on_from_memory():
    child("""
for rows, n, k in ((9000, 1501, 30), (5000, 4000, 200), (2500, 8190, 3), (1000, 12003, 600), (600, 30001, 99)):
    r = torch.randn(rows, n, device="cuda")
    idx, _ = R.select(r, k)
    dw = torch.randn(rows, k, device="cuda")
    b = torch.full((rows,), 1.3, dtype=torch.float64, device="cuda")
    for row in (0, 1):
        want, got = given_up(READ, row, lambda: (R.select_backward(r, b, idx, dw, 0.1),))
        off = (want[0] != got[0]).any(dim=1).nonzero().flatten().tolist()
        assert not off, (n, row, len(off), off[:5])
""")


def test_rows_back_to_tokens_are_marked():
    child("""
for tokens, k, d, dtype in ((9000, 2, 2048, torch.bfloat16), (5000, 3, 1001, torch.float32), (3000, 2, 5001, torch.float16)):
    ids = torch.randint(0, 40, (tokens, k), device="cuda", dtype=torch.int32)
    ids[5] = -1
    route = R.route_tokens(ids, 40)
    h, w = torch.randn(tokens * k, d, device="cuda").to(dtype), torch.rand(tokens, k, device="cuda")
    for call in (lambda: (R.combine(h, w, route),), lambda: (R.dispatch_backward(h, route),)):
        for row in (0, 1):
            want, got = given_up(READ, row, call)
            nan = torch.isnan(got[0])
            assert nan.any() and nan.all() == (row == 0), (d, row)
            assert torch.equal(got[0][~nan], want[0][~nan])
""")
