"""The routing steps with outputs of the caller's, at other alignments than the inputs, and
select_backward with several rows a block.

An output's alignment changes how wide it is stored, not what is summed in which order: the
results are the same bits, but for grad_w, whose lanes' shares follow the vectors (a chain of
d / 32 products a lane in fp32, then the lanes: (d / 32 + 24) 2^-24 of the products' sum)."""
import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import routing_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def R():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from exact_budget_soft_b200 import routing
    return routing


class Room:
    """A tensor inside a larger buffer, `off` values past an aligned address; intact() tells
    whether what lies around it is as it was."""

    def __init__(self, shape, dtype, off):
        self.n = int(np.prod(shape))
        self.flat = torch.full((self.n + off + 64,), 77, dtype=dtype, device="cuda")
        self.off, self.t = off, self.flat[off:off + self.n].view(shape)

    def intact(self):
        return bool((self.flat[:self.off] == 77).all() and (self.flat[self.off + self.n:] == 77).all())


@pytest.mark.parametrize("off", [0, 1, 2, 3])
@pytest.mark.parametrize("rows,n,k", [(9, 60, 7), (5, 1000, 100), (5, 1501, 20), (5, 1501, 700), (3, 7000, 50), (3, 20_003, 200),
                                      (3, 20_003, 1100), (2, 20_003, 9000), (2, 50_001, 900)])
def test_select_into_given_outputs(R, rows, n, k, off):
    torch.manual_seed(n)
    r, p = torch.randn(rows, n, device="cuda"), torch.rand(rows, n, device="cuda")
    want, ww = R.select(r, k, p)
    idx, w = Room((rows, k), torch.int32, off), Room((rows, k), torch.float32, (off + 1) % 4)
    got = R.select(r, k, p, idx_out=idx.t, w_out=w.t)
    assert got[0] is idx.t and got[1] is w.t
    assert torch.equal(idx.t, want) and torch.equal(w.t, ww) and idx.intact() and w.intact()
    idx.t.fill_(-5)
    R.select(r, k, idx_out=idx.t)
    assert torch.equal(idx.t, want) and idx.intact()


@pytest.mark.parametrize("off", [1, 2, 3])
@pytest.mark.parametrize("rows,n,k", [(9, 60, 7), (5, 1000, 100), (5, 1501, 20), (4, 4096, 700), (3, 7000, 50), (3, 16_384, 64),
                                      (3, 20_003, 200), (2, 50_001, 900)])
def test_select_backward_into_a_given_output(R, rows, n, k, off):
    torch.manual_seed(n)
    r = torch.randn(rows, n, device="cuda")
    idx, _ = R.select(r, k)
    dw = torch.randn(rows, k, device="cuda")
    b = torch.full((rows,), 1.1, dtype=torch.float64, device="cuda")
    want = R.select_backward(r, b, idx, dw, 0.2)
    out = Room((rows, n), torch.float32, off)
    assert R.select_backward(r, b, idx, dw, 0.2, grad_out=out.t) is out.t
    assert torch.equal(out.t, want) and out.intact()


@pytest.mark.parametrize("rows,n,k", [(9000, 700, 30), (6000, 1501, 20), (4000, 4001, 700), (1500, 8190, 3), (900, 16_001, 200),
                                      (500, 30_003, 400)])
def test_select_backward_several_rows_a_block(R, rows, n, k):
    g = np.random.default_rng(n)
    r = g.standard_normal((rows, n)).astype(np.float32)
    rd = torch.from_numpy(r).cuda()
    idx, _ = R.select(rd, k)
    b = np.sort(r[:, ::7], axis=1)[:, -max(1, k // 7)].astype(np.float64) + 0.013
    dw = g.standard_normal((rows, k)).astype(np.float32)
    got = R.select_backward(rd, torch.from_numpy(b).cuda(), idx, torch.from_numpy(dw).cuda(), 0.1).cpu().numpy()
    want, bound = ref.select_backward(r, b, idx.cpu().numpy(), dw, 0.1)
    assert np.all(np.abs(got - want) <= bound), np.max(np.abs(got - want) / bound)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("off", [1, 2, 4])
@pytest.mark.parametrize("d", [1, 24, 130, 401, 1000, 1001, 2048, 4104])
@pytest.mark.parametrize("by_tokens,tokens,experts,k", [(True, 37, 5, 3), (False, 900, 30, 300), (True, 4200, 8, 2)])
def test_row_passes_into_given_outputs(R, by_tokens, tokens, experts, k, d, off, dtype):
    g = torch.Generator(device="cuda").manual_seed(d)
    rows, other = (tokens, experts) if by_tokens else (experts, tokens)
    ids = torch.randint(-1, other, (rows, k), device="cuda", dtype=torch.int32, generator=g)
    route = R.route_tokens(ids, experts) if by_tokens else R.route_experts(ids, tokens)

    def randn(m):
        return torch.randn(m, d, device="cuda", generator=g).to(dtype)

    x, gx, h, gs, w = randn(tokens), randn(tokens), randn(route.slots), randn(route.slots), torch.randn(rows, k, device="cuda", generator=g)
    for call, shape, name in ((lambda **o: R.dispatch(x, route, **o), (route.slots, d), "out"),
                              (lambda **o: R.dispatch_backward(gs, route, **o), (tokens, d), "grad_out"),
                              (lambda **o: R.combine(h, w, route, **o), (tokens, d), "out")):
        want, out = call(), Room(shape, dtype, off)
        assert call(**{name: out.t}) is out.t
        assert torch.equal(out.t, want) and out.intact(), name
    gh, gw = R.combine_backward(h, w, gx, route)
    oh, ow = Room((route.slots, d), dtype, off), Room((rows, k), torch.float32, off)
    got = R.combine_backward(h, w, gx, route, grad_h=oh.t, grad_w=ow.t)
    assert got[0] is oh.t and got[1] is ow.t and torch.equal(oh.t, gh) and oh.intact() and ow.intact()
    used = int(route.token_offsets[-1])
    token, entry = route.slot_token[:used].long(), route.slot_entry[:used].long()
    prod = h[:used].double() * gx[token].double()
    dot, mass = (torch.zeros(route.slots, dtype=torch.float64, device="cuda") for _ in range(2))
    dot[entry], mass[entry] = prod.sum(1), prod.abs().sum(1)
    for v in (gw, ow.t):
        assert torch.all((v.view(-1).double() - dot).abs() <= 1.001 * ((d / 32 + 24) * U * mass + U * dot.abs()) + 2.0 ** -149)
