"""A routed layer around the exact-budget soft gate: who goes where, and back.

The soft gate (``forward``, ``soft_topk``) prices every score of a row so that a
row's prices add up to the budget k.  A routed layer sends each row's k best
scores somewhere -- a token to its experts, or an expert to its tokens -- and
weights what comes back with the prices of the chosen scores.  Every step runs in
the library's kernels (``lapsum_select*``, ``lapsum_route_build``,
``lapsum_dispatch*``, ``lapsum_combine*`` of include/lapsum.h):

    w, idx = soft_gate(scores, k, t)             # prices and indices of the k best per row
    route = route_experts(idx, tokens)           # rows of scores are experts: they choose tokens
    route = route_tokens(idx, experts)           # rows of scores are tokens: they choose experts
    xs = to_experts(x, route)                    # [slots, d]: token rows, sorted by expert
    ...                                          # expert e works on rows expert_offsets[e] .. [e + 1]
    y = from_experts(h, w, route)                # [tokens, d]: weighted and added up per token

``soft_gate``, ``to_experts`` and ``from_experts`` are differentiable; ``select``,
``dispatch``, ``combine`` and their ``*_backward`` are the steps themselves.
Results are the same on every run.  No step keeps a workspace in the library, so
all but ``soft_gate`` (its solver has one per stream) may be captured into graphs
that run side by side.  A captured backward pass needs, as in all of torch, that no
eager graph of the same leaves is alive meanwhile; the ``*_backward`` steps do not.
A step given a ``stream`` runs there and its results belong to it; its inputs have to
live, and to be ready, for that stream (``record_stream``, ``wait_stream``), as in all of
torch.  Tables, rows and lists hold at least one of each: an empty batch is refused.
"""
from __future__ import annotations

import contextlib
import ctypes as C

import torch
from torch.autograd.function import once_differentiable

import exact_budget_soft_b200 as L

TYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}   # LAPSUM_TYPE_*
BY_TOKENS, BY_EXPERTS = 0, 1                                      # LAPSUM_ROUTE_BY_*
MAX_ENTRIES = 2 ** 31 - 1
SHORT = 32768                                                     # rows up to here need no scratch


_HERE = contextlib.nullcontext()


def _on(dev: torch.device, stream):
    """The device, and the stream when one is given, made current for the call: what the
    call allocates belongs to the stream that it runs on."""
    if stream is None:
        return _HERE if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)
    if stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
    return torch.cuda.stream(stream)


def _stream(dev: torch.device) -> int:
    """The current stream's handle: the raw query, a twentieth of current_stream()'s time,
    which would be a fifth of a small call's."""
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _out(given: torch.Tensor | None, shape, dtype, like: torch.Tensor, name: str) -> torch.Tensor:
    if given is None:
        return like.new_empty(shape, dtype=dtype)
    L._need(given, name, dtype, device=like.device)
    if tuple(given.shape) != tuple(shape):
        raise ValueError(f"{name} must have the shape {tuple(shape)}, not {tuple(given.shape)}")
    return given


def _apart(out: torch.Tensor, name: str, *ins: torch.Tensor):
    """No output may share memory with an input: rows are read while others are written."""
    a, b = out.data_ptr(), out.data_ptr() + out.numel() * out.element_size()
    for x in ins:
        if x.data_ptr() < b and a < x.data_ptr() + x.numel() * x.element_size():
            raise ValueError(f"{name} must not overlap an input")


def _scratch(need: int, dev, where: str):
    """(tensor, address, bytes) of a call's own scratch."""
    L._check(min(need, 0), where)
    if not need:
        return None, None, 0
    s = torch.empty(need, dtype=torch.uint8, device=dev)
    return s, s.data_ptr(), need


# ------------------------------------------------------------------- select --
def select(scores: torch.Tensor, k: int, p: torch.Tensor | None = None, idx_out: torch.Tensor | None = None,
           w_out: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """The k largest scores of every row: idx int32 [rows, k], ascending within a row, and,
    with the prices p of the soft gate, w [rows, k] = p at idx (else None).  Ties go to the
    lowest index; -0 equals 0; a NaN is below every number."""
    L._need(scores, "scores")
    rows, n = L._as_rows(scores)
    dev = scores.device
    if isinstance(k, bool) or int(k) != k or not 1 <= k <= n:
        raise ValueError(f"k must be a whole number from 1 to n = {n}, not {k}")
    k = int(k)
    if p is not None:
        L._need(p, "p", numel=rows * n, device=dev)
    elif w_out is not None:
        raise ValueError("w_out needs p")
    with _on(dev, stream):
        idx = _out(idx_out, (rows, k), torch.int32, scores, "idx_out")
        w = _out(w_out, (rows, k), torch.float32, scores, "w_out") if p is not None else None
        if idx_out is not None or w_out is not None:
            _apart(idx, "idx_out", scores, *(x for x in (p, w) if x is not None))
            if w is not None:
                _apart(w, "w_out", scores, p)
        keep, at, size = (None, None, 0) if n <= SHORT else _scratch(L.lib.lapsum_select_scratch(rows, n, k), dev,
                                                                     "lapsum_select")
        L._check(L.lib.lapsum_select(scores.data_ptr(), None if p is None else p.data_ptr(), rows, n, k,
                                     idx.data_ptr(), None if w is None else w.data_ptr(), at, size, _stream(dev)),
                 "lapsum_select")
    return idx, w


def select_backward(scores: torch.Tensor, b: torch.Tensor, idx: torch.Tensor, dw: torch.Tensor, t: float,
                    grad_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The gradient of the soft gate when only its selected prices were used: ``backward``
    for an upstream gradient that is dw at idx (as ``select`` returns it) and zero elsewhere.
    A row whose indices do not ascend within [0, n), or with a NaN score or threshold, gets NaN."""
    L._need(scores, "scores")
    rows, n = L._as_rows(scores)
    dev = scores.device
    if idx.dim() != 2 or idx.shape[0] != rows or not 1 <= idx.shape[1] <= n:
        raise ValueError(f"idx must be [rows, k] with rows = {rows} and k from 1 to {n}")
    k = idx.shape[1]
    L._need(idx, "idx", torch.int32, device=dev)
    L._need(dw, "dw", numel=rows * k, device=dev)
    L._need(b, "b", torch.float64, numel=rows, device=dev)
    with _on(dev, stream):
        grad = _out(grad_out, scores.shape, torch.float32, scores, "grad_out")
        if grad_out is not None:
            _apart(grad, "grad_out", scores, b, idx, dw)
        keep, at, size = (None, None, 0) if n <= SHORT else _scratch(L.lib.lapsum_select_backward_scratch(rows, n), dev,
                                                                     "lapsum_select_backward")
        L._check(L.lib.lapsum_select_backward(scores.data_ptr(), b.data_ptr(), idx.data_ptr(), dw.data_ptr(), rows, n,
                                              k, float(t), grad.data_ptr(), at, size, _stream(dev)),
                 "lapsum_select_backward")
    return grad


class _SoftGate(torch.autograd.Function):
    @staticmethod
    def forward(ctx, scores, k, t, opts):
        scores = scores.contiguous()
        p, b = L.forward(scores, float(k), t, opts=opts)
        idx, w = select(scores, k, p)
        ctx.save_for_backward(scores, b, idx)
        ctx.t = t
        ctx.mark_non_differentiable(idx)
        return w, idx

    @staticmethod
    @once_differentiable
    def backward(ctx, dw, _):
        scores, b, idx = ctx.saved_tensors
        return select_backward(scores, b, idx, dw.float().contiguous(), ctx.t), None, None, None


def soft_gate(scores: torch.Tensor, k: int, t: float, opts: L.Options | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """(w, idx), both [rows, k]: the k best scores of every row and their soft prices, the
    prices differentiable in the scores (the whole row's: the budget ties them together).
    As for ``forward``, the scores are finite and 0 < k < n."""
    return _SoftGate.apply(scores, k, t, opts)


# -------------------------------------------------------------------- route --
class Route:
    """Who goes where: the arrays of ``lapsum_route`` as int32 tensors (read only).

    slot_token, slot_entry [slots]      the token and the entry (row * k + j) of every slot
    expert_offsets [experts + 1]        an expert's first slot
    token_offsets [tokens + 1]          a token's first place in the next two
    token_slots, token_entries [slots]  a token's slots and entries, ascending by entry

    Entries that go nowhere take no slot; the last places then hold -1."""

    __slots__ = ("tokens", "experts", "k", "by", "slots", "device", "c", "_buf", "_views")

    def __init__(self, tokens: int, experts: int, k: int, by: int, device: torch.device):
        n = (tokens if by == BY_TOKENS else experts) * k
        self.tokens, self.experts, self.k, self.by, self.slots, self.device = tokens, experts, k, by, n, device
        # one allocation for the six arrays, cut up when they are asked for: a route is
        # built in every step, and the row passes take the addresses alone
        self._buf = torch.empty(4 * n + experts + tokens + 2, dtype=torch.int32, device=device)
        self._views = None
        at = self._buf.data_ptr()
        self.c = L.RouteArrays(tokens, experts, n, at, at + 4 * n, at + 16 * n, at + 16 * n + 4 * (experts + 1), at + 8 * n,
                               at + 12 * n)

    def arrays(self) -> tuple[torch.Tensor, ...]:
        if self._views is None:
            n = self.slots
            st, se, ts, te, eo, to = self._buf.split((n, n, n, n, self.experts + 1, self.tokens + 1))
            self._views = (st, se, eo, to, ts, te)
        return self._views

    slot_token = property(lambda self: self.arrays()[0])
    slot_entry = property(lambda self: self.arrays()[1])
    expert_offsets = property(lambda self: self.arrays()[2])
    token_offsets = property(lambda self: self.arrays()[3])
    token_slots = property(lambda self: self.arrays()[4])
    token_entries = property(lambda self: self.arrays()[5])


def _route(ids: torch.Tensor, by: int, other: int, stream) -> Route:
    L._need(ids, "ids", torch.int32)
    if ids.dim() != 2 or ids.numel() == 0:
        raise ValueError("ids must be [rows, k], at least one of each")
    if int(other) != other or not 1 <= other < MAX_ENTRIES:
        raise ValueError(f"{'experts' if by == BY_TOKENS else 'tokens'} must be a whole number from 1 on, not {other}")
    rows, k = ids.shape
    other, dev = int(other), ids.device
    if ids.numel() > MAX_ENTRIES:
        raise ValueError("a route holds fewer than 2**31 entries")
    with _on(dev, stream):
        r = Route(rows, other, k, by, dev) if by == BY_TOKENS else Route(other, rows, k, by, dev)
        c = C.byref(r.c)
        keep, s, size = _scratch(L.lib.lapsum_route_scratch(by, k, c), dev, "lapsum_route_build")
        L._check(L.lib.lapsum_route_build(ids.data_ptr(), by, k, c, s, size, _stream(dev)), "lapsum_route_build")
    return r


def route_tokens(ids: torch.Tensor, experts: int, stream=None) -> Route:
    """The route of ids int32 [tokens, k], the experts that every token chose.  An id
    outside [0, experts) goes nowhere (-1 for padding)."""
    return _route(ids, BY_TOKENS, experts, stream)


def route_experts(ids: torch.Tensor, tokens: int, stream=None) -> Route:
    """The route of ids int32 [experts, k], the tokens that every expert chose.  An id
    outside [0, tokens) goes nowhere."""
    return _route(ids, BY_EXPERTS, tokens, stream)


# ----------------------------------------------------------- there and back --
def _rows(x: torch.Tensor, name: str, side: str, route: Route) -> int:
    """The type code of x, a [tokens, d] or [slots, d] tensor on the route's device."""
    if not isinstance(route, Route):
        raise ValueError("route must come from route_tokens or route_experts")
    rows = getattr(route, side)
    code = TYPES.get(x.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32, float16 or bfloat16, not {x.dtype}")
    L._need(x, name, x.dtype, device=route.device)
    if x.dim() != 2 or x.shape[0] != rows or x.shape[1] < 1:
        raise ValueError(f"{name} must be [{rows}, d], not {list(x.shape)}")
    return code


def _weights(w: torch.Tensor, route: Route):
    L._need(w, "w", numel=route.slots, device=route.device)


def dispatch(x: torch.Tensor, route: Route, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """[slots, d]: the token's row of x [tokens, d] in every slot; zero behind the last slot."""
    code = _rows(x, "x", "tokens", route)
    d, dev = x.shape[1], route.device
    with _on(dev, stream):
        y = _out(out, (route.slots, d), x.dtype, x, "out")
        if out is not None:
            _apart(y, "out", x, route._buf)
        L._check(L.lib.lapsum_dispatch(x.data_ptr(), code, d, C.byref(route.c), y.data_ptr(), _stream(dev)),
                 "lapsum_dispatch")
    return y


def dispatch_backward(g: torch.Tensor, route: Route, grad_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The gradient of dispatch: [tokens, d], the sum of g [slots, d] over a token's slots."""
    code = _rows(g, "g", "slots", route)
    d, dev = g.shape[1], route.device
    with _on(dev, stream):
        y = _out(grad_out, (route.tokens, d), g.dtype, g, "grad_out")
        if grad_out is not None:
            _apart(y, "grad_out", g, route._buf)
        L._check(L.lib.lapsum_dispatch_backward(g.data_ptr(), code, d, C.byref(route.c), y.data_ptr(),
                                                _stream(dev)), "lapsum_dispatch_backward")
    return y


def combine(h: torch.Tensor, w: torch.Tensor, route: Route, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """[tokens, d]: the sum over a token's slots of h [slots, d] times the entry's weight
    w (float32, one per entry, in the choosing table's layout)."""
    code = _rows(h, "h", "slots", route)
    _weights(w, route)
    d, dev = h.shape[1], route.device
    with _on(dev, stream):
        y = _out(out, (route.tokens, d), h.dtype, h, "out")
        if out is not None:
            _apart(y, "out", h, w, route._buf)
        L._check(L.lib.lapsum_combine(h.data_ptr(), w.data_ptr(), code, d, C.byref(route.c), y.data_ptr(),
                                      _stream(dev)), "lapsum_combine")
    return y


def combine_backward(h: torch.Tensor, w: torch.Tensor, g: torch.Tensor, route: Route,
                     grad_h: torch.Tensor | None = None, grad_w: torch.Tensor | None = None,
                     stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """The gradients of combine for g [tokens, d]: grad_h [slots, d] (zero behind the last
    slot) and grad_w, like w (zero where an entry went nowhere)."""
    code = _rows(h, "h", "slots", route)
    _weights(w, route)
    if _rows(g, "g", "tokens", route) != code or g.shape[1] != h.shape[1]:
        raise ValueError("g must have the type and the width of h")
    dev = route.device
    with _on(dev, stream):
        gh = _out(grad_h, h.shape, h.dtype, h, "grad_h")
        gw = _out(grad_w, w.shape, torch.float32, w, "grad_w")
        if grad_h is not None or grad_w is not None:
            _apart(gh, "grad_h", h, w, g, gw, route._buf)
            _apart(gw, "grad_w", h, w, g, route._buf)
        L._check(L.lib.lapsum_combine_backward(h.data_ptr(), w.data_ptr(), g.data_ptr(), code, h.shape[1],
                                               C.byref(route.c), gh.data_ptr(), gw.data_ptr(), _stream(dev)),
                 "lapsum_combine_backward")
    return gh, gw


class _ToExperts(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, route):
        ctx.route = route
        return dispatch(x.contiguous(), route)

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        return dispatch_backward(g.contiguous(), ctx.route), None


class _FromExperts(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, w, route):
        h, w = h.contiguous(), w.contiguous()
        ctx.save_for_backward(h, w)
        ctx.route = route
        return combine(h, w, route)

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        h, w = ctx.saved_tensors
        gh, gw = combine_backward(h, w, g.contiguous(), ctx.route)
        return gh, gw, None


def to_experts(x: torch.Tensor, route: Route) -> torch.Tensor:
    """``dispatch``, differentiable in x."""
    return _ToExperts.apply(x, route)


def from_experts(h: torch.Tensor, w: torch.Tensor, route: Route) -> torch.Tensor:
    """``combine``, differentiable in h and w."""
    return _FromExperts.apply(h, w, route)
