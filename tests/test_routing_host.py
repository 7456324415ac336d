"""Refusals of the routing and clipping entry points, found on the host before
anything is enqueued: no GPU is needed, and no pointer is dereferenced."""
import ctypes as C
import os
import subprocess
import sys

import pytest
import torch

import exact_budget_soft_b200 as L
from exact_budget_soft_b200 import grads, routing

F = 0x1000          # never dereferenced
BIG = 1 << 40       # more scratch than any call asks for


def route(tokens=4, experts=3, slots=8, **null):
    a = dict(slot_token=F, slot_entry=F, expert_offsets=F, token_offsets=F, token_slots=F, token_entries=F)
    a.update(null)
    return C.byref(L.RouteArrays(tokens, experts, slots, *a.values()))


@pytest.mark.parametrize("rows,n,k", [(0, 8, 2), (1, 0, 1), (1, 8, 0), (1, 8, 9), (-1, 8, 2), (1, 1 << 31, 2),
                                      (1 << 20, 1 << 20, 1 << 12)])
def test_select_refuses_bad_sizes(rows, n, k):
    assert L.lib.lapsum_select_scratch(rows, n, k) == L.ERR_ARG
    assert L.lib.lapsum_select(F, None, rows, n, k, F, None, F, BIG, None) == L.ERR_ARG
    assert L.lib.lapsum_select_backward(F, F, F, F, rows, n, k, 0.1, F, F, BIG, None) == L.ERR_ARG


def test_select_refuses_null_pointers_and_half_a_pair():
    assert L.lib.lapsum_select(None, None, 1, 8, 2, F, None, F, BIG, None) == L.ERR_ARG
    assert L.lib.lapsum_select(F, None, 1, 8, 2, None, None, F, BIG, None) == L.ERR_ARG
    assert L.lib.lapsum_select(F, F, 1, 8, 2, F, None, F, BIG, None) == L.ERR_ARG
    assert L.lib.lapsum_select(F, None, 1, 8, 2, F, F, F, BIG, None) == L.ERR_ARG
    for null in range(5):
        p = [F] * 5
        p[null] = None
        assert L.lib.lapsum_select_backward(*p[:4], 1, 8, 2, 0.1, p[4], F, BIG, None) == L.ERR_ARG


@pytest.mark.parametrize("t", [0.0, -1.0, float("nan"), float("inf"), 1e-37, 1e37])
def test_select_backward_refuses_bad_temperatures(t):
    assert L.lib.lapsum_select_backward(F, F, F, F, 1, 8, 2, t, F, F, BIG, None) == L.ERR_ARG


@pytest.mark.parametrize("rows,n", [(1, 32769), (3, 100_000), (1, 100_000_000), (5000, 40_000)])
def test_long_rows_need_scratch(rows, n):
    need = L.lib.lapsum_select_scratch(rows, n, 5)
    assert 0 < need < 64 << 20
    assert L.lib.lapsum_select(F, None, rows, n, 5, F, None, None, 0, None) == L.ERR_ARG
    assert L.lib.lapsum_select(F, None, rows, n, 5, F, None, F, need - 1, None) == L.ERR_ARG
    assert L.lib.lapsum_select(F, None, rows, n, 5, F, None, F + 4, need, None) == L.ERR_ARG
    need = L.lib.lapsum_select_backward_scratch(rows, n)
    assert 0 < need < 64 << 20
    assert L.lib.lapsum_select_backward(F, F, F, F, rows, n, 5, 0.1, F, F, need - 1, None) == L.ERR_ARG


@pytest.mark.parametrize("by,k,kw", [(2, 2, {}), (-1, 2, {}), (0, 0, {}), (0, 3, {}), (1, 2, {}), (0, 2, dict(tokens=0)),
                                     (0, 2, dict(experts=0)), (0, 2, dict(slots=9)),
                                     (0, 1 << 16, dict(tokens=1 << 16, slots=1 << 32)),
                                     (0, 2, dict(experts=(1 << 31) - 1))])
def test_route_refuses_bad_sizes(by, k, kw):
    assert L.lib.lapsum_route_scratch(by, k, route(**kw)) == L.ERR_ARG
    assert L.lib.lapsum_route_build(F, by, k, route(**kw), F, BIG, None) == L.ERR_ARG


@pytest.mark.parametrize("name", ["slot_token", "slot_entry", "expert_offsets", "token_offsets", "token_slots",
                                  "token_entries"])
def test_route_refuses_null_arrays(name):
    assert L.lib.lapsum_route_build(F, 0, 2, route(**{name: None}), F, BIG, None) == L.ERR_ARG


def test_route_refuses_missing_scratch_and_ids():
    big = dict(tokens=100_000, experts=3, slots=200_000)
    need = L.lib.lapsum_route_scratch(0, 2, route(**big))
    assert need > 0
    assert L.lib.lapsum_route_build(F, 0, 2, route(**big), None, 0, None) == L.ERR_ARG
    assert L.lib.lapsum_route_build(F, 0, 2, route(**big), F, need - 1, None) == L.ERR_ARG
    assert L.lib.lapsum_route_build(None, 0, 2, route(), F, BIG, None) == L.ERR_ARG
    assert L.lib.lapsum_route_build(F, 0, 2, None, F, BIG, None) == L.ERR_ARG


def test_row_passes_refuse_bad_arguments():
    for kind, d, r in ((3, 8, route()), (-1, 8, route()), (0, 0, route()), (0, 1 << 30, route()), (0, 8, None),
                       (0, 8, route(slots=0)), (0, 8, route(tokens=0)), (0, 8, route(token_slots=None))):
        assert L.lib.lapsum_dispatch(F, kind, d, r, F, None) == L.ERR_ARG
        assert L.lib.lapsum_dispatch_backward(F, kind, d, r, F, None) == L.ERR_ARG
        assert L.lib.lapsum_combine(F, F, kind, d, r, F, None) == L.ERR_ARG
        assert L.lib.lapsum_combine_backward(F, F, F, kind, d, r, F, F, None) == L.ERR_ARG
    assert L.lib.lapsum_dispatch(None, 0, 8, route(), F, None) == L.ERR_ARG
    assert L.lib.lapsum_dispatch(F, 0, 8, route(), F + 2, None) == L.ERR_ARG     # not aligned to its type
    assert L.lib.lapsum_combine(F, None, 0, 8, route(), F, None) == L.ERR_ARG
    for null in range(5):
        p = [F] * 5
        p[null] = None
        assert L.lib.lapsum_combine_backward(*p[:3], 0, 8, route(), p[3], p[4], None) == L.ERR_ARG


def clip(ptrs, sizes, types, max_norm=1.0, outs=None, norm=0x9000, scratch=0x10, have=BIG):
    n = len(ptrs)
    a = (C.c_uint64 * n)(*ptrs)
    o = a if outs is None else (C.c_uint64 * n)(*outs)
    return L.lib.lapsum_clip_grads(n, a, (C.c_int64 * n)(*sizes), (C.c_int32 * n)(*types), max_norm, o, norm, scratch,
                                   have, None)


def test_clip_refuses_bad_arguments():
    assert L.lib.lapsum_clip_scratch(0) == L.ERR_ARG
    assert clip([F], [4], [3]) == L.ERR_ARG                       # type
    assert clip([F], [-1], [0]) == L.ERR_ARG                      # size
    assert clip([F + 2], [4], [0]) == L.ERR_ARG                   # alignment
    assert clip([0], [4], [0]) == L.ERR_ARG                       # null
    assert clip([F], [4], [0], max_norm=-1.0) == L.ERR_ARG
    assert clip([F], [4], [0], max_norm=float("nan")) == L.ERR_ARG
    assert clip([F], [4], [0], norm=None) == L.ERR_ARG
    assert clip([F], [4], [0], scratch=None) == L.ERR_ARG
    assert clip([F], [4], [0], have=8) == L.ERR_ARG


def test_clip_refuses_overlaps():
    assert clip([F, F], [4, 4], [0, 0]) == L.ERR_ARG                          # the same tensor twice, in place
    assert clip([F, F + 8], [4, 4], [0, 0]) == L.ERR_ARG                      # two that overlap, in place
    assert clip([F, F], [4, 4], [0, 0], outs=[0x2000, 0x2008]) == L.ERR_ARG   # outputs that overlap
    assert clip([F], [8], [0], outs=[F + 4]) == L.ERR_ARG                     # an output over its input, shifted
    assert clip([F, 0x2000], [4, 4], [0, 0], outs=[0x2000, F]) == L.ERR_ARG   # outputs over each other's inputs
    assert clip([F], [4], [0], norm=F + 4) == L.ERR_ARG                       # the norm inside a tensor
    assert clip([F, 0x3000, 0x2000], [0x800, 4, 4], [0, 0, 0]) == L.ERR_ARG   # not sorted by address


def test_python_refusals_name_the_argument():
    x = torch.zeros(4, 8)
    for call in (lambda: routing.select(x, 2), lambda: routing.route_tokens(torch.zeros(4, 2, dtype=torch.int32), 3),
                 lambda: grads.clip_grads([x], 1.0)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="route"):
        routing.dispatch(x, None)
    with pytest.raises(ValueError, match="at least one"):
        grads.clip_grads([], 1.0)
    with pytest.raises(ValueError, match="max_norm"):
        grads.clip_grads([x], -1.0)
    with pytest.raises(ValueError, match="outs"):
        grads.clip_grads([x], 1.0, outs=[x, x])


def test_exports_cover_the_routing_calls():
    for name in ("lapsum_select", "lapsum_route_build", "lapsum_dispatch", "lapsum_combine", "lapsum_clip_grads"):
        assert name in L.EXPORTS and getattr(L.lib, name)


def test_waits_give_up_on_request_in_the_checked_build_alone():
    if not L.CHECKED:
        assert L.lib.lapsum_selftest_give_up(0, 1) == L.ERR_ARG
    for wait, row in ((3, 0), (-1, 0), (0, -1)):
        assert L.lib.lapsum_selftest_give_up(wait, row) == L.ERR_ARG


NO_MEMORY = r"""
#include <cstdlib>
#include <new>
static thread_local bool none = false;
extern "C" void no_more_memory(int on) { none = on; }
void *operator new(std::size_t n) {
    void *p = none ? nullptr : std::malloc(n ? n : 1);
    if (!p) throw std::bad_alloc();
    return p;
}
void operator delete(void *p) noexcept { std::free(p); }
void operator delete(void *p, std::size_t) noexcept { std::free(p); }
"""

NO_MEMORY_CALLS = r"""
import ctypes as C, sys
lib, shim = C.CDLL(sys.argv[1]), C.CDLL(None)
i64, vp = C.c_int64, C.c_void_p
for name in ("lapsum_select_scratch", "lapsum_route_scratch"):
    getattr(lib, name).restype = i64
class Route(C.Structure):
    _fields_ = [(n, i64) for n in ("tokens", "experts", "slots")] + [(str(i), vp) for i in range(6)]
F = 0x1000                                     # never dereferenced: nothing can be launched
p, big = vp(F), i64(1 << 40)
r = C.byref(Route(4, 3, 8, F, F, F, F, F, F))
large = C.byref(Route(4000, 3, 8000, F, F, F, F, F, F))
n = lambda *v: [i64(x) for x in v]
calls = {
    "scratch": lambda: lib.lapsum_select_scratch(*n(2, 40000, 5)),
    "select": lambda: lib.lapsum_select(p, None, *n(2, 2000, 5), p, None, p, big, None),
    "long": lambda: lib.lapsum_select(p, None, *n(2, 40000, 5), p, None, p, big, None),
    "backward": lambda: lib.lapsum_select_backward(p, p, p, p, *n(2, 2000, 5), C.c_double(0.1), p, p, big, None),
    "route": lambda: lib.lapsum_route_build(p, C.c_int32(0), i64(2), r, p, big, None),
    "combine": lambda: lib.lapsum_combine(p, p, C.c_int32(0), i64(8), r, p, None),
    "rows": lambda: lib.lapsum_dispatch_backward(p, C.c_int32(0), i64(2048), large, p, None),
}
shim.no_more_memory(1)
code = calls[sys.argv[2]]()
shim.no_more_memory(0)
print("code", code)
"""


@pytest.mark.parametrize("call", ["scratch", "select", "long", "backward", "route", "combine", "rows"])
def test_no_exception_leaves_an_entry_when_host_memory_runs_out(tmp_path, call):
    (tmp_path / "shim.cpp").write_text(NO_MEMORY)
    shim = str(tmp_path / "shim.so")
    subprocess.check_call(["g++", "-O1", "-shared", "-fPIC", "-o", shim, str(tmp_path / "shim.cpp")])
    out = subprocess.run([sys.executable, "-c", NO_MEMORY_CALLS, L.LIB_PATH, call], capture_output=True, text=True, timeout=120,
                         env=dict(os.environ, LD_PRELOAD=shim, CUDA_VISIBLE_DEVICES=""))
    assert out.returncode == 0 and f"code {L.ERR_ALLOC}\n" in out.stdout, (out.returncode, out.stdout, out.stderr[-500:])


def off(at, count, by=2):
    return [F + by if i == at else F for i in range(count)]


def test_addresses_off_their_types_are_refused():
    for at in range(4):
        scores, p, idx, w = off(at, 4)
        assert L.lib.lapsum_select(scores, p, 1, 8, 2, idx, w, F, BIG, None) == L.ERR_ARG
    for at, by in ((0, 2), (1, 2), (1, 4), (2, 2), (3, 2), (4, 2)):
        scores, b, idx, dw, grad = off(at, 5, by)
        assert L.lib.lapsum_select_backward(scores, b, idx, dw, 1, 8, 2, 0.1, grad, F, BIG, None) == L.ERR_ARG
    assert L.lib.lapsum_route_build(F + 2, 0, 2, route(), F, BIG, None) == L.ERR_ARG
    arrays = ("slot_token", "slot_entry", "expert_offsets", "token_offsets", "token_slots", "token_entries")
    for name in arrays:
        assert L.lib.lapsum_route_build(F, 0, 2, route(**{name: F + 2}), F, BIG, None) == L.ERR_ARG
    for name in (arrays[0], *arrays[3:]):          # the arrays that the row passes read
        r = route(**{name: F + 2})
        assert L.lib.lapsum_dispatch(F, 0, 8, r, F, None) == L.ERR_ARG
        assert L.lib.lapsum_dispatch_backward(F, 0, 8, r, F, None) == L.ERR_ARG
        assert L.lib.lapsum_combine(F, F, 0, 8, r, F, None) == L.ERR_ARG
        assert L.lib.lapsum_combine_backward(F, F, F, 0, 8, r, F, F, None) == L.ERR_ARG
    assert L.lib.lapsum_combine(F, F + 2, 0, 8, route(), F, None) == L.ERR_ARG
    assert L.lib.lapsum_combine_backward(F, F + 2, F, 0, 8, route(), F, F, None) == L.ERR_ARG
    assert L.lib.lapsum_combine_backward(F, F, F, 0, 8, route(), F, F + 2, None) == L.ERR_ARG


def test_clip_refuses_a_list_without_a_gradient():
    for none in ([None], [None, None]):
        with pytest.raises(ValueError, match="at least one"):
            grads.clip_grads(none, 1.0)
    with pytest.raises(ValueError, match="outs"):
        grads.clip_grads([None, torch.zeros(3)], 1.0, outs=[torch.zeros(3)])
    with pytest.raises(ValueError, match="CUDA"):
        grads.clip_grads([None, torch.zeros(3)], 1.0)
