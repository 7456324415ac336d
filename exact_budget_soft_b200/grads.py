"""Clipping gradients by their global norm (``lapsum_clip_grads`` of include/lapsum.h).

The soft gate's gradient grows as 1/t, so a step that anneals the temperature
clips.  Two launches whatever the number of tensors (per 512 of them):

    norm = clip_grads([p.grad for p in params], max_norm)           # in place
    norm = clip_grads(grads, max_norm, outs=buffers)                # into other tensors
"""
from __future__ import annotations

from array import array

import torch

import exact_budget_soft_b200 as L
from exact_budget_soft_b200.routing import TYPES, _on, _stream


def _table(xs, name: str, index: int):
    """(sizes, type codes, addresses) of the tensors: a list is walked by mapped calls, since
    at hundreds of tensors a small model's clipping is otherwise the host's time."""
    T = torch.Tensor
    types = [TYPES.get(x.dtype, -1) for x in xs]
    if -1 in types or set(map(T.get_device, xs)) != {index} or not all(map(T.is_contiguous, xs)):
        raise ValueError(f"{name} must be contiguous float32, float16 or bfloat16 tensors on cuda:{index}")
    return array("q", map(T.numel, xs)), array("i", types), array("Q", map(T.data_ptr, xs))


def clip_grads(grads, max_norm: float, outs=None, norm_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """norm = sqrt(sum of all squares) of the tensors in `grads` (float32, float16 or
    bfloat16, contiguous, on one GPU), as a float32 scalar tensor; each is multiplied by
    min(1, max_norm / (norm + 1e-6)) into `outs` (default: in place).  max_norm may be
    infinite: the norm alone.  A None among grads, of a parameter that took no part, is
    skipped (with its place in outs).  The squares of a 16-byte vector are summed in 32 bits, the
    rest in 64, in an order fixed by the sizes and alignments."""
    given = list(grads)
    grads = [g for g in given if g is not None]
    if not grads:
        raise ValueError("grads must hold at least one tensor")
    outs = grads if outs is None else list(outs)
    if outs is not grads:
        if len(outs) != len(given):
            raise ValueError(f"outs must hold {len(given)} tensors, not {len(outs)}")
        if len(grads) != len(given):
            outs = [o for g, o in zip(given, outs) if g is not None]
    if not max_norm >= 0:
        raise ValueError(f"max_norm must be 0 or more, not {max_norm}")
    dev = grads[0].device
    if dev.type != "cuda":
        raise ValueError("grads must be CUDA tensors (there is no CPU path)")
    sizes, types, ins = _table(grads, "grads", dev.index)
    to = ins
    if outs is not grads:
        out_sizes, out_types, to = _table(outs, "outs", dev.index)
        if out_sizes != sizes or out_types != types:
            raise ValueError("outs must have the types and sizes of grads")
    if norm_out is not None:
        L._need(norm_out, "norm_out", numel=1, device=dev)
    with _on(dev, stream):
        norm = torch.empty((), dtype=torch.float32, device=dev) if norm_out is None else norm_out
        need = L.lib.lapsum_clip_scratch(len(grads))
        L._check(min(need, 0), "lapsum_clip_grads")
        scratch = torch.empty(need, dtype=torch.uint8, device=dev)
        L._check(L.lib.lapsum_clip_grads(len(grads), ins.buffer_info()[0], sizes.buffer_info()[0],
                                         types.buffer_info()[0], float(max_norm), to.buffer_info()[0],
                                         norm.data_ptr(), scratch.data_ptr(), need, _stream(dev)),
                 "lapsum_clip_grads")
    return norm
