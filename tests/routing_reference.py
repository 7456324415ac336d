"""Plain 64-bit definitions of the routing operators, for the tests (numpy, on the host)."""
import numpy as np


def select(scores, k):
    """Ranks by value (descending, NaN last, -0 == 0), ties by index; the first k, ascending."""
    out = np.empty((scores.shape[0], k), np.int32)
    for i, r in enumerate(scores.astype(np.float64)):
        value = np.where(np.isnan(r), -np.inf, r) + 0.0
        order = np.lexsort((np.arange(r.size), -value, np.isnan(r)))
        out[i] = np.sort(order[:k])
    return out


def select_backward(scores, b, idx, dw, t):
    """(gradient, bound of a fp32 evaluation's error) of the gate for dw at idx, 0 elsewhere.

    A density 2^{l2h - |x|} whose exponent is formed in fp32 from r, b = hi + lo and
    log2(e)/t carries at most four roundings of |x| and |l2h| (relative 2^-24 each) and
    exp2's own error (two units): eps_i = 2^-24 (4 ln 2 (|x_i| + |l2h|) + 8).  lambda is a
    quotient of sums of such terms, each thread's share (at most 32 terms) added up in fp32."""
    r, dw = scores.astype(np.float64), dw.astype(np.float64)
    grad, bound = np.empty_like(r), np.empty_like(r)
    u = 2.0 ** -24
    for i in range(r.shape[0]):
        x = np.abs(r[i] - b[i]) / t
        m = x.min()
        e = np.exp(m - x)                      # densities up to a common factor, none lost
        eps = u * (4 * (x / np.log(2) + abs(np.log2(0.5 / t))) * np.log(2) + 8 + 32)
        at = idx[i]
        lam = (dw[i] * e[at]).sum() / e.sum()
        dlam = ((np.abs(dw[i]) * e[at] * eps[at]).sum() + abs(lam) * (e * eps).sum()) / e.sum()
        g = np.zeros_like(x)
        g[at] = dw[i]
        f = np.exp(-x) / (2 * t)
        grad[i] = f * (g - lam)
        bound[i] = 1.01 * f * (np.abs(g - lam) * eps + dlam + u * (np.abs(g) + abs(lam))) + 2.0 ** -126
    return grad, bound


def route(ids, by_tokens, other):
    """The six arrays of a route from nested loops over the table, in entry order."""
    rows, k = ids.shape
    entries = [(e, int(v)) for e, v in enumerate(ids.reshape(-1).tolist()) if 0 <= v < other]
    slots = ids.size
    if by_tokens:
        tokens, experts = rows, other
        order = sorted(entries, key=lambda ev: ev[1])              # stable
        slot_entry = [e for e, _ in order]
        slot_token = [e // k for e in slot_entry]
        expert_of = [v for _, v in order]
    else:
        tokens, experts = other, rows
        slot_entry = [e for e, _ in entries]
        slot_token = [v for _, v in entries]
        expert_of = [e // k for e in slot_entry]
    where = {e: s for s, e in enumerate(slot_entry)}
    token_of = dict(zip(slot_entry, slot_token))
    token_entries = sorted(slot_entry, key=lambda e: (token_of[e], e))
    token_slots = [where[e] for e in token_entries]
    pad = [-1] * (slots - len(entries))
    expert_offsets = np.concatenate([[0], np.cumsum(np.bincount(expert_of, minlength=experts)[:experts])])
    token_offsets = np.concatenate([[0], np.cumsum(np.bincount(slot_token, minlength=tokens)[:tokens])])
    return [np.asarray(v, np.int32) for v in (slot_token + pad, slot_entry + pad, expert_offsets, token_offsets,
                                              token_slots + pad, token_entries + pad)]


def half_step(dtype):
    """Relative rounding of a torch type, and half its smallest subnormal."""
    import torch
    f = torch.finfo(dtype)
    return f.eps / 2, f.smallest_normal * f.eps / 2


ABOUT_ZERO = ["zeros and subnormals", "mostly subnormals", "deep", "both signs", "normals below", "zeros alone"]


def about_zero(kind, n, k, seed=0):
    """A row of zeros of both signs and subnormals: the keys just below zero's.  k - k / 16 of its
    scores (deep: two thirds of k) are zero or more, so that the k-th largest is a negative subnormal."""
    g = np.random.default_rng(seed + n + k)
    tiny = 2.0 ** -149
    top = max(k - max(k // (3 if kind == "deep" else 16), 1), 1)
    r = np.empty(n)
    place = g.permutation(n)
    zero, rest = place[:top], place[top:]
    r[zero] = np.where(g.random(zero.size) < 0.5, 0.0, -0.0)
    if kind == "zeros and subnormals":           # few subnormals, then ordinary scores far below
        r[rest] = -1.0 - g.random(rest.size)
        some = rest[:k - top + (n - k) // 4 + 1]
        r[some] = -tiny * g.integers(1, 1 << 21, some.size)
    elif kind == "mostly subnormals":
        r[rest] = -tiny * g.integers(1, 1 << 23, rest.size)
    elif kind == "deep":
        r[rest] = -tiny * g.integers(1, 4096, rest.size)
    elif kind == "both signs":
        r[zero] = np.where(g.random(zero.size) < 0.5, r[zero], tiny * g.integers(1, 4096, zero.size))
        r[rest] = -tiny * g.integers(1, 4096, rest.size)
    elif kind == "normals below":                # the last subnormals, and normals about the smallest
        r[rest] = -tiny * g.integers((1 << 23) - 2048, (1 << 23) + 2048, rest.size)
    else:
        r[rest] = np.where(g.random(rest.size) < 0.5, 0.0, -0.0)
    return r.astype(np.float32)
