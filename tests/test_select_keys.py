"""The key arithmetic of the selection, on the host: csrc/select_keys.cuh is compiled by
itself, and the passes over a long row are restated around it with every index checked,
so that an index past a buffer is a count here and not an access.

Whole numbers throughout: no tolerances."""
import ctypes as C
import os
import subprocess
import sys

import numpy as np
import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import routing_reference as ref  # noqa: E402

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_budget_soft_b200", "csrc")

HARNESS = r"""
#include <algorithm>
#include <vector>
#include "select_keys.cuh"
using namespace lapsum;

extern "C" {

// Pairs (score, range) that a range's bounds and its keys see differently: the range
// holds the keys first .. last, one score's key at least among them.
int64_t disagreements(const uint32_t *ends, int64_t m, const float *scores, int64_t n) {
    int64_t bad = 0;
    for (int64_t i = 0; i < m; ++i)
        for (int64_t j = i; j < m; ++j) {
            const uint32_t first = ends[i], last = ends[j];
            const SelRange r(first, last - first);
            if (r.nan != (first == 0u)) ++bad;
            bool any = false;
            int64_t wrong = 0;
            for (int64_t s = 0; s < n; ++s) {
                const uint32_t key = sel_key(scores[s]);
                any |= key >= first && key <= last;
                if (r.nan) continue;               // such a range's passes compare keys
                const bool from = scores[s] >= r.lo, above = scores[s] > r.hi;
                wrong += from != (key >= first) || (from && above != (key > last));
            }
            if (any) bad += wrong;
        }
    return bad;
}

int32_t key_of(float f) { return (int32_t)sel_key(f); }
int64_t values_that_differ(const float *scores, int64_t n) {
    int64_t bad = 0;
    for (int64_t i = 0; i < n; ++i)
        if (scores[i] == scores[i] && !(sel_value(sel_key(scores[i])) == scores[i])) ++bad;
    return bad;
}

static int clz(uint32_t v) { return v ? __builtin_clz(v) : 32; }

// The passes over one long row: sample, three of histograms, count, emit.  Returns the
// number of indices that would leave their buffers (bins, ties, places of the result).
int64_t long_row(const float *r, int64_t n, int64_t k, int rank_lo, int rank_hi, int32_t *idx, int32_t *route) {
    constexpr int BITS = 11, BINS = 1 << BITS, FEW = 8192, SAMPLE = 2048, TIE = 1 << (32 - 2 * BITS);
    int64_t bad = 0;
    std::vector<uint32_t> key(SAMPLE);
    for (int64_t s = 0; s < SAMPLE; ++s) {
        const int64_t a = s * n / SAMPLE, b = (s + 1) * n / SAMPLE;
        key[s] = sel_key(r[a + (s * 37 & 63) * (b - a) / 64]);
    }
    uint32_t lo = 0u, hi = 0u;
    for (int bit = 31; bit >= 12; --bit) {
        const uint32_t tl = lo | (1u << bit), th = hi | (1u << bit);
        int cl = 0, ch = 0;
        for (uint32_t x : key) { cl += x >= tl; ch += x >= th; }
        if (cl >= rank_lo) lo = tl;
        if (ch >= rank_hi) hi = th;
    }
    hi = rank_hi < 1 ? 0xffffffffu : hi | 0xfffu;
    uint32_t span = hi - lo, shift = (uint32_t)std::max(0, 32 - BITS - clz(span | 1u)), need = (uint32_t)k;
    bool found = false;
    // a score's place against the range, as the kernels ask: below, within, above
    auto side = [&](const SelRange &range, float f) {
        if (range.nan) return sel_key(f) - lo > span ? 1 : 0;
        return !(f >= range.lo) ? -1 : f > range.hi ? 1 : 0;
    };
    for (int pass = 0; pass < 3 && !found; ++pass) {
        std::vector<uint32_t> hist(BINS, 0u);
        const SelRange range(lo, span);
        uint32_t over = 0, total = 0;
        for (int64_t i = 0; i < n; ++i) {
            const int at = side(range, r[i]);
            if (at > 0) ++over;
            if (at) continue;
            const uint32_t bin = (sel_key(r[i]) - lo) >> shift;
            if (bin >= BINS) { ++bad; continue; }
            ++hist[bin];
            ++total;
        }
        if (pass) over = 0;
        if (over >= need || over + total < need) {
            if (pass) return bad + 1;
            lo = 0u;
            span = 0xffffffffu;
            shift = 32 - BITS;
            *route |= 1;                   // the bracket missed
            continue;
        }
        uint32_t want = need - over, c = 0;
        for (int q = BINS - 1; q >= 0; --q) {
            if (c < want && c + hist[q] >= want) {
                const uint32_t bin = (uint32_t)q << shift;
                found = shift == 0u || hist[q] <= FEW;
                lo += bin;
                span = std::min((1u << shift) - 1u, span - bin);
                shift = shift > BITS ? shift - BITS : 0u;
                need = want - c;
                break;
            }
            c += hist[q];
        }
    }
    if (span) {
        const SelRange range(lo, span);
        std::vector<uint32_t> list;
        uint32_t few = 0;
        for (int64_t i = 0; i < n; ++i)
            if (side(range, r[i]) == 0) {
                if (few++ < FEW) list.push_back(sel_key(r[i]));
            }
        uint32_t A = lo, above;
        if (few > FEW) {                   // one block alone
            *route |= 2;
            std::vector<uint32_t> tie(TIE, 0u);
            if (span >= TIE) return bad + 1;
            for (int64_t i = 0; i < n; ++i) {
                const uint32_t d = sel_key(r[i]) - lo;
                if (d <= span) ++tie[d];
            }
            for (int d = (int)span; d >= 0; --d) {
                A = lo + d;
                if (tie[d] >= need) break;
                need -= tie[d];
            }
        } else {
            *route |= 4;
            auto count = [&](uint32_t from) { uint32_t c = 0; for (uint32_t x : list) c += x >= from; return c; };
            for (uint32_t bit = 1u << (31 - clz(span)); bit; bit >>= 1)
                if (bit <= span - (A - lo) && count(A + bit) >= need) A += bit;
            above = A == 0xffffffffu ? 0u : count(A + 1u);
            need -= above;
        }
        lo = A;
    }
    const SelRange range(lo, 0u);
    int64_t o = 0;
    uint32_t equal = 0;
    for (int64_t i = 0; i < n; ++i) {
        bool take;
        if (range.nan) take = sel_key(r[i]) > lo || (sel_key(r[i]) == lo && equal++ < need);
        else take = r[i] > range.lo || (r[i] == range.lo && equal++ < need);
        if (!take) continue;
        if (o >= k) ++bad; else idx[o] = (int32_t)i;
        ++o;
    }
    return bad + (o < k);
}
}
"""


@pytest.fixture(scope="module")
def keys(tmp_path_factory):
    d = tmp_path_factory.mktemp("keys")
    (d / "keys.cpp").write_text(HARNESS)
    so = str(d / "libkeys.so")
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, "-o", so,
                           str(d / "keys.cpp")])
    lib = C.CDLL(so)
    lib.disagreements.restype = lib.values_that_differ.restype = lib.long_row.restype = C.c_int64
    lib.key_of.argtypes = [C.c_float]
    return lib


def ptr(a):
    return a.ctypes.data_as(C.c_void_p)


def border_scores():
    """Every kind of score, and neighbours of each in the last bits."""
    base = np.array([0.0, 2.0 ** -149, 2.0 ** -126, 1e-40, 1e-20, 1.0, 1.5, 3.4028235e38], np.float32)
    at = np.concatenate([base.view(np.uint32).astype(np.int64) + d for d in (-2, -1, 0, 1, 2, 4095, 4096)])
    at = at[(at >= 0) & (at <= 0x7f800000)].astype(np.uint32)
    v = np.concatenate([at, at | np.uint32(0x80000000), np.array([0x7fc00000, 0xffc00000], np.uint32)])
    return np.unique(v).view(np.float32)


def test_keys_order_as_the_scores_do(keys):
    s = border_scores()
    assert keys.values_that_differ(ptr(s), C.c_int64(s.size)) == 0
    k = np.array([keys.key_of(float(v)) & 0xffffffff for v in s])
    real = ~np.isnan(s)
    assert np.all(k[~real] == 0) and np.all(k[real] >= 0x7fffff)
    for v, kv in zip(s[real], k[real]):
        assert np.array_equal(k[real] < kv, s[real] < v) and np.array_equal(k[real] == kv, s[real] == v)
    assert 0x7fffffff not in k                                 # -0 has +0's key, and no score that one


def test_a_range_of_keys_and_its_bounds_are_the_same(keys):
    s = border_scores()
    k = np.array([keys.key_of(float(v)) & 0xffffffff for v in s], np.int64)
    ends = np.concatenate([k + d for d in (-1, 0, 1)] + [k & ~0xfff, k | 0xfff, k & ~0x1fffff, k | 0x1fffff,
                                                         [0, 0x7fffffff, 0x80000000, 0xffffffff]])
    ends = np.unique(ends[(ends >= 0) & (ends <= 0xffffffff)]).astype(np.uint32)
    assert 0x7fffffff in ends
    assert keys.disagreements(ptr(ends), C.c_int64(ends.size), ptr(s), C.c_int64(s.size)) == 0


def ranks(n, k):
    """The bracket's ranks in the sample, as the entry point forms them."""
    mu = k * 2048.0 / n
    sd = np.sqrt(mu)
    lo, hi = int(np.ceil(mu + 4 * sd + 4)), int(np.floor(mu - 4 * sd))
    return lo, 1 if hi < 1 and mu >= 12 else hi


def long_row(keys, r, k):
    idx, route = np.full(k, -1, np.int32), np.zeros(1, np.int32)
    bad = keys.long_row(ptr(r), C.c_int64(r.size), C.c_int64(k), *ranks(r.size, k), ptr(idx), ptr(route))
    return bad, idx, int(route[0])


@pytest.mark.parametrize("kind", ref.ABOUT_ZERO)
@pytest.mark.parametrize("n,k", [(40_000, 38_400), (40_000, 100), (100_000, 60_000), (33_000, 32_999)])
def test_long_rows_about_zero(keys, n, k, kind):
    r = ref.about_zero(kind, n, k)
    bad, idx, _ = long_row(keys, r, k)
    assert bad == 0
    assert np.array_equal(idx, ref.select(r[None], k)[0])


def test_the_restated_passes_on_ordinary_rows(keys):
    g = np.random.default_rng(1)
    seen = 0
    for r in (g.standard_normal(50_000), np.round(g.standard_normal(50_000)), np.zeros(50_000), np.sort(g.standard_normal(50_000)),
              np.where(g.random(50_000) < 0.5, -np.inf, g.standard_normal(50_000)),
              np.where(g.random(50_000) < 0.9, np.nan, 1 + g.integers(0, 64, 50_000) * 2.0 ** -23)):
        for k in (1, 300, 25_000, 50_000):
            r32 = np.ascontiguousarray(r, np.float32)
            bad, idx, route = long_row(keys, r32, k)
            seen |= route
            assert bad == 0 and np.array_equal(idx, ref.select(r32[None], k)[0]), k
    assert seen & 4


@pytest.mark.parametrize("value", [np.nan, -np.inf, np.inf, -0.0, -2.0 ** -149, -3.4028235e38])
@pytest.mark.parametrize("others", [0, 1, 40])
def test_long_rows_of_one_value(keys, value, others):
    r = np.full(40_000, value, np.float32)
    r[np.random.default_rng(1).integers(0, r.size, others)] = 1.0
    for k in (1, 30, 20_000, 40_000):
        bad, idx, _ = long_row(keys, r, k)
        assert bad == 0 and np.array_equal(idx, ref.select(r[None], k)[0]), k
