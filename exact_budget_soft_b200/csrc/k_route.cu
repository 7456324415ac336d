// k_route.cu -- tokens sorted by expert, and the way back.
//
// The entries of a choosing table (entry = row k + j) that go somewhere are
// ranked twice: by entry (the row's side: a running count) and, stably, by id
// (the bin's side: a counting sort, one pass per digit of the id).  Both ranks of
// every entry give all arrays of a route:
//   tokens chose   slot = rank by expert, a token's places = ranks by entry
//   experts chose  slot = rank by entry,  a token's places = ranks by token
//
// A pass over digits: every block counts the digits of its contiguous share; the
// next launch adds up, per digit, the blocks before and all smaller digits, ranks
// its own entries in order (a warp ranks 32 at a time by the lanes that share
// a digit) and writes, a further pass's counts among it.  Ids of up to ROUTE_BITS
// bits take one pass; a table that one block holds takes one launch in all.  Bound by
// the chain of L2 latencies: 65536 x 4 choices of 128 experts 21 us, 1024 x 256 of
// 32768 tokens 30 us, the bytes alone 0.8 us.
#include <algorithm>

#include "lapsum_kernels.h"
#include "lapsum_launch.h"
#include "route_common.cuh"

namespace lapsum {
namespace {

constexpr int RT = 512;                    // threads
constexpr int RW = RT / 32;
constexpr int R_IPT = 4;                   // entries a thread holds of a tile
constexpr int R_TILE = RT * R_IPT;
constexpr int ROUTE_BITS = 10;
constexpr int R_MAX_BINS = 1 << ROUTE_BITS;
constexpr int R_MAX_BLOCKS = 128;

struct RouteArgs {
    const int32_t *ids;
    int64_t k, entries, bins;
    int32_t *slot_token, *slot_entry, *token_slots, *token_entries;
    int32_t *row_offsets, *bin_offsets;
    int64_t rows;
    int by_tokens;
    int blocks, tiles;                     // tiles: of each block
    int32_t *tops;                         // first place of every digit of the last pass, and the end
    uint32_t *counts;                      // [pass][block][R_MAX_BINS + 1]: digits, then entries that go somewhere
    int32_t *key[2], *entry[2], *rank[2];  // entries between passes, and the sorted keys after the last
};

struct RoutePass {
    int pass, passes, shift, bits;
};

// What a thread sees of entry i in this pass: its id, or -1 when it goes nowhere
// or does not exist.  The first pass reads the table, a later one the entries
// that the pass before has sorted (`total` of them).
__device__ __forceinline__ int32_t route_key(const RouteArgs &A, const RoutePass &P, int64_t i, int64_t total) {
    if (i >= total) return -1;
    if (P.pass) return A.key[(P.pass - 1) & 1][i];
    const int32_t v = A.ids[i];
    return v >= 0 && v < A.bins ? v : -1;
}

__device__ __forceinline__ uint32_t *route_counts(const RouteArgs &A, int pass, int block) {
    return A.counts + ((int64_t)pass * R_MAX_BLOCKS + block) * (R_MAX_BINS + 1);
}

// Entries that go somewhere, over all blocks, and in the blocks before `block` (by
// every warp: a lane a block).
__device__ __forceinline__ uint32_t route_total(const RouteArgs &A, int block, uint32_t &before) {
    const int lane = threadIdx.x & 31;
    uint32_t t = 0, b = 0;
#pragma unroll
    for (int q = 0; q < R_MAX_BLOCKS / 32; ++q) {
        const int c = q * 32 + lane;
        const uint32_t v = __ldcg(route_counts(A, 0, min(c, A.blocks - 1)) + R_MAX_BINS);
        t += c < A.blocks ? v : 0u;
        b += c < block ? v : 0u;
    }
    before = __reduce_add_sync(FULL, b);
    return __reduce_add_sync(FULL, t);
}

__global__ void __launch_bounds__(RT) route_count_kernel(RouteArgs A, RoutePass P) {
    __shared__ uint32_t s_hist[R_MAX_BINS];
    __shared__ uint32_t s_valid;
    pdl_enter();
    const int bins = 1 << P.bits;
    for (int d = threadIdx.x; d < bins; d += RT) s_hist[d] = 0u;
    if (threadIdx.x == 0) s_valid = 0u;
    __syncthreads();
    const int64_t a = (int64_t)blockIdx.x * A.tiles * R_TILE;
    const int64_t b = min(a + (int64_t)A.tiles * R_TILE, A.entries);
    unsigned valid = 0;
#pragma unroll 8
    for (int64_t i = a + threadIdx.x; i < b; i += RT) {
        const int32_t v = route_key(A, P, i, A.entries);
        if (v >= 0) {
            atomicAdd(&s_hist[((uint32_t)v >> P.shift) & (bins - 1)], 1u);
            ++valid;
        }
    }
    valid = __reduce_add_sync(FULL, valid);
    if ((threadIdx.x & 31) == 0 && valid) atomicAdd(&s_valid, valid);
    __syncthreads();
    uint32_t *out = route_counts(A, 0, blockIdx.x);
    for (int d = threadIdx.x; d < bins; d += RT) out[d] = s_hist[d];
    if (threadIdx.x == 0) out[R_MAX_BINS] = s_valid;
    for (int pass = 1; pass < P.passes; ++pass)   // added to by the pass before
        for (int d = threadIdx.x; d < bins; d += RT) route_counts(A, pass, blockIdx.x)[d] = 0u;
}

// (sum before this thread, sum of all) over the CTA.
__device__ __forceinline__ uint32_t route_scan(uint32_t v, uint32_t *s_warp, uint32_t &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(FULL, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    const uint32_t w = lane < RW ? s_warp[lane] : 0u;
    total = __reduce_add_sync(FULL, w);
    const uint32_t before = incl - v + __reduce_add_sync(FULL, lane < warp ? w : 0u);
    __syncthreads();
    return before;
}

// Ranks and writes.  With one block and one tile the counts of this very launch
// are all there is (`alone`): no launch before it.  A tile's entries pass through
// shared memory in the order of their digits, so that what is written by place goes
// out in runs; what is written by entry goes out as it comes.
__global__ void __launch_bounds__(RT) route_place_kernel(RouteArgs A, RoutePass P, int alone) {
    constexpr int PD = R_MAX_BINS / RT;    // digits of a thread at most
    extern __shared__ uint32_t s_dyn[];    // [RW][bins] of the warps; [bins] first places, of the block and of the tile
    __shared__ uint32_t s_scan[RW], s_wv[RW], s_tot[RT], s_before[RT];
    __shared__ uint32_t s_pos[R_TILE];
    __shared__ int32_t s_key[R_TILE], s_entry[R_TILE], s_rank[R_TILE];
    const int bins = 1 << P.bits;
    uint32_t *s_w = s_dyn, *s_base = s_dyn + RW * bins, *s_local = s_base + bins;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned below = lanes_below(lane);
    const int pd = max(1, bins / RT);      // digits of a thread: [t pd, (t + 1) pd)
    const bool first_pass = P.pass == 0, last_pass = P.pass == P.passes - 1;
    pdl_enter();
    int32_t key[R_IPT];                    // of the tile at hand: the first one is on its way while the counts are
    const int64_t a = (int64_t)blockIdx.x * A.tiles * R_TILE, stop = min(a + (int64_t)A.tiles * R_TILE, A.entries);
    auto fetch = [&](int64_t t0) {
#pragma unroll
        for (int j = 0; j < R_IPT; ++j) key[j] = route_key(A, P, t0 + warp * 32 * R_IPT + j * 32 + lane, stop);
    };
    fetch(a);
    uint32_t all = 0;                      // entries that go somewhere
    uint32_t valid_at = 0;                 // those before this tile (first pass)
    // the block's first place of every digit: smaller digits of all blocks, this
    // digit of the blocks before
    auto bases = [&](const uint32_t (&tot)[PD], const uint32_t (&before)[PD]) {
        uint32_t mine = 0, total;
#pragma unroll
        for (int q = 0; q < PD; ++q) mine += tot[q];
        uint32_t at = route_scan(mine, s_scan, total);
#pragma unroll
        for (int q = 0; q < PD; ++q) {
            const int d = threadIdx.x * pd + q;
            if (q >= pd || d >= bins) continue;
            s_base[d] = at + before[q];
            if (last_pass && blockIdx.x == 0) {
                if (P.passes > 1) {
                    A.tops[d] = (int32_t)at;
                    if (d == bins - 1) A.tops[bins] = (int32_t)(at + tot[q]);
                } else {
                    if (d <= (int)A.bins) A.bin_offsets[d] = (int32_t)at;
                    if (d == bins - 1) A.bin_offsets[A.bins] = (int32_t)(at + tot[q]);
                }
            }
            at += tot[q];
        }
        __syncthreads();
    };
    if (!alone) {
        all = route_total(A, blockIdx.x, valid_at);
        uint32_t tot[PD] = {}, before[PD] = {};
        const uint32_t *counts = route_counts(A, P.pass, 0);
        auto sum = [&](int d, int from, int step, uint32_t &t, uint32_t &b) {
#pragma unroll 32
            for (int c = from; c < A.blocks; c += step) {
                const uint32_t v = __ldcg(counts + (size_t)c * (R_MAX_BINS + 1) + d);
                b += c < (int)blockIdx.x ? v : 0u;
                t += v;
            }
        };
        if (bins >= RT) {
            for (int q = 0; q < pd; ++q) sum(threadIdx.x * pd + q, 0, 1, tot[q], before[q]);
        } else {                           // several threads share a digit's sum
            const int groups = RT / bins;
            uint32_t t = 0, b = 0;
            sum(threadIdx.x & (bins - 1), threadIdx.x >> P.bits, groups, t, b);
            s_tot[threadIdx.x] = t;
            s_before[threadIdx.x] = b;
            __syncthreads();
            if ((int)threadIdx.x < bins)
                for (int g = 0; g < groups; ++g) {
                    tot[0] += s_tot[g * bins + threadIdx.x];
                    before[0] += s_before[g * bins + threadIdx.x];
                }
        }
        bases(tot, before);
    }
    const int64_t total = first_pass ? A.entries : (int64_t)all;
    const int64_t b = min(stop, total);
    for (int64_t t0 = a; t0 < b; t0 += R_TILE) {
        for (int d = threadIdx.x; d < RW * bins; d += RT) s_w[d] = 0u;
        __syncthreads();
        const int64_t first = t0 + warp * 32 * R_IPT;
        uint32_t rank[R_IPT], vrank[R_IPT];
        uint32_t *mine = s_w + warp * bins;
        uint32_t wv = 0;
        if (t0 != a) fetch(t0);
#pragma unroll
        for (int j = 0; j < R_IPT; ++j) {
            if (first + j * 32 + lane >= b) key[j] = -1;   // (a later pass: behind the entries that go somewhere)
            const unsigned ok = __ballot_sync(FULL, key[j] >= 0);
            vrank[j] = wv + __popc(ok & below);
            wv += __popc(ok);
            const uint32_t d = ((uint32_t)key[j] >> P.shift) & (bins - 1);
            unsigned peers = ok;           // the lanes of this digit, by its bits (a match instruction took ten times as long)
            for (int bit = 0; bit < P.bits; ++bit) {
                const bool one = (d >> bit) & 1;
                const unsigned m = __ballot_sync(FULL, one);
                peers &= one ? m : ~m;
            }
            if (key[j] >= 0) rank[j] = mine[d] + __popc(peers & below);
            __syncwarp();
            if (key[j] >= 0 && (peers & below) == 0) mine[d] += __popc(peers);
            __syncwarp();
        }
        if (lane == 0) s_wv[warp] = wv;
        __syncthreads();
        // the warps' places within a digit; the digits' within the tile, and the next tile's
        uint32_t count[PD] = {}, sum = 0, staged;
#pragma unroll
        for (int q = 0; q < PD; ++q) {
            const int d = threadIdx.x * pd + q;
            if (q >= pd || d >= bins) continue;
            uint32_t c[RW], at = 0;
#pragma unroll
            for (int w = 0; w < RW; ++w) c[w] = s_w[w * bins + d];
#pragma unroll
            for (int w = 0; w < RW; ++w) {
                s_w[w * bins + d] = at;
                at += c[w];
            }
            count[q] = at;
            sum += at;
        }
        uint32_t local = route_scan(sum, s_scan, staged);
        if (alone) {
            const uint32_t none[PD] = {};
            bases(count, none);
        }
#pragma unroll
        for (int q = 0; q < PD; ++q) {
            const int d = threadIdx.x * pd + q;
            if (q >= pd || d >= bins) continue;
            s_local[d] = local;
            local += count[q];
        }
        const uint32_t wc = lane < RW ? s_wv[lane] : 0u;
        const uint32_t v0 = valid_at + __reduce_add_sync(FULL, lane < warp ? wc : 0u);
        valid_at += __reduce_add_sync(FULL, wc);
        __syncthreads();
        const int src = (P.pass - 1) & 1, dst = P.pass & 1;
#pragma unroll
        for (int j = 0; j < R_IPT; ++j) {
            const int64_t i = first + j * 32 + lane;
            if (i >= b) continue;
            const uint32_t seen = v0 + vrank[j];           // first pass: rank by entry
            if (first_pass) {
                const uint32_t row = (uint32_t)i / (uint32_t)A.k;
                if ((uint32_t)i == row * (uint32_t)A.k) A.row_offsets[row] = (int32_t)seen;
            }
            if (key[j] < 0) continue;
            const uint32_t d = ((uint32_t)key[j] >> P.shift) & (bins - 1);
            const uint32_t in = mine[d] + rank[j], pos = s_base[d] + in, at = s_local[d] + in;
            const int32_t e = first_pass ? (int32_t)i : A.entry[src][i];
            const int32_t re = first_pass ? (int32_t)seen : A.rank[src][i];
            s_pos[at] = pos;
            s_key[at] = key[j];
            s_entry[at] = e;
            s_rank[at] = re;
            if (first_pass) {              // by entry
                if (A.by_tokens) {
                    A.token_entries[re] = e;
                } else {
                    A.slot_token[re] = key[j];
                    A.slot_entry[re] = e;
                }
            }
            if (last_pass && A.by_tokens) A.token_slots[re] = (int32_t)pos;
        }
        __syncthreads();
        for (uint32_t z = threadIdx.x; z < staged; z += RT) {   // by place
            const uint32_t pos = s_pos[z];
            const int32_t k = s_key[z], e = s_entry[z], re = s_rank[z];
            if (!last_pass) {
                A.key[dst][pos] = k;
                A.entry[dst][pos] = e;
                A.rank[dst][pos] = re;
                // the next pass's counts: of the block that will hold this entry
                const uint32_t next = ((uint32_t)k >> (P.shift + P.bits)) & (bins - 1);
                atomicAdd(route_counts(A, P.pass + 1, (int)(pos / (uint32_t)(A.tiles * R_TILE))) + next, 1u);
                continue;
            }
            if (P.passes > 1) A.key[dst][pos] = k;   // for the offsets
            if (A.by_tokens) {
                A.slot_token[pos] = (int32_t)((uint32_t)e / (uint32_t)A.k);
                A.slot_entry[pos] = e;
            } else {
                A.token_slots[pos] = re;
                A.token_entries[pos] = e;
            }
        }
        // the next tile's first places
#pragma unroll
        for (int q = 0; q < PD; ++q) {
            const int d = threadIdx.x * pd + q;
            if (q < pd && d < bins) s_base[d] += count[q];
        }
        __syncthreads();
    }
    if (!first_pass) return;
    if (alone) all = valid_at;
    // behind the last slot: -1; the row side's end
    const int64_t end = min(a + (int64_t)A.tiles * R_TILE, A.entries);
    for (int64_t i = max(a, (int64_t)all) + threadIdx.x; i < end; i += RT)
        A.slot_token[i] = A.slot_entry[i] = A.token_slots[i] = A.token_entries[i] = -1;
    if (blockIdx.x == 0 && threadIdx.x == 0) A.row_offsets[A.rows] = (int32_t)all;
}

// After several passes: a bin's first place, by bisection of the sorted keys that
// share its highest digit.
__global__ void __launch_bounds__(256) route_offsets_kernel(RouteArgs A, int last, int shift, int bits) {
    pdl_enter();
    const int64_t d = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (d > A.bins) return;
    const int32_t *key = A.key[last];
    const int top = (int)min(d >> shift, int64_t(1) << bits);
    int32_t lo = A.tops[top], hi = A.tops[min(top + 1, 1 << bits)];
    while (lo < hi) {
        const int32_t mid = lo + ((hi - lo) >> 1);
        if (key[mid] < d) lo = mid + 1; else hi = mid;
    }
    A.bin_offsets[d] = lo;
}

struct RoutePlan {
    int64_t rows, bins;
    int passes, bits, blocks, tiles;
    bool alone;
    size_t scratch;
};

bool route_plan(int32_t by, int64_t k, const lapsum_route *R, RoutePlan *out) {
    const int64_t lim = int64_t(1) << 31;
    if (!R || (by != LAPSUM_ROUTE_BY_TOKENS && by != LAPSUM_ROUTE_BY_EXPERTS)) return false;
    if (k < 1 || R->tokens < 1 || R->experts < 1 || R->tokens >= lim - 1 || R->experts >= lim - 1 || k >= lim) return false;
    const int64_t rows = by == LAPSUM_ROUTE_BY_TOKENS ? R->tokens : R->experts;
    if (rows * k >= lim || R->slots != rows * k) return false;
    out->rows = rows;
    out->bins = by == LAPSUM_ROUTE_BY_TOKENS ? R->experts : R->tokens;
    int bits = 1;
    while ((int64_t(1) << bits) < out->bins) ++bits;
    out->passes = (bits + ROUTE_BITS - 1) / ROUTE_BITS;
    out->bits = (bits + out->passes - 1) / out->passes;
    const int64_t tiles = (R->slots + R_TILE - 1) / R_TILE;
    out->blocks = (int)std::min<int64_t>(tiles, R_MAX_BLOCKS);
    out->tiles = (int)((tiles + out->blocks - 1) / out->blocks);
    out->blocks = (int)((tiles + out->tiles - 1) / out->tiles);
    out->alone = out->passes == 1 && tiles == 1;
    out->scratch = out->alone ? 0 : (size_t)out->passes * R_MAX_BLOCKS * (R_MAX_BINS + 1) * 4;
    if (out->passes > 1) out->scratch += (size_t)6 * ((size_t)R->slots * 4 + 16) + (R_MAX_BINS + 4) * 4;
    return true;
}

}  // namespace
}  // namespace lapsum

using namespace lapsum;

extern "C" {

int64_t lapsum_route_scratch(int32_t by, int64_t k, const lapsum_route *route) {
    RoutePlan p;
    return route_plan(by, k, route, &p) ? (int64_t)p.scratch : LAPSUM_ERR_ARG;
}

int lapsum_route_build(const int32_t *ids, int32_t by, int64_t k, const lapsum_route *R, void *scratch,
                       int64_t scratch_bytes, struct CUstream_st *stream_in) try {
    RoutePlan p;
    if (!ids || !route_plan(by, k, R, &p)) return LAPSUM_ERR_ARG;
    if (!R->slot_token || !R->slot_entry || !R->expert_offsets || !R->token_offsets || !R->token_slots ||
        !R->token_entries)
        return LAPSUM_ERR_ARG;
    if (!multiples_of(4, ids, R->slot_token, R->slot_entry, R->expert_offsets, R->token_offsets, R->token_slots,
                      R->token_entries))
        return LAPSUM_ERR_ARG;
    if (p.scratch && (!scratch || (reinterpret_cast<uintptr_t>(scratch) & 15) || scratch_bytes < (int64_t)p.scratch))
        return LAPSUM_ERR_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream_in);
    RouteArgs A{};
    A.ids = ids;
    A.k = k;
    A.entries = R->slots;
    A.bins = p.bins;
    A.rows = p.rows;
    A.by_tokens = by == LAPSUM_ROUTE_BY_TOKENS;
    A.slot_token = R->slot_token;
    A.slot_entry = R->slot_entry;
    A.token_slots = R->token_slots;
    A.token_entries = R->token_entries;
    A.row_offsets = A.by_tokens ? R->token_offsets : R->expert_offsets;
    A.bin_offsets = A.by_tokens ? R->expert_offsets : R->token_offsets;
    A.blocks = p.blocks;
    A.tiles = p.tiles;
    if (!p.alone) {
        char *s = static_cast<char *>(scratch);
        A.counts = reinterpret_cast<uint32_t *>(s);
        s += (size_t)p.passes * R_MAX_BLOCKS * (R_MAX_BINS + 1) * 4;
        if (p.passes > 1) {
            A.tops = reinterpret_cast<int32_t *>(s);
            s += (R_MAX_BINS + 4) * 4;
        }
        for (int i = 0; i < 2 && p.passes > 1; ++i) {
            for (int32_t **q : {&A.key[i], &A.entry[i], &A.rank[i]}) {
                *q = reinterpret_cast<int32_t *>(s);
                s += (size_t)R->slots * 4;
                s += (16 - (reinterpret_cast<uintptr_t>(s) & 15)) & 15;
            }
        }
    }
    const size_t smem = (size_t)(RW + 2) * (size_t(1) << p.bits) * 4;
    LAPSUM_TRY(set_max_dynamic_smem(reinterpret_cast<const void *>(route_place_kernel), (size_t)(RW + 2) * R_MAX_BINS * 4));
    for (int pass = 0; pass < p.passes; ++pass) {
        const RoutePass P{pass, p.passes, pass * p.bits, p.bits};
        if (!p.alone && pass == 0) {
            Launch L("route_count", st);
            LAPSUM_TRY(launch_k(route_count_kernel, p.blocks, RT, 0, st, A, P));
        }
        Launch L("route_place", st);
        LAPSUM_TRY(launch_k(route_place_kernel, p.blocks, RT, smem, st, A, P, (int)p.alone));
    }
    if (p.passes > 1) {
        Launch L("route_offsets", st);
        LAPSUM_TRY(launch_k(route_offsets_kernel, (unsigned)((p.bins + 256) / 256), 256, 0, st, A, (p.passes - 1) & 1,
                            (p.passes - 1) * p.bits, p.bits));
    }
    return LAPSUM_OK;
} catch (...) {   // the launch set-up's host memory: no exception leaves a C entry
    return LAPSUM_ERR_ALLOC;
}

}  // extern "C"
