// k_select.cu -- the k largest scores of every row by index, with their gate
// values, and the gate's gradient at them.
//
// Selection.  With keys that order like the scores (ties share a key), let A be
// the k-th largest key: every key above A is selected, and of the keys equal to
// A the first k - #{key > A} by index.
//   n <= 1024     one warp a row, the keys in its registers; A by bisection on the
//                 key's bits (for a prefix c, #{key >= c} >= k tells whether A >= c;
//                 a count of exactly k ends it: no tie at the border)
//   n <= 32768    a group of warps a row, read once through shared memory
//   longer rows   a bracket from a sample, then three passes shared by all SMs
//
// Gradient.  The upstream gradient is zero off the selected scores, so with
// e_i = 2^{m - |x_i|} (x in base 2, m the row's smallest |x|)
//   lambda = sum_j dw_j e(idx_j) / sum_i e_i,
//   grad_i = -(f_i/t) lambda, and (f_i/t)(dw_j - lambda) at i = idx_j:
// the row is read once and written once, and no dense upstream row exists.
#include <algorithm>
#include <cmath>

#include "give_up.cuh"
#include "lapsum_kernels.h"
#include "lapsum_launch.h"
#include "route_common.cuh"

namespace lapsum {
namespace {

constexpr int64_t SEL_WARP_MAX = 1024;     // longest row of the one-warp kernels
constexpr int64_t SEL_CTA_MAX = 32768;     // longest row of the one-CTA kernels

// ------------------------------------------------------- one warp a row --
template <int I>
__global__ void __launch_bounds__(256)
select_warp_kernel(const float *__restrict__ scores, const float *__restrict__ p, int64_t rows, int n, int k,
                   int32_t *__restrict__ idx_out, float *__restrict__ w_out) {
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= rows) return;
    const float *r = scores + row * n;
    uint32_t key[I];
    uint32_t hi = 0u, lo = 0xffffffffu;
#pragma unroll
    for (int j = 0; j < I; ++j) {
        const int i = j * 32 + lane;
        key[j] = 0u;   // places behind the row: below every prefix asked for, and last by index
        if (i < n) {
            key[j] = sel_key(r[i]);
            hi = max(hi, key[j]);
            lo = min(lo, key[j]);
        }
    }
    hi = __reduce_max_sync(FULL, hi);
    lo = __reduce_min_sync(FULL, lo);
    uint32_t A = hi;
    bool exact = false;
    if (hi != lo) {
        const int top = 31 - __clz(hi ^ lo);
        A = top == 31 ? 0u : hi & ~((2u << top) - 1u);
        for (int bit = top; bit >= 0; --bit) {
            const uint32_t c = A | (1u << bit);
            unsigned cnt = 0;
#pragma unroll
            for (int j = 0; j < I; ++j) cnt += key[j] >= c;
            cnt = __reduce_add_sync(FULL, cnt);
            if (cnt >= (unsigned)k) {
                A = c;
                if (cnt == (unsigned)k) { exact = true; break; }
            }
        }
    }
    unsigned above = 0;
#pragma unroll
    for (int j = 0; j < I; ++j) above += key[j] > A;
    above = __reduce_add_sync(FULL, above);
    unsigned need = exact ? (unsigned)n : (unsigned)k - above;   // equals of A to take
    int base = 0;
#pragma unroll
    for (int j = 0; j < I; ++j) {
        const unsigned ge = __ballot_sync(FULL, key[j] >= A && j * 32 + lane < n);
        if (!ge) continue;
        const unsigned eq = __ballot_sync(FULL, key[j] == A) & ge;
        const unsigned below = lanes_below(lane);
        const bool mine = (ge >> lane) & 1;
        const bool take = mine && (!((eq >> lane) & 1) || __popc(eq & below) < need);
        const unsigned took = __ballot_sync(FULL, take);
        if (take) {
            const int64_t o = row * k + base + __popc(took & below);
            idx_out[o] = j * 32 + lane;
            if (p) w_out[o] = p[row * n + j * 32 + lane];
        }
        base += __popc(took);
        need -= min(need, (unsigned)__popc(eq));
    }
}

// ---------------------------------------------------- a group of warps a row --
// One CTA an SM: groups of G warps take rows of up to 4096 G scores in turn, and
// one more warp keeps a ring of 16 KB chunks full with the rows in their order
// (bulk copies, one mbarrier a chunk).  One row streams at the SM's whole rate
// while the other groups search theirs: at n = 16384 six groups of four warps, at
// n <= 4096 twenty-four of one.  Bound by the latency of a row's chain (filter, bin,
// mark, write) and its instructions, not by memory: 2^25 scores, k = n / 128, 47 us at
// n = 16384, 58 at 8192, 71 at 4096 and 66 at 2048, against 21 us for reading them.
//
// A group samples its next row ahead (512 scores, as 64 maxima) and takes as a bound
// the maximum of a rank that the k best exceed only with a margin of four standard
// deviations.  Each streamed score is compared with the bound once; what reaches it
// goes to a list per warp, without gaps: two to five k of a row.  Among those A is found
// by a histogram over the keys between the bound and the largest, then within one bin.
// The chosen scores are marked in a bitmap of the row, which gives them back in index
// order.  (A list per thread overflows at a third of the k and leaves lanes idle: n = 2048,
// k = 16, 76 us; n = 4096, k = 128, 170 against 90.)
//
// Where the bound missed or a list overflowed the row is read from memory instead:
// three histogram passes (11 + 11 + 10 key bits, or of as many bits as the group has
// bins) and one that marks.  A k too large for the lists goes to the kernel that holds
// its rows (below).
constexpr int RS_WARPS = 24;               // that select; one more streams
constexpr int RS_CHUNK = 4096;             // floats
constexpr int RS_RING = 5;
constexpr int RS_LIST = 768;               // kept scores of a warp
constexpr int RS_MAXIMA = 64;              // of a sample
constexpr int RS_WIDE = 16;                // warps of the one group that takes the longest rows
constexpr int RS_FEW = 64;                 // scores of one bin that a warp ranks by itself
constexpr uint32_t RS_MISSING = 1u << 20;  // a count that says: read the row from memory
constexpr uint32_t RS_BROKEN = RS_MISSING + 1;

template <int G>                           // warps of a group
struct RowSizes {
    static constexpr int T = 32 * G;
    static constexpr int BINS = T < 256 ? 8 * T : 2048;
};
// What the search of one row of at most 16 B scores works on (by G warps).
template <int G, int B = RowSizes<G>::BINS>
struct RowState {
    static constexpr int WORDS = B / 2;
    union {                                // zero between their uses, which never meet
        uint4 hist4[B / 4];
        uint32_t hist[B];
        struct {
            uint32_t gt[WORDS], eq[WORDS];
        };
    };
    uint32_t few[RS_FEW];
    uint32_t scan[G];
    uint32_t bin, above, in, got, need;
    uint16_t few_at[RS_FEW];
};
template <int G>
struct RowGroup : RowState<G> {
    uint32_t key[G][RS_LIST];
    uint32_t count[G], top[G], bound;
    uint16_t at[G][RS_LIST];
};
template <int G>
struct RowShared {
    float ring[RS_RING][RS_CHUNK];
    uint64_t full[RS_RING], empty[RS_RING];
    uint64_t turn[RS_WARPS / G];           // a group's next row has begun to arrive
    RowGroup<G> group[RS_WARPS / G];
};


// The wait of a whole warp, the same answer in every lane.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, int times = 1) {
    bool ok = false;
    for (int z = 0; z < times && !ok; ++z) ok = mbar_wait(bar, parity, RING_WAIT_CAP);
    return __all_sync(FULL, ok);
}

// Chunk c of the stream is in its slot (`use`: how often the slot was used before).
// A barrier tells a phase from the next one only, so the chunk that the slot held
// before has to be consumed first: it may be another group's.
__device__ __forceinline__ bool chunk_wait(uint64_t *full, uint64_t *empty, uint32_t use) {
    return warp_wait(empty, (use & 1u) ^ 1u) && warp_wait(full, use & 1u);
}

// A thread's place in its group.
template <int G>
struct Member {
    int lane, warp, tid, id;               // warp, thread: within the group
    __device__ __forceinline__ void sync() const {
        if (G == 1) __syncwarp();
        else asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(32 * G) : "memory");
    }
    // (before, total) of one count per thread; ends behind a barrier
    __device__ __forceinline__ void scan(unsigned v, uint32_t *s_warp, unsigned &before, unsigned &total) const {
        unsigned incl = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned u = __shfl_up_sync(FULL, incl, o);
            if (lane >= o) incl += u;
        }
        if (G == 1) {
            before = incl - v;
            total = __shfl_sync(FULL, incl, 31);
            __syncwarp();
            return;
        }
        if (lane == 31) s_warp[warp] = incl;
        sync();
        const unsigned w = lane < G ? s_warp[lane] : 0u;
        before = incl - v + __reduce_add_sync(FULL, lane < warp ? w : 0u);
        total = __reduce_add_sync(FULL, w);
        sync();
    }
};

// The histogram's bin that holds the need-th largest, counted from the top bin;
// the bins are left at zero.  (bin, scores above it, scores in it) for every thread.
template <int G, int B>
__device__ __forceinline__ void rs_bin(RowState<G, B> &S, const Member<G> &M, unsigned need, uint32_t &bin, uint32_t &above,
                                       uint32_t &in) {
    constexpr int PER = B / RowSizes<G>::T, V = PER / 4;   // a thread's bins, in vectors of four
    const int first = B - 1 - M.tid * PER;
    uint32_t h[PER], sum = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const uint4 x = S.hist4[first / 4 - v];
        S.hist4[first / 4 - v] = uint4{};
        h[4 * v] = x.w;
        h[4 * v + 1] = x.z;
        h[4 * v + 2] = x.y;
        h[4 * v + 3] = x.x;
        sum += x.x + x.y + x.z + x.w;
    }
    unsigned before, total;
    M.scan(sum, S.scan, before, total);
    if (before < need && before + sum >= need) {
        uint32_t c = before;
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            if (c < need && c + h[q] >= need) {
                S.bin = first - q;
                S.above = c;
                S.in = h[q];
            }
            c += h[q];
        }
    }
    M.sync();
    bin = S.bin;
    above = S.above;
    in = S.in;
}

template <int N>
constexpr int log2_of() { return N <= 1 ? 0 : 1 + log2_of<N / 2>(); }

// Narrows the keys lo .. lo + span to those that hold the wanted rank until they are one
// key (shift 0) or at most RS_FEW (`in`).  each(f): f(key, ...) of this thread's keys;
// need_of(), asked once behind a barrier: the rank, or 0 where it is not among them (false
// is returned); `need` becomes the rank within what is left.
template <int G, int B, typename Each, typename NeedOf>
__device__ __forceinline__ bool rs_narrow(RowState<G, B> &S, const Member<G> &M, Each &&each, NeedOf &&need_of, uint32_t &lo,
                                          uint32_t &span, int &shift, uint32_t &in, unsigned &need) {
    constexpr int BITS = log2_of<B>();
    const uint32_t top = lo + span;        // inside the last bin, which holds no key above it
    for (bool first = true;; first = false) {
        shift = max(0, 32 - BITS - __clz(span | 1u));   // the span in at most B bins
        each([&](uint32_t key, auto &&) {
            if (key - lo <= span) atomicAdd(&S.hist[(key - lo) >> shift], 1u);
        });
        M.sync();
        if (first) need = need_of();
        uint32_t bin, above;
        rs_bin(S, M, need, bin, above, in);
        if (!need) return false;
        need -= above;
        lo += bin << shift;
        span = min((1u << shift) - 1u, top - lo);
        if (!shift || in <= RS_FEW) return true;
    }
}
// The few keys left: each is marked if fewer than `need` of them are above it; `need`
// becomes how many of the equals of A are selected.
template <int G, int B>
__device__ __forceinline__ void rs_few(RowState<G, B> &S, const Member<G> &M, uint32_t in, unsigned &need) {
    M.sync();
    if (M.warp == 0) {
        uint32_t lowest = 0xffffffffu; // the smallest selected: A
        uint32_t mine[RS_FEW / 32];
        unsigned over[RS_FEW / 32] = {};
#pragma unroll
        for (int z = 0; z < RS_FEW / 32; ++z) mine[z] = z * 32 + M.lane < (int)in ? S.few[z * 32 + M.lane] : 0u;
        for (int j = 0; j < (int)in; ++j) {
            const uint32_t other = S.few[j];
#pragma unroll
            for (int z = 0; z < RS_FEW / 32; ++z) over[z] += other > mine[z];
        }
#pragma unroll
        for (int z = 0; z < RS_FEW / 32; ++z)
            if (z * 32 + M.lane < (int)in && over[z] < need) lowest = min(lowest, mine[z]);
        lowest = __reduce_min_sync(FULL, lowest);
        unsigned gt = 0;
#pragma unroll
        for (int z = 0; z < RS_FEW / 32; ++z) {
            const bool real = z * 32 + M.lane < (int)in;
            gt += __popc(__ballot_sync(FULL, real && mine[z] > lowest));
            if (real && mine[z] >= lowest) {
                const int at = S.few_at[z * 32 + M.lane];
                atomicOr(mine[z] > lowest ? &S.gt[at >> 5] : &S.eq[at >> 5], 1u << (at & 31));
            }
        }
        if (M.lane == 0) {
            S.need = need - gt;
            S.got = 0u;
        }
    }
    M.sync();
    need = S.need;
}
// Marks the k largest of the kept keys (from `lo` to `hi`; each(f): f(key, at) of this
// thread's, at() a key's place) in the bitmaps; `need`: how many of the equals are selected.
template <int G, int B, typename Each>
__device__ __forceinline__ void rs_choose(RowState<G, B> &S, const Member<G> &M, Each &&each, unsigned k, uint32_t lo, uint32_t hi,
                                          unsigned &need) {
    uint32_t span = hi - lo, in;
    int shift;
    rs_narrow(S, M, each, [=] { return k; }, lo, span, shift, in, need);
    // above what is left: selected; in it: equals of A, or a few to be ranked
    each([&](uint32_t key, auto &&place) {
        if (key < lo) return;
        const int at = place();
        uint32_t *map = key - lo > span ? S.gt : S.eq;
        if (map == S.gt || !shift) atomicOr(&map[at >> 5], 1u << (at & 31));
        else {
            const uint32_t o = atomicAdd(&S.got, 1u);
            S.few[o] = key;
            S.few_at[o] = (uint16_t)at;
        }
    });
    if (shift) rs_few(S, M, in, need);
}

// The same over the row in memory; marks the bitmaps.
template <int G, int B>
__device__ __forceinline__ void rs_from_memory(RowState<G, B> &S, const Member<G> &M, const float *r, int n, unsigned k,
                                               unsigned &need) {
    constexpr int BITS = log2_of<B>(), T = 32 * G, U = 16;   // loads in flight
    const int lane = M.lane;
    uint32_t A = 0u, fixed = 0u;
    need = k;
    for (int at = 32; at > 0; at -= BITS) {
        const int shift = max(0, at - BITS);
        const uint32_t bins = 1u << (at - shift);
        for (int i0 = M.warp * 32; i0 < n; i0 += U * T) {
            float f[U];
#pragma unroll
            for (int u = 0; u < U; ++u) f[u] = i0 + u * T + lane < n ? r[i0 + u * T + lane] : 0.f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t key = sel_key(f[u]);
                const bool in = i0 + u * T + lane < n && (key & fixed) == A;
                const uint32_t d = in ? (key >> shift) & (bins - 1) : 0xffffffffu;
                int same;                  // ties come in runs: one add for a warp of them
                __match_all_sync(FULL, d, &same);
                if (same) {
                    if (in && lane == 0) atomicAdd(&S.hist[d], 32u);
                } else if (in) {
                    atomicAdd(&S.hist[d], 1u);
                }
            }
        }
        M.sync();
        uint32_t bin, above, in;
        rs_bin(S, M, need, bin, above, in);
        need -= above;
        A |= bin << shift;
        fixed |= (bins - 1u) << shift;
    }
    for (int i0 = M.warp * 32; i0 < n; i0 += U * T) {
        float f[U];
#pragma unroll
        for (int u = 0; u < U; ++u) f[u] = i0 + u * T + lane < n ? r[i0 + u * T + lane] : 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * T;
            const uint32_t key = sel_key(f[u]);
            const uint32_t g = __ballot_sync(FULL, i + lane < n && key > A), e = __ballot_sync(FULL, i + lane < n && key == A);
            if (lane == 0 && i < n) {
                S.gt[i >> 5] = g;
                S.eq[i >> 5] = e;
            }
        }
    }
}

// Of the equals the first `need` stay: clears the others of this thread's words e (ne in
// them; before: the greater ones and, in the upper half, the equals of the threads below).
// Returns the place of the thread's first.
template <int PER>
__device__ __forceinline__ unsigned rs_trim(uint32_t (&e)[PER], unsigned ne, unsigned before, unsigned need) {
    const unsigned be = min(before >> 16, need);
    if (ne > need - be) {
        unsigned drop = ne - (need - be);
#pragma unroll
        for (int q = PER - 1; q >= 0; --q)
            for (; drop && e[q]; --drop) e[q] ^= 0x80000000u >> __clz(e[q]);
    }
    return (before & 0xffffu) + be;
}
// What the bitmaps mark, in order, to put(place, index); clears them.
template <int G, int B, typename Put>
__device__ __forceinline__ void rs_marked(RowState<G, B> &S, const Member<G> &M, unsigned need, Put &&put) {
    constexpr int PER = RowState<G, B>::WORDS / RowSizes<G>::T;
    const int first = M.tid * PER;
    M.sync();
    uint32_t g[PER], e[PER];
    unsigned ng = 0, ne = 0;
#pragma unroll
    for (int q = 0; q < PER; q += 2) {
        uint2 *a = reinterpret_cast<uint2 *>(S.gt + first + q), *b = reinterpret_cast<uint2 *>(S.eq + first + q);
        const uint2 x = *a, y = *b;
        *a = *b = uint2{};
        g[q] = x.x;
        g[q + 1] = x.y;
        e[q] = y.x;
        e[q + 1] = y.y;
        ng += __popc(x.x) + __popc(x.y);
        ne += __popc(y.x) + __popc(y.y);
    }
    unsigned before, total;
    M.scan(ng | ne << 16, S.scan, before, total);
    unsigned o = rs_trim<PER>(e, ne, before, need);
#pragma unroll
    for (int q = 0; q < PER; ++q)
        for (uint32_t m = g[q] | e[q]; m; m &= m - 1) put(o++, (first + q) * 32 + __ffs(m) - 1);
}

// Writes the row's selection through the lists' room, so that its gate values are fetched
// together.  (k is no more than the room: row_rank sends larger ones to the held rows.)
template <int G>
__device__ __forceinline__ void rs_emit(RowGroup<G> &S, const Member<G> &M, unsigned need, int k, const float *p, int32_t *idx,
                                        float *w) {
    int32_t *to = reinterpret_cast<int32_t *>(&S.key[0][0]);
    rs_marked(S, M, need, [&](unsigned o, int i) { to[o] = i; });
    M.sync();
    for (int j = M.tid; j < k; j += 32 * G) {
        const int i = to[j];
        idx[j] = i;
        if (p) w[j] = p[i];
    }
}

// The 16-byte granules wholly inside a row: `head` scores before them, `body` in them.
__device__ __forceinline__ void rs_granules(const float *r, int n, int &head, int &body) {
    head = (int)((4 - ((reinterpret_cast<uintptr_t>(r) >> 2) & 3)) & 3);
    body = (n - head) & ~3;
}

// The warp that streams: the rows of this CTA in order, chunk by chunk.
// It laps no group: the ring holds no group's row and its next one.
template <int RING, int CHUNK>
__device__ __forceinline__ void rs_stream(float (*ring)[CHUNK], uint64_t *full, uint64_t *empty, uint64_t *turn, int groups,
                                          const float *scores, int rows, int n) {
    int group = 0;
    int slot = 0, phase = 1;               // a fresh barrier's phase before the first counts as done
    uint32_t sent = 0;
    bool ok = true;
    for (int row = blockIdx.x; row < rows && ok; row += gridDim.x) {
        const float *r = scores + (int64_t)row * n;
        int head, body;
        rs_granules(r, n, head, body);
        for (int a = 0; a < body; a += CHUNK) {
            ok = mbar_wait(&empty[slot], phase, RING_WAIT_CAP);
            if (!ok) break;
            const uint32_t bytes = (uint32_t)min(CHUNK, body - a) * 4u;
            fence_proxy_async_smem();
            mbar_expect_tx(&full[slot], bytes);
            bulk_load(ring[slot], r + head + a, bytes, &full[slot]);
            if (a == 0) mbar_arrive(&turn[group]);
            ++sent;
            if (++slot == RING) { slot = 0; phase ^= 1; }
        }
        if (++group == groups) group = 0;
    }
    // no CTA ends with copies in flight: the last of every slot
    for (uint32_t z = 0; z < min(sent, (uint32_t)RING); ++z) {
        const uint32_t seq = sent - 1 - z;
        mbar_wait(&full[seq % RING], (seq / RING) & 1, RING_WAIT_CAP);
    }
}

// The sample of a row: 128 granules spread over it, 512 scores, as 64 maxima.
// (512 lone scores take a warp 5800 cycles to ask for, the granules 400: 43 and 36 us of
// 1024 rows of 32768.  Where neighbours are alike a maximum is one of fewer scores, which
// lowers the bound.)
struct RowSample {
    static constexpr int SCORES = 512;
    float4 f[4];
    __device__ __forceinline__ void fetch(const float *r, int n, int lane) {
        int head, body;
        rs_granules(r, n, head, body);
        const float4 *g = reinterpret_cast<const float4 *>(r + head);
        const int m = body >> 2;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int s = q * 32 + lane;
            const int a = s * m / 128, b = (s + 1) * m / 128;
            f[q] = g[a + (((s * 37) & 63) * (b - a) >> 6)];
        }
    }
    __device__ __forceinline__ void maxima(uint32_t &a, uint32_t &b) const {
        auto of = [](const float4 &v) { return max(max(sel_key(v.x), sel_key(v.y)), max(sel_key(v.z), sel_key(v.w))); };
        a = max(of(f[0]), of(f[1]));
        b = max(of(f[2]), of(f[3]));
    }
};
// The maximum of that rank: the smallest that fewer than `rank` are above.
__device__ __forceinline__ uint32_t sample_bound(uint32_t a, uint32_t b, int rank) {
    int over_a = 0, over_b = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        const uint32_t x = __shfl_sync(FULL, a, j), y = __shfl_sync(FULL, b, j);
        over_a += (x > a) + (y > a);
        over_b += (x > b) + (y > b);
    }
    return __reduce_min_sync(FULL, min(over_a < rank ? a : 0xffffffffu, over_b < rank ? b : 0xffffffffu));
}

// The largest score below lo (a NaN at -infinity): a score reaches lo if the sign of `under` -
// score is set, which no NaN's is.  Nothing reaches lo = -infinity, where lists would overflow.
__device__ __forceinline__ float sel_under(float lo) {
    return lo > -INFINITY ? sel_value(sel_key(lo) - (lo == 0.f ? 2u : 1u)) : __int_as_float(0x7fffffff);
}
// The signs of `under` - score: one bit each, the first score's in the highest.
__device__ __forceinline__ void sel_signs(uint32_t &reach, float under, const float4 &v) {
    reach = __funnelshift_l(__float_as_uint(under - v.x), reach, 1);
    reach = __funnelshift_l(__float_as_uint(under - v.y), reach, 1);
    reach = __funnelshift_l(__float_as_uint(under - v.z), reach, 1);
    reach = __funnelshift_l(__float_as_uint(under - v.w), reach, 1);
}
// Adds the scores of the set bits of `reach` (the j-th highest: place_of(thread's lane, j) in src,
// index at + that) to a warp's list: their places first, then their keys, 32 at a time.  Past the
// list's end only the count goes on.
template <int ROOM, typename PlaceOf>
__device__ __forceinline__ void sel_append(uint32_t *keys, uint16_t *ats, int &len, uint32_t &top, uint32_t reach, int lane,
                                           const float *src, int at, PlaceOf &&place_of) {
    const int mine = __popc(reach);
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(FULL, upto, d);
        if (lane >= d) upto += x;
    }
    const int found = __shfl_sync(FULL, upto, 31);
    if (len + found <= ROOM) {
        uint16_t *to = ats + len + upto - mine;
        for (; reach; ++to) {
            const int j = __clz(reach);
            *to = (uint16_t)(lane * 32 + j);
            reach &= 0x7fffffffu >> j;
        }
        __syncwarp();
#pragma unroll 1
        for (int j = len + lane; j < len + found; j += 32) {
            const int c = ats[j], o = place_of(c >> 5, c & 31);
            const uint32_t key = sel_key(src[o]);
            keys[j] = key;
            ats[j] = (uint16_t)(at + o);
            top = max(top, key);
        }
    }
    len += found;
}

// What a group keeps of a row: the scores that reach the bound, in a list a warp.
template <int G>
struct Kept {
    RowGroup<G> &S;
    const Member<G> &M;
    const float lo, under;
    uint32_t top;
    int len = 0;                           // the warp's
    __device__ __forceinline__ Kept(RowGroup<G> &s, const Member<G> &m, uint32_t bound)
        : S(s), M(m), lo(sel_value(bound)), under(sel_under(lo)), top(bound) {}
    // the scores before and behind the granules; comes first
    __device__ __forceinline__ void ends(const float *r, int n, int head, int body) {
        if (M.warp != 0) return;
        const int e = M.lane < 4 ? M.lane : head + body + M.lane - 4;
        float v = 0.f;
        bool in = M.lane < 4 ? M.lane < head : e < n;
        if (in) {
            v = r[e];
            in = v >= lo;
        }
        const unsigned who = __ballot_sync(FULL, in);
        if (in) {
            const int o = __popc(who & lanes_below(M.lane));
            S.key[0][o] = top = sel_key(v);
            S.at[0][o] = (uint16_t)e;
        }
        len = __popc(who);
    }
    // m floats of a chunk, the first of them score `at`
    template <int CHUNK>
    __device__ __forceinline__ void chunk(const float *src, int m, int at) {
        constexpr int T = 32 * G, VEC = CHUNK / 4 / T, U = VEC < 8 ? VEC : 8;
#pragma unroll 1
        for (int v0 = 0; v0 < VEC && 4 * v0 * T < m; v0 += U) {
            uint32_t reach = 0u;
#pragma unroll
            for (int u = 0; u < U; ++u)
                sel_signs(reach, under, lds128(reinterpret_cast<const float4 *>(src + 4 * (M.tid + (v0 + u) * T))));
            if (U < 8) reach <<= 32 - 4 * U;
            const int vecs = (m / 4 - M.tid + T - 1) / T - v0;   // of this thread's vectors those in the row
            if (vecs < U) reach &= vecs > 0 ? ~(0xffffffffu >> 4 * vecs) : 0u;
            if (!__any_sync(FULL, reach)) continue;
            sel_append<RS_LIST>(S.key[M.warp], S.at[M.warp], len, top, reach, M.lane, src, at, [&](int lane, int j) {
                return 4 * (M.warp * 32 + lane + (v0 + (j >> 2)) * T) + (j & 3);
            });
        }
    }
    // the group's count (RS_MISSING where a list is too short, RS_BROKEN where a wait
    // gave up) and its largest key, for every thread
    __device__ __forceinline__ void close(bool ok, unsigned &total, uint32_t &hi, bool &broken) {
        const uint32_t h = __reduce_max_sync(FULL, top);
        const bool bad = __any_sync(FULL, !ok);
        if (M.lane == 0) {
            S.count[M.warp] = bad ? RS_BROKEN : len > RS_LIST ? RS_MISSING : (unsigned)len;
            S.top[M.warp] = h;
        }
        M.sync();
        const unsigned l = M.lane < G ? S.count[M.lane] : 0u;
        hi = __reduce_max_sync(FULL, M.lane < G ? S.top[M.lane] : 0u);
        total = __reduce_add_sync(FULL, min(l, RS_MISSING));
        broken = __any_sync(FULL, l == RS_BROKEN);
    }
};

// rank: of the bound among a row's sample maxima.
template <int G>
__global__ void __launch_bounds__(RS_WARPS * 32 + 32, 1)
select_row_kernel(const float *__restrict__ scores, const float *__restrict__ p, int rows, int n, int k, int rank,
                  int32_t *__restrict__ idx_out, float *__restrict__ w_out) {
    constexpr int NG = RS_WARPS / G, T = 32 * G;
    extern __shared__ __align__(16) unsigned char smem[];
    RowShared<G> &All = *reinterpret_cast<RowShared<G> *>(smem);
    if (threadIdx.x == 0) {
        for (int i = 0; i < RS_RING; ++i) {
            mbar_init(&All.full[i], 1);
            mbar_init(&All.empty[i], G);
        }
        for (int i = 0; i < NG; ++i) mbar_init(&All.turn[i], 1);
        mbar_init_fence();
    }
    const int warp_all = threadIdx.x >> 5;
    Member<G> M;
    M.lane = threadIdx.x & 31;
    M.id = warp_all / G;
    M.warp = warp_all % G;
    M.tid = M.warp * 32 + M.lane;
    if (warp_all < RS_WARPS) {
        for (int i = M.tid; i < RowSizes<G>::BINS; i += T) All.group[M.id].hist[i] = 0u;
        if (M.tid == 0) All.group[M.id].got = 0u;
    }
    pdl_enter();
    __syncthreads();
    if (warp_all == RS_WARPS) {
        if (M.lane == 0) rs_stream<RS_RING, RS_CHUNK>(All.ring, All.full, All.empty, All.turn, NG, scores, rows, n);
        return;
    }

    RowGroup<G> &S = All.group[M.id];
    const int step = gridDim.x * NG;       // rows from one of this group to its next
    RowSample sample;
    const int row0 = blockIdx.x + M.id * gridDim.x;
    if (M.warp == 0 && row0 < rows) sample.fetch(scores + (int64_t)row0 * n, n, M.lane);
    bool ring = true;                      // false once a wait has given up
    uint32_t chunk = 0;                    // of the CTA's stream, at the row of this turn
    uint32_t turn = 0;                     // rows that this group has begun
    int walked = blockIdx.x;               // the row that `chunk` belongs to
    for (int row = row0; row < rows; row += step) {
        const float *r = scores + (int64_t)row * n;
        unsigned need;
        bool done = false;
        if (ring) {
            if (M.warp == 0) {
                uint32_t a, b;
                sample.maxima(a, b);
                if (row + step < rows) sample.fetch(r + (int64_t)step * n, n, M.lane);   // arrives while this row streams
                const uint32_t c = sample_bound(a, b, rank);
                if (M.lane == 0) S.bound = c;
            }
            // the chunks of the rows before this one, other groups'
            int head, body;
            while (walked < row) {
                rs_granules(scores + (int64_t)walked * n, n, head, body);
                chunk += (uint32_t)(body + RS_CHUNK - 1) / RS_CHUNK;
                walked += gridDim.x;
            }
            rs_granules(r, n, head, body);
            uint32_t slot = chunk % RS_RING, use = chunk / RS_RING;
            M.sync();
            const uint32_t bound = S.bound;
            Kept<G> kept(S, M, bound);
            bool ok = waited(warp_wait(&All.turn[M.id], turn & 1u), GIVE_UP_READ, (int)turn);
            ++turn;
            kept.ends(r, n, head, body);
            for (int a = 0; a < body && ok; a += RS_CHUNK) {
                ok = chunk_wait(&All.full[slot], &All.empty[slot], use);
                kept.template chunk<RS_CHUNK>(All.ring[slot], min(RS_CHUNK, body - a), head + a);
                __syncwarp();
                if (M.lane == 0) mbar_arrive(&All.empty[slot]);
                if (++slot == RS_RING) { slot = 0; ++use; }
            }
            unsigned total;
            uint32_t hi;
            bool broken;
            kept.close(ok, total, hi, broken);
            ring = !broken;
            if (bound && total >= (unsigned)k && total < RS_MISSING) {
                auto each = [&](auto &&f) {
#pragma unroll 2
                    for (int j = M.lane; j < kept.len + M.lane; j += 32) {
                        const uint32_t key = j < kept.len ? S.key[M.warp][j] : 0u;   // below every bound
                        f(key, [&] { return (int)S.at[M.warp][j]; });
                    }
                };
                rs_choose(S, M, each, (unsigned)k, bound, hi, need);
                done = true;
            }
        }
        if (!done) rs_from_memory(S, M, r, n, (unsigned)k, need);
        rs_emit(S, M, need, k, p ? p + (int64_t)row * n : nullptr, idx_out + (int64_t)row * k,
                w_out + (p ? (int64_t)row * k : 0));
        M.sync();                          // the lists' room is free
    }
}

// The longest rows, 16385 to 32768, one of which fills most of the ring: one CTA an SM
// in which 27 warps share the work on consecutive rows.  One streams and one samples,
// ahead; sixteen filter a row into lists; two sets of four search the rows before (each
// its own lists, every other row); one writes what they found, with the gate values that
// it fetches meanwhile.  The filter's instructions and the search's barriers bound it
// (about 4.5 us a row and SM, where the row's bytes take 3).
// (1024 rows of 32768, k = 256: 36 us; one search of eight warps 43 us; sixteen warps that
// filter and search 52 us, three groups of eight 62 us, a row's keys in a CTA's registers
// and bisection 247 us.)
constexpr int RW_SEARCH = 4, RW_SETS = 2;  // warps of a search, searches
constexpr int RW_FIRST = RS_WIDE + RW_SEARCH * RW_SETS;
constexpr int RW_WARPS = RW_FIRST + 3;
constexpr int RW_CHUNK = 8192;             // floats: four vectors a filtering thread
constexpr int RW_RING = 4;
constexpr int RW_STAGE = 1024;             // indices handed to the warp that writes; more are written by the search
constexpr int RW_LIST = 384;               // kept scores of a filtering warp
struct WideShared {
    float ring[RW_RING][RW_CHUNK];
    uint64_t full[RW_RING], empty[RW_RING], turn[1];
    uint64_t bound_full[2], bound_empty[2], list_full[2], list_empty[2], stage_full[2], stage_empty[2];
    uint32_t bound[2], handed[2];
    volatile int direct[2];                // this CTA's row from which on a search writes by itself
    RowState<RW_SEARCH, 2048> search[RW_SETS];
    uint32_t key[2][RS_WIDE][RW_LIST];
    uint32_t count[2][RS_WIDE], top[2][RS_WIDE], from[2];
    uint16_t at[2][RS_WIDE][RW_LIST];
    uint16_t stage[2][RW_STAGE];
};
static_assert(sizeof(WideShared) <= 227 * 1024 && sizeof(RowShared<1>) <= 227 * 1024 && sizeof(RowShared<8>) <= 227 * 1024,
              "shared memory of one CTA");

__global__ void __launch_bounds__(RW_WARPS * 32, 1)
select_wide_kernel(const float *__restrict__ scores, const float *__restrict__ p, int rows, int n, int k, int rank,
                   int32_t *__restrict__ idx_out, float *__restrict__ w_out) {
    constexpr int F = RS_WIDE, T = 32 * F;
    extern __shared__ __align__(16) unsigned char smem[];
    WideShared &All = *reinterpret_cast<WideShared *>(smem);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < RW_RING; ++i) {
            mbar_init(&All.full[i], 1);
            mbar_init(&All.empty[i], F);
        }
        mbar_init(&All.turn[0], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&All.bound_full[i], 1);
            mbar_init(&All.bound_empty[i], F);
            mbar_init(&All.list_full[i], F);
            mbar_init(&All.list_empty[i], RW_SEARCH);
            mbar_init(&All.stage_full[i], RW_SEARCH);
            mbar_init(&All.stage_empty[i], 1);
        }
        for (int i = 0; i < RW_SETS; ++i) {
            All.search[i].got = 0u;
            All.direct[i] = INT_MAX;
        }
        mbar_init_fence();
    }
    for (int i = threadIdx.x; i < 2048; i += RW_WARPS * 32) All.search[0].hist[i] = All.search[1].hist[i] = 0u;
    pdl_enter();
    __syncthreads();
    const bool staged = k <= RW_STAGE;
    if (warp == RW_FIRST) {           // ---- streams
        if (lane == 0) rs_stream<RW_RING, RW_CHUNK>(All.ring, All.full, All.empty, All.turn, 1, scores, rows, n);
        return;
    }
    if (warp == RW_FIRST + 1) {       // ---- samples, at most two rows ahead
        RowSample sample;
        if ((int)blockIdx.x < rows) sample.fetch(scores + (int64_t)blockIdx.x * n, n, lane);
        int i = 0;
        for (int row = blockIdx.x; row < rows; row += gridDim.x, ++i) {
            uint32_t a, b;
            sample.maxima(a, b);
            if (row + (int)gridDim.x < rows) sample.fetch(scores + ((int64_t)row + gridDim.x) * n, n, lane);
            const uint32_t c = sample_bound(a, b, rank);
            if (!warp_wait(&All.bound_empty[i & 1], ((i >> 1) & 1) ^ 1)) return;
            if (lane == 0) {
                All.bound[i & 1] = c;
                mbar_arrive(&All.bound_full[i & 1]);
            }
        }
        return;
    }
    if (warp == RW_FIRST + 2) {       // ---- writes
        if (!staged) return;
        int i = 0;
        for (int row = blockIdx.x; row < rows; row += gridDim.x, ++i) {
            int32_t *idx = idx_out + (int64_t)row * k;
            if (!waited(warp_wait(&All.stage_full[i & 1], (i >> 1) & 1, 16), GIVE_UP_WRITE, i)) {   // longer than the search's own waits can take
                // never seen: two rows at most were handed over, and none of them is left stale
                for (int z = 0; z < 2 && i + z < All.direct[(i + z) & 1] && row + z * (int)gridDim.x < rows; ++z)
                    for (int j = lane; j < k; j += 32) {
                        idx[(int64_t)z * gridDim.x * k + j] = -1;
                        if (p) w_out[((int64_t)row + (int64_t)z * gridDim.x) * k + j] = CUDART_NAN_F;
                    }
                return;
            }
            const uint16_t *from = All.stage[i & 1];
            const float *pr = p ? p + (int64_t)row * n : nullptr;
            for (int j0 = lane; j0 < k; j0 += 256) {
                float v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (pr && j0 + 32 * u < k) v[u] = pr[from[j0 + 32 * u]];
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (j0 + 32 * u < k) {
                        idx[j0 + 32 * u] = from[j0 + 32 * u];
                        if (pr) w_out[(int64_t)row * k + j0 + 32 * u] = v[u];
                    }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&All.stage_empty[i & 1]);
        }
        return;
    }
    if (warp < F) {                        // ---- filter
        uint32_t slot = 0, phase = 0;
        bool ok = true;                    // false once a wait has given up: the search then reads from memory
        int i = 0;
        for (int row = blockIdx.x; row < rows; row += gridDim.x, ++i) {
            const int buf = i & 1;
            const float *r = scores + (int64_t)row * n;
            int head, body;
            rs_granules(r, n, head, body);
            // a search that still reads these lists' counts must not see them change: without
            // room this warp ends, and the searches' waits for it run out
            if (!warp_wait(&All.list_empty[buf], ((i >> 1) & 1) ^ 1)) return;
            ok = ok && waited(warp_wait(&All.bound_full[buf], (i >> 1) & 1), GIVE_UP_READ, i);
            const uint32_t bound = All.bound[buf];
            const float lo = sel_value(bound);
            const float under = sel_under(lo);
            uint32_t top = bound;
            int len = 0;
            uint32_t *keys = All.key[buf][warp];
            uint16_t *ats = All.at[buf][warp];
            if (ok && warp == 0) {         // the scores before and behind the granules
                const int e = lane < 4 ? lane : head + body + lane - 4;
                float v = 0.f;
                bool in = lane < 4 ? lane < head : e < n;
                if (in) {
                    v = r[e];
                    in = v >= lo;
                }
                const unsigned who = __ballot_sync(FULL, in);
                if (in) {
                    const int o = __popc(who & lanes_below(lane));
                    keys[o] = top = sel_key(v);
                    ats[o] = (uint16_t)e;
                }
                len = __popc(who);
            }
            for (int a = 0; a < body && ok; a += RW_CHUNK) {
                ok = warp_wait(&All.full[slot], phase);
                const float *src = All.ring[slot];
                const int m = min(RW_CHUNK, body - a);
                uint32_t reach = 0u;       // a bit a score, the first in the highest
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    sel_signs(reach, under, lds128(reinterpret_cast<const float4 *>(src + 4 * ((int)threadIdx.x + u * T))));
                }
                reach <<= 16;
                if (m < RW_CHUNK) {        // of this thread's vectors those in the row
                    const int vecs = max(0, (m / 4 - (int)threadIdx.x + T - 1) / T);
                    if (vecs < 4) reach &= ~(0xffffffffu >> (4 * vecs));
                }
                sel_append<RW_LIST>(keys, ats, len, top, reach, lane, src, head + a, [&](int who, int j) {
                    return 4 * (warp * 32 + who + (j >> 2) * T) + (j & 3);
                });
                __syncwarp();
                if (lane == 0) mbar_arrive(&All.empty[slot]);
                if (++slot == RW_RING) { slot = 0; phase ^= 1u; }
            }
            const uint32_t h = __reduce_max_sync(FULL, top);
            if (lane == 0) {
                All.count[buf][warp] = !ok ? RS_BROKEN : len > RW_LIST ? RS_MISSING : (unsigned)len;
                All.top[buf][warp] = h;
                if (warp == 0) All.from[buf] = bound;
                mbar_arrive(&All.bound_empty[buf]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&All.list_full[buf]);
        }
        return;
    }
    // ---- search
    Member<RW_SEARCH> M;
    M.lane = lane;
    M.id = (warp - F) / RW_SEARCH;
    M.warp = (warp - F) % RW_SEARCH;
    M.tid = M.warp * 32 + lane;
    const int buf = M.id;
    auto &S = All.search[buf];
    bool lists = true, hand = staged;      // false once a wait has given up
    int i = M.id;
    for (int64_t at = blockIdx.x + (int64_t)M.id * gridDim.x; at < rows; at += 2 * (int64_t)gridDim.x, i += 2) {
        const int row = (int)at;
        const float *r = scores + at * n;
        const bool got = lists && warp_wait(&All.list_full[buf], (i >> 1) & 1, 8);   // longer than the filter's own waits can take
        if (M.lane == 0) S.scan[M.warp] = got;
        if (M.tid == 0) {
            const bool was = hand;
            All.handed[buf] = hand = hand && mbar_wait(&All.stage_empty[buf], ((i >> 1) & 1) ^ 1, RING_WAIT_CAP);
            if (was && !hand) All.direct[buf] = i;
        }
        M.sync();
        lists = __all_sync(FULL, lane < RW_SEARCH ? S.scan[lane] != 0u : true);
        unsigned need, total = RS_MISSING;
        uint32_t bound = 0u, hi = 0u;
        if (lists) {
            bound = All.from[buf];
            const unsigned l = lane < F ? All.count[buf][lane] : 0u;
            hi = __reduce_max_sync(FULL, lane < F ? All.top[buf][lane] : 0u);
            total = __reduce_add_sync(FULL, min(l, RS_MISSING));
        }
        if (bound && total >= (unsigned)k && total < RS_MISSING) {
            constexpr int L = F / RW_SEARCH;   // this warp's lists, read together
            int len[L], most = 0;
#pragma unroll
            for (int q = 0; q < L; ++q) {
                len[q] = All.count[buf][M.warp * L + q];
                most = max(most, len[q]);
            }
            auto each = [&](auto &&f) {
#pragma unroll 1
                for (int j = lane; j < most + lane; j += 32) {
                    uint32_t key[L];
#pragma unroll
                    for (int q = 0; q < L; ++q) key[q] = j < len[q] ? All.key[buf][M.warp * L + q][j] : 0u;   // below every bound
#pragma unroll
                    for (int q = 0; q < L; ++q) f(key[q], [&] { return (int)All.at[buf][M.warp * L + q][j]; });
                }
            };
            rs_choose(S, M, each, (unsigned)k, bound, hi, need);
            __syncwarp();
            if (lane == 0) mbar_arrive(&All.list_empty[buf]);
        } else {
            if (lane == 0 && lists) mbar_arrive(&All.list_empty[buf]);
            rs_from_memory(S, M, r, n, (unsigned)k, need);
        }
        if (All.handed[buf]) {                  // (written before the barriers of the search)
            uint16_t *to = All.stage[buf];
            rs_marked(S, M, need, [&](unsigned o, int j) { to[o] = (uint16_t)j; });
            __syncwarp();
            if (lane == 0) mbar_arrive(&All.stage_full[buf]);
        } else {
            int32_t *idx = idx_out + (int64_t)row * k;
            rs_marked(S, M, need, [&](unsigned o, int j) { idx[o] = j; });
            M.sync();
            if (p)
                for (int j = M.tid; j < k; j += 32 * RW_SEARCH)
                    w_out[(int64_t)row * k + j] = p[(int64_t)row * n + __ldcg(idx + j)];
        }
    }
}

// ----------------------------------------------------------- rows held --
// Rows of 1025 to 32768 whose k is too large for lists: a CTA of T threads holds the row
// in shared memory (one bulk copy; several CTAs an SM but for the longest).  Of 128
// scores of it two ranks, four standard deviations to either side of k's, bracket A.
// One pass counts the keys above the bracket and a histogram within it, one marks; more
// only for ties and about zero, where keys lie far apart.  The next row is fetched while
// this one is written, 32 places a warp.  (2^25 scores, k = n / 4: 162, 155, 132 and 143 us
// at n = 2048, 4096, 16384 and 32768; with four passes over the row in memory, on all key
// bits, 242, 305, 311 and 283.)  Bound by the passes' instructions: the SM issues in 81 of
// 100 cycles.
constexpr int RH_SAMPLE = 128;
template <int T, int B>
struct HeldShared {
    RowState<T / 32, B> state;
    alignas(16) uint32_t sample[RH_SAMPLE];
    uint32_t lo, hi, counts[T / 32];
    uint64_t bar;
    alignas(16) float row[4];              // from here on: the row, its granules on 16 bytes
};
// Asks for n floats' whole 16-byte granules in L2.
__device__ __forceinline__ void prefetch_l2(const float *r, int n) {
    int head, body;
    rs_granules(r, n, head, body);
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(r + head), "r"(body * 4) : "memory");
}
// Marks the rows from `row` on that this block would take.  (A call of its own: written out
// it costs the passes registers, 165 us instead of 161 at n = 2048.)
__device__ __noinline__ void rh_mark(int row, int rows, int k, int32_t *idx_out, float *w_out) {
    for (int64_t z = row; z < rows; z += gridDim.x)
        for (int j = threadIdx.x; j < k; j += blockDim.x) {
            idx_out[z * k + j] = -1;
            if (w_out) w_out[z * k + j] = CUDART_NAN_F;
        }
}
template <int T, int B>
__global__ void __launch_bounds__(T, T == 1024 ? 1 : 1536 / T)
select_held_kernel(const float *__restrict__ scores, const float *__restrict__ p, int rows, int n, int k, int rank_hi, int rank_lo,
                   int32_t *__restrict__ idx_out, float *__restrict__ w_out) {
    constexpr int G = T / 32, PER = B / 2 / T, U = 8;
    extern __shared__ __align__(16) unsigned char smem[];
    HeldShared<T, B> &H = *reinterpret_cast<HeldShared<T, B> *>(smem);
    auto &S = H.state;
    Member<G> M;
    M.tid = threadIdx.x;
    M.lane = M.tid & 31;
    M.warp = M.tid >> 5;
    M.id = 0;
    if (M.tid == 0) {
        mbar_init(&H.bar, 1);
        S.got = 0u;
        mbar_init_fence();
    }
    for (int i = M.tid; i < B; i += T) S.hist[i] = 0u;
    pdl_enter();
    __syncthreads();
    bool bulk = true;                      // false once a wait has given up: plain loads
    // score e of a row lies at row[pad + e]; the CTA is done with the row before
    auto fetch = [&](int64_t row) {
        const float *r = scores + row * n;
        int head, body;
        rs_granules(r, n, head, body);
        float *to = H.row + ((4 - head) & 3);
        if (!bulk) {
            for (int e = M.tid; e < n; e += T) to[e] = r[e];
            return;
        }
        if (M.tid == 0) {
            fence_proxy_async_smem();
            mbar_expect_tx(&H.bar, (uint32_t)body * 4u);
            bulk_load(to + head, r + head, (uint32_t)body * 4u, &H.bar);
            if (p) prefetch_l2(p + row * n, n);
        }
        const int e = M.tid < 4 ? M.tid : head + body + M.tid - 4;
        if (M.tid < 4 ? M.tid < head : M.tid < 8 && e < n) to[e] = r[e];
    };
    if (blockIdx.x < rows) fetch(blockIdx.x);
    uint32_t phase = 0;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, phase ^= 1u, ++turn) {
        int head, body;
        rs_granules(scores + row * n, n, head, body);
        const float *x = H.row + ((4 - head) & 3);
        if (M.tid == 0) {
            H.lo = 0xffffffffu;
            H.hi = 0xff800000u;            // +infinity
        }
        const bool ok = !bulk || waited(mbar_wait(&H.bar, phase, RING_WAIT_CAP), GIVE_UP_READ, turn);
        if (!__syncthreads_and(ok)) {
            // a copy that is late may still write to the only room there is: then this block's rows
            // from here on are marked, and none of them is left stale
            if (!__syncthreads_and(waited(mbar_wait(&H.bar, phase, RING_WAIT_CAP), GIVE_UP_AGAIN, turn))) {
                rh_mark((int)row, rows, k, idx_out, p ? w_out : nullptr);
                return;
            }
            bulk = false;
            fetch(row);
            __syncthreads();
        }
        // the bracket
        if (M.tid < RH_SAMPLE) {
            const int a = M.tid * n / RH_SAMPLE, b = (M.tid + 1) * n / RH_SAMPLE;
            H.sample[M.tid] = sel_key(x[a + (((M.tid * 37) & 63) * (b - a) >> 6)]);
        }
        M.sync();
        if (M.tid < RH_SAMPLE) {
            const uint32_t mine = H.sample[M.tid];
            int over = 0;
#pragma unroll 8
            for (int j = 0; j < RH_SAMPLE; j += 4) {
                const uint4 o = *reinterpret_cast<const uint4 *>(&H.sample[j]);
                over += (o.x > mine) + (o.y > mine) + (o.z > mine) + (o.w > mine);
            }
            const uint32_t hi = __reduce_min_sync(FULL, over < rank_hi ? mine : 0xffffffffu);
            const uint32_t lo = __reduce_min_sync(FULL, over < rank_lo ? mine : 0xffffffffu);
            if (M.lane == 0) {
                atomicMin(&H.hi, hi);
                atomicMin(&H.lo, lo);
            }
        }
        M.sync();
        uint32_t lo = rank_lo ? H.lo : 0u, span = H.hi - lo, in;
        unsigned need, above = 0u, within = 0u;
        int shift;
        // In scores: keys above lo + span are those of v >= over, keys from lo on those of v >= from (and
        // NaN's, if lo is 0).  Past +infinity's key `over` is a NaN, which nothing reaches.
        float from, over;
        auto range = [&] {
            auto value = [](uint32_t key) {    // no key is -0's
                return sel_value(max(key == 0x7fffffffu ? 0x80000000u : key, 0x007fffffu));   // -infinity
            };
            from = value(lo);
            over = value(lo + span + 1u);
        };
        auto each = [&](auto &&f) {
            above = within = 0u;
            range();
            auto one = [&](float v) {
                const uint32_t key = sel_key(v);
                above += v >= over;
                within += key - lo <= span;
                f(key, 0);
            };
            const float4 *x4 = reinterpret_cast<const float4 *>(x + head);
            for (int i = M.tid; i < body >> 2; i += T) {
                const float4 v = lds128(x4 + i);
                one(v.x);
                one(v.y);
                one(v.z);
                one(v.w);
            }
            const int e = M.tid < 4 ? M.tid : head + body + M.tid - 4;
            if (M.tid < 4 ? M.tid < head : M.tid < 8 && e < n) one(x[e]);
        };
        auto need_of = [&] {
            const unsigned both = __reduce_add_sync(FULL, above | within << 16);   // each at most 32768
            if (M.lane == 0) H.counts[M.warp] = both;
            M.sync();
            const unsigned all = __reduce_add_sync(FULL, M.lane < G ? H.counts[M.lane] : 0u);
            const unsigned a = all & 0xffffu, w = all >> 16;
            return a < (unsigned)k && a + w >= (unsigned)k ? (unsigned)k - a : 0u;
        };
        if (!rs_narrow(S, M, each, need_of, lo, span, shift, in, need)) {   // the bracket missed: all keys
            lo = 0u;
            span = 0xff800000u;
            rs_narrow(S, M, each, [=] { return (unsigned)k; }, lo, span, shift, in, need);
        }
        range();
        const bool from_nan = lo == 0u;
        auto mark = [&](float v, int i, bool real) {
            const bool o = real && v >= over, inside = real && !o && (from_nan || v >= from);
            const uint32_t g = __ballot_sync(FULL, o), e = __ballot_sync(FULL, inside);
            if (M.lane == 0) {
                S.gt[i >> 5] = g;
                if (!shift) S.eq[i >> 5] = e;
            }
            if (shift && e) {              // few
                if (inside) {
                    const uint32_t place = atomicAdd(&S.got, 1u);
                    S.few[place] = sel_key(v);
                    S.few_at[place] = (uint16_t)(i + M.lane);
                }
                __syncwarp();
            }
        };
        int i0 = M.warp * 32;
        for (; i0 + (U - 1) * T + 32 <= n; i0 += U * T) {
            float v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] = x[i0 + u * T + M.lane];
#pragma unroll
            for (int u = 0; u < U; ++u) mark(v[u], i0 + u * T, true);
        }
        for (; i0 < n; i0 += T) mark(x[min(i0 + M.lane, n - 1)], i0, i0 + M.lane < n);
        if (shift) rs_few(S, M, in, need);
        M.sync();
        if (row + gridDim.x < rows) fetch(row + gridDim.x);
        // each word's selected bits and its first place
        {
            uint32_t g[PER], e[PER];
            unsigned ng = 0, ne = 0;
#pragma unroll
            for (int q = 0; q < PER; ++q) {
                g[q] = S.gt[M.tid * PER + q];
                e[q] = S.eq[M.tid * PER + q];
                ng += __popc(g[q]);
                ne += __popc(e[q]);
            }
            unsigned before, total;
            M.scan(ng | ne << 16, S.scan, before, total);
            unsigned o = rs_trim<PER>(e, ne, before, need);
#pragma unroll
            for (int q = 0; q < PER; ++q) {
                S.gt[M.tid * PER + q] = g[q] | e[q];
                S.eq[M.tid * PER + q] = o;
                o += __popc(g[q] | e[q]);
            }
        }
        M.sync();
        const float *pr = p ? p + row * n : nullptr;
        int32_t *idx = idx_out + row * k;
        float *w = w_out + (p ? row * k : 0);
        for (int i0 = M.warp * 32; i0 < n; i0 += U * T) {
            float v[U];
            int o[U];                      // a place of the selection, or -1
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int word = (i0 + u * T) >> 5;
                const uint32_t m = word < B / 2 ? S.gt[word] : 0u;   // past the row: empty ones
                o[u] = m >> M.lane & 1u ? (int)(S.eq[word] + __popc(m & lanes_below(M.lane))) : -1;
                v[u] = 0.f;
                if (pr && o[u] >= 0) v[u] = pr[i0 + u * T + M.lane];
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (o[u] >= 0) {
                    idx[o[u]] = i0 + u * T + M.lane;
                    if (pr) w[o[u]] = v[u];
                }
        }
        M.sync();
#pragma unroll
        for (int q = 0; q < PER; ++q) S.gt[M.tid * PER + q] = S.eq[M.tid * PER + q] = 0u;
    }
}

template <int T, int B, int NMAX>
cudaError_t run_select_held(const float *s, const float *p, int64_t rows, int64_t n, int64_t k, int32_t *idx, float *w,
                            cudaStream_t st) {
    const double mu = (double)k * RH_SAMPLE / (double)n, sd = std::sqrt(mu * (1.0 - (double)k / (double)n));
    const int rank_hi = std::max(0, (int)std::floor(mu - 4.0 * sd - 1.0));   // 0: open above
    int rank_lo = (int)std::ceil(mu + 4.0 * sd + 2.0);
    if (rank_lo > RH_SAMPLE) rank_lo = 0;  // open below
    const auto kern = select_held_kernel<T, B>;
    const size_t bytes = sizeof(HeldShared<T, B>) + (size_t)n * 4;
    // (one limit a kernel, whatever n: a smaller one set later would refuse the larger rows)
    const cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void *>(kern), sizeof(HeldShared<T, B>) + NMAX * 4);
    if (e != cudaSuccess) return e;
    const int64_t fit = std::min<int64_t>(2048 / T, 227 * 1024 / (int64_t)(bytes + 1024));   // CTAs an SM
    return launch_k(kern, (unsigned)std::min<int64_t>(rows, device_sm_count() * std::max<int64_t>(fit, 1)), T, bytes, st, s, p,
                    (int)rows, (int)n, (int)k, rank_hi, rank_lo, idx, w);
}

// The bound's rank among a row's sample maxima, or 0 where the lists would not hold
// what reaches it: each maximum stands for eight scores of the sample, so rank m of the
// maxima is about rank -64 ln(1 - m/64) of the sample, and a score of the sample for n/512
// of the row.  That varies from row to row: `room` is two thirds of the lists'.  (Where a
// row overflows all the same, one SM reads it from memory: 1024 rows of 32768, k = 1024,
// 57 us, with such a row 85, held 158.)
int row_rank(int64_t n, int64_t k, int room) {
    constexpr double S = RowSample::SCORES, M = RS_MAXIMA;
    const double mu = (double)k * S / (double)n;
    const int rank = (int)std::ceil(mu + 4.0 * std::sqrt(mu) + 4.0);
    if (rank >= RS_MAXIMA) return 0;
    return -M * std::log1p(-rank / M) * (double)n / S <= room ? rank : 0;
}

template <int G>
cudaError_t run_select_row(const float *s, const float *p, int64_t rows, int64_t n, int64_t k, int rank, int32_t *idx, float *w,
                           cudaStream_t st) {
    auto kern = select_row_kernel<G>;
    const cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void *>(kern), sizeof(RowShared<G>));
    if (e != cudaSuccess) return e;
    return launch_k(kern, (unsigned)std::min<int64_t>(rows, device_sm_count()), RS_WARPS * 32 + 32, sizeof(RowShared<G>), st,
                    s, p, (int)rows, (int)n, (int)k, rank, idx, w);
}

cudaError_t run_select_wide(const float *s, const float *p, int64_t rows, int64_t n, int64_t k, int rank, int32_t *idx, float *w,
                            cudaStream_t st) {
    const cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void *>(select_wide_kernel), sizeof(WideShared));
    if (e != cudaSuccess) return e;
    return launch_k(select_wide_kernel, (unsigned)std::min<int64_t>(rows, device_sm_count()), RW_WARPS * 32,
                    sizeof(WideShared), st, s, p, (int)rows, (int)n, (int)k, rank, idx, w);
}

// Warps of a group: what the row's length needs, and more where all rows find room at
// once all the same (64 rows of 3000 scores, k = 30: one warp each 37 us, eight 6 us).
// (Then a group sees one row only; where it sees several, its rows and those of the
// groups between them are longer than the ring, which therefore laps no group.)
int sel_warps(int64_t rows, int64_t n) {
    int g = n <= 4096 ? 1 : n <= 8192 ? 2 : n <= 16384 ? 4 : RS_WIDE;
    while (g < 8 && rows <= device_sm_count() * (RS_WARPS / (2 * g))) g *= 2;
    return g;
}

// Rows of 1025 to 32768.
cudaError_t run_select_rows(const float *s, const float *p, int64_t rows, int64_t n, int64_t k, int32_t *idx, float *w,
                            cudaStream_t st) {
    const int g = sel_warps(rows, n);
    const int rank = row_rank(n, k, g == RS_WIDE ? RS_WIDE * RW_LIST * 2 / 3 : g * RS_LIST * 2 / 3);
    if (!rank) {
        if (n <= 2048) return run_select_held<128, 1024, 2048>(s, p, rows, n, k, idx, w, st);
        if (n <= 8192) return run_select_held<256, 2048, 8192>(s, p, rows, n, k, idx, w, st);
        if (n <= 16384) return run_select_held<512, 2048, 16384>(s, p, rows, n, k, idx, w, st);
        return run_select_held<1024, 4096, 32768>(s, p, rows, n, k, idx, w, st);
    }
    switch (g) {
        case 1: return run_select_row<1>(s, p, rows, n, k, rank, idx, w, st);
        case 2: return run_select_row<2>(s, p, rows, n, k, rank, idx, w, st);
        case 4: return run_select_row<4>(s, p, rows, n, k, rank, idx, w, st);
        case 8: return run_select_row<8>(s, p, rows, n, k, rank, idx, w, st);
        default: return run_select_wide(s, p, rows, n, k, rank, idx, w, st);
    }
}

// ---------------------------------------------------------- longer rows --
// Rows are taken in batches of at most SEL_BATCH, each row cut into chunks.
//   sample   2048 scores of a row bracket A: the sample's values at ranks that lie
//            four standard deviations to either side of A's (one CTA a row)
//   hist     one pass counts the keys above the bracket and a histogram within it;
//            A's bin becomes the range.  Two more passes narrow it, and return at
//            once where the range is one key or holds at most SEL_FEW (ties need
//            them); a bracket that missed starts again from all keys
//   count    keys above the range per chunk, and the few within it; then A itself,
//            and the chunks' first places
//   emit     each chunk writes its share, in order
// Three reads of the row, whatever k is (1e7 Laplace scores, k = 1e5: 50 us; five
// passes over all key bits 104 us).  A row's last block to finish a pass digests what
// the pass counted: no block waits for another.
constexpr int SEL_BITS = 11;
constexpr int SEL_BINS = 1 << SEL_BITS;
constexpr int64_t SEL_BATCH = 256;
constexpr int SEL_MAX_CHUNKS = 4096;       // a row's chunks are scanned by one CTA
constexpr int SEL_T = 512;
constexpr int SEL_I = 16;                  // scores a thread has in flight
constexpr int SEL_TILE = SEL_T * SEL_I;
constexpr int SEL_FEW = 8192;
constexpr int SEL_SAMPLE = 2048;
constexpr int SEL_PASSES = 3;

struct alignas(16) SelRow {
    uint32_t hist[SEL_BINS];               // zero between passes
    uint32_t lo, span, shift;              // keys lo .. lo + span are looked at, in bins of 2^shift
    uint32_t need;                         // A's rank among them, from the top
    uint32_t found;                        // the range is one key, or a few
    uint32_t above, few;                   // keys above the bracket; keys in the few's list
    uint32_t ticket[SEL_PASSES + 1];
    uint2 list[SEL_FEW];                   // (key, chunk)
};

struct SelLong {
    const float *scores, *p;
    int32_t *idx;
    float *w;
    int64_t n, k, chunk;                   // chunk: places, a multiple of SEL_TILE
    int chunks;
    int rank_lo, rank_hi;                  // of the bracket in the sample; rank_hi < 1: open above
    SelRow *row;
    uint32_t *counts;                      // [row][chunk][2]: above A, equal to A; then their places
};

// True in every thread of the row's last block to get here.
__device__ __forceinline__ bool last_of_row(uint32_t *ticket, int chunks, bool *s_last) {
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        *s_last = atomicAdd(ticket, 1u) == (unsigned)chunks - 1u;
        __threadfence();
    }
    __syncthreads();
    return *s_last;
}

// (sum before this thread, sum of all) over the CTA.
__device__ __forceinline__ void sel_scan(uint32_t v, uint32_t *s_warp, uint32_t &before, uint32_t &total) {
    constexpr int NW = SEL_T / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(FULL, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    const uint32_t w = lane < NW ? s_warp[lane] : 0u;
    before = incl - v + __reduce_add_sync(FULL, lane < warp ? w : 0u);
    total = __reduce_add_sync(FULL, w);
    __syncthreads();
}

__global__ void __launch_bounds__(256) select_sample_kernel(SelLong L) {
    constexpr int T = 256, PER = SEL_SAMPLE / T, LAST = 12;
    __shared__ unsigned s_add[2 * (T / 32)];
    pdl_enter();
    SelRow *R = L.row + blockIdx.x;
    const float *r = L.scores + (int64_t)blockIdx.x * L.n;
    uint32_t key[PER];
#pragma unroll
    for (int q = 0; q < PER; ++q) {
        const int64_t s = q * T + threadIdx.x, a = s * L.n / SEL_SAMPLE, b = (s + 1) * L.n / SEL_SAMPLE;
        key[q] = sel_key(r[a + (s * 37 & 63) * (b - a) / 64]);
    }
    for (int i = threadIdx.x; i < SEL_BINS; i += T) R->hist[i] = 0u;
    BlockAdd<T / 32> add(s_add);
    uint32_t lo = 0u, hi = 0u;             // the keys of both ranks, bit by bit; the lowest bits are left open
    for (int bit = 31; bit >= LAST; --bit) {
        const uint32_t tl = lo | (1u << bit), th = hi | (1u << bit);
        unsigned c = 0;
#pragma unroll
        for (int q = 0; q < PER; ++q) c += (unsigned)(key[q] >= tl) | (unsigned)(key[q] >= th) << 16;
        c = add(c);
        if ((int)(c & 0xffffu) >= L.rank_lo) lo = tl;
        if ((int)(c >> 16) >= L.rank_hi) hi = th;
    }
    hi = L.rank_hi < 1 ? 0xffffffffu : hi | ((1u << LAST) - 1u);
    if (threadIdx.x == 0) {
        R->lo = lo;
        R->span = hi - lo;
        R->shift = (uint32_t)max(0, 32 - SEL_BITS - __clz((hi - lo) | 1u));
        R->need = (uint32_t)L.k;
        R->found = R->above = R->few = 0u;
        for (int i = 0; i <= SEL_PASSES; ++i) R->ticket[i] = 0u;
    }
}

// body(score, place, real) for the scores of a chunk [a, b) that thread t sees: places
// a + j SEL_T + t, SEL_I loads in flight.
template <typename Body>
__device__ __forceinline__ void sel_walk(const float *r, int64_t a, int64_t b, Body &&body) {
    for (; a + SEL_TILE <= b; a += SEL_TILE) {
        const float *q = r + a + threadIdx.x;
        float f[SEL_I];
#pragma unroll
        for (int j = 0; j < SEL_I; ++j) f[j] = q[j * SEL_T];
#pragma unroll
        for (int j = 0; j < SEL_I; ++j) body(f[j], true);
    }
    if (a < b) {
        const int m = (int)(b - a);
        float f[SEL_I];
#pragma unroll
        for (int j = 0; j < SEL_I; ++j) f[j] = r[a + min(j * SEL_T + (int)threadIdx.x, m - 1)];
#pragma unroll
        for (int j = 0; j < SEL_I; ++j) body(f[j], j * SEL_T + (int)threadIdx.x < m);
    }
}

__global__ void __launch_bounds__(SEL_T, 3) select_hist_kernel(SelLong L, int pass) {
    __shared__ uint32_t s_hist[SEL_BINS];
    __shared__ uint32_t s_warp[SEL_T / 32], s_above;
    __shared__ bool s_last;
    pdl_enter();
    SelRow *R = L.row + blockIdx.y;
    if (R->found) return;
    const float *r = L.scores + (int64_t)blockIdx.y * L.n;
    const uint32_t lo = R->lo, span = R->span, shift = R->shift;
    for (int i = threadIdx.x; i < SEL_BINS; i += SEL_T) s_hist[i] = 0u;
    if (threadIdx.x == 0) s_above = 0u;
    __syncthreads();
    const SelRange range(lo, span);
    uint32_t above = 0;
    // (a later pass mostly returns above: few blocks, each with several chunks)
    for (int c = blockIdx.x; c < L.chunks; c += gridDim.x) {
        const int64_t a = (int64_t)c * L.chunk, b = min(a + L.chunk, L.n);
        if (range.nan)
            sel_walk(r, a, b, [&](float f, bool real) {
                const uint32_t d = sel_key(f) - lo;
                if (!real) return;
                if (d <= span) atomicAdd(&s_hist[d >> shift], 1u); else ++above;
            });
        else
            sel_walk(r, a, b, [&](float f, bool real) {
                if (!real || !(f >= range.lo)) return;
                if (f > range.hi) ++above; else atomicAdd(&s_hist[(sel_key(f) - lo) >> shift], 1u);
            });
    }
    above = __reduce_add_sync(FULL, above);
    if ((threadIdx.x & 31) == 0 && above) atomicAdd(&s_above, above);
    __syncthreads();
    for (int i = threadIdx.x; i < SEL_BINS; i += SEL_T)
        if (s_hist[i]) atomicAdd(&R->hist[i], s_hist[i]);
    if (threadIdx.x == 0 && pass == 0 && s_above) atomicAdd(&R->above, s_above);
    if (!last_of_row(&R->ticket[pass], gridDim.x, &s_last)) return;
    // the bin that holds A: thread t owns PER bins, counted from the top
    constexpr int PER = SEL_BINS / SEL_T;
    static_assert(PER == 4, "a thread's bins are one vector");
    uint4 *bins = reinterpret_cast<uint4 *>(R->hist) + (SEL_BINS / PER - 1 - threadIdx.x);
    const uint4 four = __ldcg(bins);
    *bins = uint4{};
    const uint32_t h[PER] = {four.w, four.z, four.y, four.x}, mine = four.x + four.y + four.z + four.w;
    uint32_t before, total;
    sel_scan(mine, s_warp, before, total);
    const uint32_t over = pass == 0 ? __ldcg(&R->above) : 0u, want = R->need;
    __syncthreads();                       // every thread has read what one changes
    if (over >= want || over + total < want) {   // (first pass only) the bracket missed: all keys
        if (threadIdx.x == 0) {
            R->lo = 0u;
            R->span = 0xffffffffu;
            R->shift = 32u - SEL_BITS;
        }
        return;
    }
    const uint32_t need = want - over;
    if (before < need && before + mine >= need) {   // one thread
        uint32_t c = before;
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            if (c < need && c + h[q] >= need) {
                const uint32_t bin = (uint32_t)(SEL_BINS - 1 - (threadIdx.x * PER + q)) << shift;
                R->lo = lo + bin;
                R->span = min((1u << shift) - 1u, span - bin);   // the last bin ends with the range
                R->shift = shift > SEL_BITS ? shift - SEL_BITS : 0u;
                R->need = need - c;
                R->found = shift == 0u || h[q] <= (uint32_t)SEL_FEW;
            }
            c += h[q];
        }
    }
}

// One block finds A among the at most SEL_TIE keys of the range (what the last pass
// leaves), and every chunk's counts, by reading the row twice.
constexpr int SEL_TIE = 1 << (32 - 2 * SEL_BITS);
__device__ void select_alone(const SelLong &L, SelRow *R, const float *r, uint32_t *cnt, uint32_t *s_tie) {
    const uint32_t lo = R->lo, span = min(R->span, (uint32_t)SEL_TIE - 1u);   // (no more than s_tie holds, whatever is there)
    for (int i = threadIdx.x; i < SEL_TIE; i += SEL_T) s_tie[i] = 0u;
    __syncthreads();
    for (int64_t i = threadIdx.x; i < L.n; i += SEL_T) {
        const uint32_t d = sel_key(r[i]) - lo;
        if (d <= span) atomicAdd(&s_tie[d], 1u);
    }
    __syncthreads();
    uint32_t need = R->need, A = lo + span;
    for (int d = (int)span; d >= 0; --d) {
        A = lo + d;
        if (s_tie[d] >= need) break;
        need -= s_tie[d];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * L.chunks; i += SEL_T) cnt[i] = 0u;
    __threadfence();
    __syncthreads();
    for (int64_t i = threadIdx.x; i < L.n; i += SEL_T) {
        const uint32_t key = sel_key(r[i]);
        if (key >= A) atomicAdd(&cnt[2 * (i / L.chunk) + (key == A)], 1u);
    }
    if (threadIdx.x == 0) {
        R->lo = A;
        R->span = 0u;
        R->need = need;
    }
}

// Keys above the range in every chunk, and the few within it (or, a range of one key,
// its equals); the last block finds A among the few and turns the counts into the
// chunks' first places.
__global__ void __launch_bounds__(SEL_T, 3) select_count_kernel(SelLong L) {
    __shared__ uint32_t s_warp[SEL_T / 32], s_g, s_e, s_tie[SEL_TIE];
    __shared__ unsigned s_add[2 * (SEL_T / 32)];
    __shared__ bool s_last;
    pdl_enter();
    SelRow *R = L.row + blockIdx.y;
    const float *r = L.scores + (int64_t)blockIdx.y * L.n;
    uint32_t *cnt = L.counts + (int64_t)blockIdx.y * L.chunks * 2;
    const uint32_t lo = R->lo, span = R->span;
    if (threadIdx.x == 0) s_g = s_e = 0u;
    __syncthreads();
    const int64_t a = (int64_t)blockIdx.x * L.chunk, b = min(a + L.chunk, L.n);
    uint32_t g = 0, e = 0;
    const SelRange range(lo, span);
    auto within = [&](float f) {
        if (span == 0u) {
            ++e;
        } else {
            const uint32_t o = atomicAdd(&R->few, 1u);
            if (o < (uint32_t)SEL_FEW) R->list[o] = uint2{sel_key(f), blockIdx.x};
        }
    };
    if (range.nan)
        sel_walk(r, a, b, [&](float f, bool real) {
            if (!real) return;
            if (sel_key(f) - lo > span) ++g; else within(f);
        });
    else
        sel_walk(r, a, b, [&](float f, bool real) {
            if (!real || !(f >= range.lo)) return;
            if (f > range.hi) ++g; else within(f);
        });
    g = __reduce_add_sync(FULL, g);
    e = __reduce_add_sync(FULL, e);
    if ((threadIdx.x & 31) == 0) {
        if (g) atomicAdd(&s_g, g);
        if (e) atomicAdd(&s_e, e);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        cnt[2 * blockIdx.x] = s_g;
        cnt[2 * blockIdx.x + 1] = s_e;
    }
    if (!last_of_row(&R->ticket[SEL_PASSES], L.chunks, &s_last)) return;
    if (span) {
        const uint32_t want = R->need, few = __ldcg(&R->few);
        if (few > (uint32_t)SEL_FEW) {     // (a bracket that missed, and many ties: the passes ended above one key)
            select_alone(L, R, r, cnt, s_tie);
        } else {
            // the first ones in registers; more than that are rare, and read again each time
            const uint32_t t = threadIdx.x;
            const uint2 mine = t < few ? __ldcg(&R->list[t]) : uint2{0u, 0u};
            auto count = [&](uint32_t from) -> uint32_t {   // of keys at or above `from`
                uint32_t c = t < few && mine.x >= from;
                for (uint32_t i = t + SEL_T; i < few; i += SEL_T) c += __ldcg(&R->list[i]).x >= from;
                return c;
            };
            BlockAdd<SEL_T / 32> add(s_add);
            uint32_t A = lo;
            for (uint32_t bit = 1u << (31 - __clz(span)); bit; bit >>= 1)
                if (bit <= span - (A - lo) && add(count(A + bit)) >= want) A += bit;
            const uint32_t c = A == 0xffffffffu ? 0u : add(count(A + 1u));
            __syncthreads();
            if (threadIdx.x == 0) {
                R->lo = A;
                R->span = 0u;
                R->need = want - c;
            }
            for (uint32_t i = t; i < few; i += SEL_T) {
                const uint2 x = i == t ? mine : __ldcg(&R->list[i]);
                if (x.x >= A) atomicAdd(&cnt[2 * x.y + (x.x == A)], 1u);
            }
        }
        __threadfence();
        __syncthreads();
    }
    // exclusive scan of both counts over at most SEL_MAX_CHUNKS chunks
    constexpr int PER = SEL_MAX_CHUNKS / SEL_T;
    uint32_t vg[PER], ve[PER], tg = 0, te = 0;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
        const int c = threadIdx.x * PER + q;
        vg[q] = c < L.chunks ? __ldcg(&cnt[2 * c]) : 0u;
        ve[q] = c < L.chunks ? __ldcg(&cnt[2 * c + 1]) : 0u;
        tg += vg[q];
        te += ve[q];
    }
    uint32_t bg, be, total;
    sel_scan(tg, s_warp, bg, total);
    sel_scan(te, s_warp, be, total);
#pragma unroll
    for (int q = 0; q < PER; ++q) {
        const int c = threadIdx.x * PER + q;
        if (c < L.chunks) { cnt[2 * c] = bg; cnt[2 * c + 1] = be; }
        bg += vg[q];
        be += ve[q];
    }
}

// Each chunk writes its share of the selection, tile by tile: warp w holds the tile's
// places [w 32 SEL_I, (w+1) 32 SEL_I), lane l of step j place 32 j + l of them.
__global__ void __launch_bounds__(SEL_T) select_emit_kernel(SelLong L) {
    constexpr int NW = SEL_T / 32, I = SEL_I;
    __shared__ unsigned s_g[2][NW], s_e[2][NW];
    pdl_enter();
    const SelRow *R = L.row + blockIdx.y;
    const float *r = L.scores + (int64_t)blockIdx.y * L.n;
    const uint32_t *cnt = L.counts + (int64_t)blockIdx.y * L.chunks * 2;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t A = R->lo;
    const unsigned need = R->need;
    unsigned gt_at = cnt[2 * blockIdx.x], eq_at = cnt[2 * blockIdx.x + 1];   // before this tile
    const int64_t a = (int64_t)blockIdx.x * L.chunk, b = min(a + L.chunk, L.n);
    const int64_t out = (int64_t)blockIdx.y * L.k, o0 = out + gt_at + min(eq_at, need);
    int flip = 0;
    const SelRange range(A, 0u);
    for (int64_t t0 = a; t0 < b; t0 += SEL_TILE, flip ^= 1) {
        const int64_t first = t0 + warp * 32 * I;
        // one bit a step: above A, equal to A
        uint32_t mg = 0u, me = 0u;
        auto look = [&](float f, int j) {
            if (range.nan) {
                const uint32_t key = sel_key(f);
                mg |= (uint32_t)(key > A) << j;
                me |= (uint32_t)(key == A) << j;
            } else {
                if (f > range.lo) mg |= 1u << j;
                if (f == range.lo) me |= 1u << j;
            }
        };
        if (first + 32 * I <= b) {
            const float *q = r + first + lane;
            float f[I];
#pragma unroll
            for (int j = 0; j < I; ++j) f[j] = q[j * 32];
#pragma unroll
            for (int j = 0; j < I; ++j) look(f[j], j);
        } else {
            for (int j = 0; j < I; ++j)
                if (first + j * 32 + lane < b) look(r[first + j * 32 + lane], j);
        }
        const unsigned g = __reduce_add_sync(FULL, (unsigned)__popc(mg)), e = __reduce_add_sync(FULL, (unsigned)__popc(me));
        if (lane == 0) { s_g[flip][warp] = g; s_e[flip][warp] = e; }
        __syncthreads();
        const unsigned wg = lane < NW ? s_g[flip][lane] : 0u, we = lane < NW ? s_e[flip][lane] : 0u;
        unsigned G = gt_at + __reduce_add_sync(FULL, lane < warp ? wg : 0u);
        unsigned E = eq_at + __reduce_add_sync(FULL, lane < warp ? we : 0u);
        gt_at += __reduce_add_sync(FULL, wg);
        eq_at += __reduce_add_sync(FULL, we);
        if (g == 0 && (e == 0 || E >= need)) continue;
        for (unsigned any = __reduce_or_sync(FULL, mg | me); any; any &= any - 1) {
            const int j = __ffs(any) - 1;
            const unsigned gb = __ballot_sync(FULL, (mg >> j) & 1), eb = __ballot_sync(FULL, (me >> j) & 1);
            const unsigned below = lanes_below(lane);
            const unsigned er = E + __popc(eb & below);
            if (((gb >> lane) & 1) || (((eb >> lane) & 1) && er < need)) {
                const int64_t o = out + G + __popc(gb & below) + min(er, need);
                L.idx[o] = (int32_t)(first + j * 32 + lane);
            }
            G += __popc(gb);
            E += __popc(eb);
        }
    }
    if (!L.p) return;
    // the gate values of what this chunk wrote, fetched together
    __syncthreads();
    const int64_t o1 = out + gt_at + min(eq_at, need);
    for (int64_t o = o0 + threadIdx.x; o < o1; o += SEL_T) L.w[o] = L.p[(int64_t)blockIdx.y * L.n + __ldcg(L.idx + o)];
}

// Chunks of a long row: none below a tile, at most SEL_MAX_CHUNKS.
void sel_chunks(int64_t rows, int64_t n, int64_t *chunk, int *chunks) {
    // one round of the blocks that fit at once, three an SM: a block's start and end cost
    // as much as a tile
    const int64_t c = std::min<int64_t>(std::max<int64_t>(1, 3 * device_sm_count() / rows), SEL_MAX_CHUNKS);
    int64_t len = std::max<int64_t>((n + c - 1) / c, SEL_TILE);
    len = (len + SEL_TILE - 1) / SEL_TILE * SEL_TILE;
    *chunk = len;
    *chunks = (int)((n + len - 1) / len);
}

size_t sel_scratch(int64_t rows, int64_t n) {
    if (n <= SEL_CTA_MAX) return 0;
    const int64_t batch = std::min(rows, SEL_BATCH);
    int64_t chunk;
    int chunks;
    sel_chunks(batch, n, &chunk, &chunks);
    return (size_t)batch * (sizeof(SelRow) + ((size_t)chunks * 8 + 15) / 16 * 16);
}

bool sel_sizes_ok(int64_t rows, int64_t n, int64_t k) {
    const int64_t lim = int64_t(1) << 31;
    return rows >= 1 && n >= 1 && n < lim && k >= 1 && k <= n && rows < lim && rows * k < lim;
}

// ---------------------------------------------------------- the gradient --
// |x| may overflow fp32 (t tiny): it is no more than this, which keeps the shift finite.
constexpr float AX_MAX = 3.0e38f;
// A shifted pair of sums: sum e and sum dw e with e = 2^{m - |x|}; m is AX_MAX before the
// first score.  A NaN score or threshold is not in m, but makes its e NaN, and so the sums
// and the row's whole gradient.
struct GradAcc {
    float m;
    double sf, sg;
};
__device__ __forceinline__ GradAcc ga_merge(GradAcc a, GradAcc b) {
    const float m = fminf(a.m, b.m);
    const double fa = (double)exp2f(m - a.m), fb = (double)exp2f(m - b.m);
    return {m, a.sf * fa + b.sf * fb, a.sg * fa + b.sg * fb};
}
__device__ __forceinline__ GradAcc ga_warp(GradAcc a) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        GradAcc q{__shfl_xor_sync(FULL, a.m, o), __shfl_xor_sync(FULL, a.sf, o), __shfl_xor_sync(FULL, a.sg, o)};
        // the same operand order in both lanes of a pair, so all lanes hold the same bits
        a = ((threadIdx.x & 31) & o) ? ga_merge(q, a) : ga_merge(a, q);
    }
    return a;
}
__device__ __forceinline__ float ax_of(const XForm &xf, float r) {
    float a;                               // (fminf would drop a NaN)
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(a) : "f"(fabsf(xf(r))), "f"(AX_MAX));
    return a;
}

struct GradRow {
    float lam_hi, lam_lo, l2h;
    __device__ __forceinline__ GradRow(double lam, double inv_t) {
        lam_hi = (float)lam;
        lam_lo = (float)(lam - (double)lam_hi);
        l2h = vjp_scale2(inv_t);
    }
    __device__ __forceinline__ float operator()(float ax, float g) const { return vjp_term2(ax, g, l2h, lam_hi, lam_lo); }
};

// Row's entry j is in order (within [0, n), above the entry before it).
__device__ __forceinline__ bool idx_ok(const int32_t *idx, int64_t j, int64_t n) {
    const int32_t i = idx[j];
    return i >= 0 && i < n && (j == 0 || idx[j - 1] < i);
}

// A warp a row, its |x| in I registers a lane.  Rows of up to 1024 scores.
template <int I>
__global__ void __launch_bounds__(256)
select_grad_kernel(const float *__restrict__ scores, const double *__restrict__ b_in, const int32_t *__restrict__ idx_in,
                   const float *__restrict__ dw_in, int64_t rows, int n, int k, double inv_t, float *__restrict__ grad) {
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= rows) return;
    const float *r = scores + row * n;
    const int32_t *idx = idx_in + row * k;
    const float *dw = dw_in + row * k;
    float *out = grad + row * n;
    const XForm xf = make_xform(b_in[row], inv_t * LOG2E);
    float ax[I];
    float m = CUDART_INF_F;
#pragma unroll
    for (int j = 0; j < I; ++j) {
        const int i = j * 32 + lane;
        ax[j] = i < n ? ax_of(xf, r[i]) : CUDART_INF_F;
        m = fminf(m, ax[j]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fminf(m, __shfl_xor_sync(FULL, m, o));
    double sg = 0.0;
    float sf = 0.f;
#pragma unroll
    for (int j = 0; j < I; ++j) sf += exp2f(m - ax[j]);   // places behind the row: 2^-inf = 0
    bool bad = false;
    for (int j = lane; j < k; j += 32) {
        if (idx_ok(idx, j, n)) sg += (double)dw[j] * (double)exp2f(m - ax_of(xf, r[idx[j]]));
        else bad = true;
    }
    if (bad) sg = CUDART_NAN;
    const double lam = warp_sum(sg) / warp_sum((double)sf);
    const GradRow G(lam, inv_t);
#pragma unroll
    for (int j = 0; j < I; ++j) {
        const int i = j * 32 + lane;
        if (i < n) out[i] = G(ax[j], 0.f);
    }
    if (lam != lam) return;   // also: an index may be out of range
    __syncwarp();
    for (int j = lane; j < k; j += 32) out[idx[j]] = G(ax_of(xf, r[idx[j]]), dw[j]);
}

// Rows of up to 2048 G scores, G warps a row, read once: one more warp keeps a ring of
// chunks full, which holds a row and more than half of the next one.  The first pass
// over the row's chunks adds up, the second one writes and leaves them free, so the
// next row arrives meanwhile.  (One row a CTA in registers, n = 32768: nothing was
// read while a row was written; 86 us for 1024 rows, this 72 us.)
constexpr int SG_RING = 13;
template <int G>
struct GradShared {
    static constexpr int CHUNK = 8 * 32 * G;   // floats: two vectors a thread
    float ring[SG_RING][CHUNK];
    uint64_t full[SG_RING], empty[SG_RING], turn[1];
    double sf[G], sg[G];
    float m[G];
    int bad[G];
};

template <int G>
__global__ void __launch_bounds__(32 * G + 32, 16 / G)
select_grad_ring_kernel(const float *__restrict__ scores, const double *__restrict__ b_in,
                        const int32_t *__restrict__ idx_in, const float *__restrict__ dw_in, int rows, int n, int k,
                        double inv_t, float *__restrict__ grad) {
    constexpr int T = 32 * G, CHUNK = GradShared<G>::CHUNK, Z = 2;   // Z: selected scores a thread keeps at hand
    extern __shared__ __align__(16) unsigned char smem[];
    GradShared<G> &S = *reinterpret_cast<GradShared<G> *>(smem);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tid = threadIdx.x;
    if (tid == 0) {
        for (int i = 0; i < SG_RING; ++i) {
            mbar_init(&S.full[i], 1);
            mbar_init(&S.empty[i], G);
        }
        mbar_init(&S.turn[0], 1);
        mbar_init_fence();
    }
    pdl_enter();
    __syncthreads();
    if (warp == G) {
        if (lane == 0) rs_stream<SG_RING, CHUNK>(S.ring, S.full, S.empty, S.turn, 1, scores, rows, n);
        return;
    }
    Member<G> M;
    M.lane = lane;
    M.warp = warp;
    M.tid = tid;
    M.id = 0;
    int slot0 = 0, phase0 = 0;             // of the row's first chunk
    bool ring = true;                      // false once a wait has given up: rows are then read from memory
    int turn = 0;
    for (int row = blockIdx.x; row < rows; row += gridDim.x, ++turn) {
        const float *r = scores + (int64_t)row * n;
        const int32_t *idx = idx_in + (int64_t)row * k;
        const float *dw = dw_in + (int64_t)row * k;
        float *out = grad + (int64_t)row * n;
        const XForm xf = make_xform(b_in[row], inv_t * LOG2E);
        int head, body;
        rs_granules(r, n, head, body);
        int at[Z];
        float dwz[Z], axz[Z];
        bool bad = false;
#pragma unroll
        for (int z = 0; z < Z; ++z) {
            const int j = tid + z * T;
            at[z] = -1;
            dwz[z] = axz[z] = 0.f;
            if (j < k) {
                if (idx_ok(idx, j, n)) at[z] = idx[j]; else bad = true;
                dwz[z] = dw[j];
            }
        }
        // the scores outside the granules: at most one a lane of the first warp
        const int edge = warp ? -1 : lane < 4 ? (lane < head ? lane : -1) : (head + body + lane - 4 < n ? head + body + lane - 4 : -1);
        const float edge_ax = edge >= 0 ? ax_of(xf, r[edge]) : CUDART_INF_F;
        const float edge_m = fminf(edge_ax, AX_MAX);
        const double edge_sf = edge >= 0 ? (double)exp2f(edge_m - edge_ax) : 0.0;
        float m = edge_m;
        double sf = edge_sf;
        auto add = [&](const float (&ax)[8]) {
            float lm = ax[0];
#pragma unroll
            for (int i = 1; i < 8; ++i) lm = fminf(lm, ax[i]);
            if (lm < m) {
                sf *= (double)exp2f(lm - m);
                m = lm;
            }
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) s += exp2f(m - ax[i]);
            sf += (double)s;
        };
        // eight |x| of this thread in chunk c, which is in `slot` (past the row's end: inf)
        auto eight = [&](int slot, int a, float (&ax)[8]) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int o = 4 * (tid + u * T);
                float4 v{};
                if (ring) v = lds128(reinterpret_cast<const float4 *>(S.ring[slot] + o));
                else if (a + o < body) v = float4{r[head + a + o], r[head + a + o + 1], r[head + a + o + 2], r[head + a + o + 3]};
                const bool real = a + o < body;
                ax[4 * u] = real ? ax_of(xf, v.x) : CUDART_INF_F;
                ax[4 * u + 1] = real ? ax_of(xf, v.y) : CUDART_INF_F;
                ax[4 * u + 2] = real ? ax_of(xf, v.z) : CUDART_INF_F;
                ax[4 * u + 3] = real ? ax_of(xf, v.w) : CUDART_INF_F;
            }
        };
        int slot = slot0, phase = phase0;
        bool ok = true;
        if (ring)                          // the whole row first: a wait that gives up is then known to all
            for (int a = 0; a < body; a += CHUNK) {
                ok = ok && waited(mbar_wait(&S.full[slot], phase, RING_WAIT_CAP), GIVE_UP_READ, turn);
                if (ok) {
                    float ax[8];
                    eight(slot, a, ax);
                    add(ax);
                }
                if (++slot == SG_RING) { slot = 0; phase ^= 1; }
            }
        const int end_slot = slot, end_phase = phase;
        // the smallest |x| of the row
        float wm = m;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) wm = fminf(wm, __shfl_xor_sync(FULL, wm, o));
        const bool warp_bad = __any_sync(FULL, !ok);
        if (lane == 0) {
            S.m[warp] = wm;
            S.bad[warp] = warp_bad;
        }
        M.sync();
        float lo = S.m[0];
        int gave_up = S.bad[0];
#pragma unroll
        for (int w = 1; w < G; ++w) {
            lo = fminf(lo, S.m[w]);
            gave_up |= S.bad[w];
        }
        if (gave_up || !ring) {            // this row and the later ones from memory
            ring = false;
            m = edge_m;
            sf = edge_sf;
            for (int a = 0; a < body; a += CHUNK) {
                float ax[8];
                eight(0, a, ax);
                add(ax);
            }
            lo = m;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) lo = fminf(lo, __shfl_xor_sync(FULL, lo, o));
            M.sync();
            if (lane == 0) S.m[warp] = lo;
            M.sync();
            for (int w = 0; w < G; ++w) lo = fminf(lo, S.m[w]);
        }
        sf *= (double)exp2f(lo - m);
        // the selected scores' part, out of the ring
        auto ax_at = [&](int i) -> float {
            const int o = i - head;
            if (!ring || o < 0 || o >= body) return ax_of(xf, r[i]);
            int q = slot0 + o / CHUNK;
            if (q >= SG_RING) q -= SG_RING;
            return ax_of(xf, S.ring[q][o & (CHUNK - 1)]);
        };
        double sg = 0.0;
#pragma unroll
        for (int z = 0; z < Z; ++z)
            if (at[z] >= 0) {
                axz[z] = ax_at(at[z]);
                sg += (double)dwz[z] * (double)exp2f(lo - axz[z]);
            }
        for (int j0 = Z * T; j0 < k; j0 += 4 * T) {   // (many selected: four at a time, their loads together)
            int i[4], before[4];
            float d[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int j = min(j0 + u * T + tid, k - 1);
                i[u] = idx[j];
                before[u] = idx[j - 1];
                d[u] = dw[j];
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (j0 + u * T + tid >= k) continue;
                if (i[u] >= 0 && i[u] < n && before[u] < i[u]) sg += (double)d[u] * (double)exp2f(lo - ax_at(i[u]));
                else bad = true;
            }
        }
        if (bad) sg = CUDART_NAN;
        sf = warp_sum(sf);
        sg = warp_sum(sg);
        if (lane == 0) {
            S.sf[warp] = sf;
            S.sg[warp] = sg;
        }
        M.sync();
        sf = S.sf[0];
        sg = S.sg[0];
#pragma unroll
        for (int w = 1; w < G; ++w) {
            sf += S.sf[w];
            sg += S.sg[w];
        }
        const double lam = sg / sf;
        const GradRow grow(lam, inv_t);
        // the second pass: -(f/t) lambda everywhere, each chunk free behind it
        const bool wide = ((reinterpret_cast<uintptr_t>(out + head) & 15) == 0);
        slot = slot0;
        for (int a = 0; a < body; a += CHUNK) {
            float ax[8];
            eight(slot, a, ax);
            if (ring) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.empty[slot]);
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int o = a + 4 * (tid + u * T);
                if (o >= body) continue;
                float4 v{grow(ax[4 * u], 0.f), grow(ax[4 * u + 1], 0.f), grow(ax[4 * u + 2], 0.f), grow(ax[4 * u + 3], 0.f)};
                float *to = out + head + o;
                if (wide) {
                    *reinterpret_cast<float4 *>(to) = v;
                } else {
                    to[0] = v.x;
                    to[1] = v.y;
                    to[2] = v.z;
                    to[3] = v.w;
                }
            }
            if (++slot == SG_RING) slot = 0;
        }
        if (edge >= 0) out[edge] = grow(edge_ax, 0.f);
        M.sync();                          // also: the sums' room is free
        if (lam == lam) {
#pragma unroll
            for (int z = 0; z < Z; ++z)
                if (at[z] >= 0) out[at[z]] = grow(axz[z], dwz[z]);
            for (int j0 = Z * T; j0 < k; j0 += 4 * T) {
                int i[4];
                float d[4], x[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int j = min(j0 + u * T + tid, k - 1);
                    i[u] = idx[j];
                    d[u] = dw[j];
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) x[u] = r[i[u]];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (j0 + u * T + tid < k) out[i[u]] = grow(ax_of(xf, x[u]), d[u]);
            }
        }
        slot0 = end_slot;
        phase0 = end_phase;
    }
}

// Longer rows: a pass of shifted sums, then a pass that writes.
struct GradLong {
    const float *scores;
    const double *b;
    const int32_t *idx;
    const float *dw;
    float *grad;
    int64_t n, k, chunk;
    int chunks;
    double inv_t;
    GradAcc *part;   // [row][chunk]
};
constexpr int GL_T = 256;

__device__ __forceinline__ GradAcc ga_block(GradAcc a, GradAcc *s) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    a = ga_warp(a);
    if (lane == 0) s[warp] = a;
    __syncthreads();
    a = s[0];
    for (int w = 1; w < GL_T / 32; ++w) a = ga_merge(a, s[w]);
    __syncthreads();
    return a;
}

__global__ void __launch_bounds__(GL_T) select_grad_sum_kernel(GradLong L) {
    __shared__ GradAcc s_acc[GL_T / 32];
    pdl_enter();
    const int64_t row = blockIdx.y;
    const float *r = L.scores + row * L.n;
    const int32_t *idx = L.idx + row * L.k;
    const float *dw = L.dw + row * L.k;
    const XForm xf = make_xform(L.b[row], L.inv_t * LOG2E);
    const int64_t a0 = (int64_t)blockIdx.x * L.chunk, a1 = min(a0 + L.chunk, L.n);
    GradAcc acc{AX_MAX, 0.0, 0.0};
    for (int64_t i0 = a0; i0 < a1; i0 += 8 * GL_T) {
        float ax[8];
        float m = acc.m;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int64_t i = i0 + q * GL_T + threadIdx.x;
            ax[q] = i < a1 ? ax_of(xf, r[i]) : CUDART_INF_F;
            m = fminf(m, ax[q]);
        }
        if (m < acc.m) {
            acc.sf *= (double)exp2f(m - acc.m);
            acc.m = m;
        }
        float s = 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q) s += exp2f(m - ax[q]);
        acc.sf += (double)s;
    }
    // this block's share of the row's selected scores
    const int64_t per = (L.k + L.chunks - 1) / L.chunks;
    const int64_t j0 = (int64_t)blockIdx.x * per, j1 = min(j0 + per, L.k);
    bool bad = false;
    for (int64_t j = j0 + threadIdx.x; j < j1; j += GL_T) {
        if (!idx_ok(idx, j, L.n)) { bad = true; continue; }
        const float ax = ax_of(xf, r[idx[j]]);
        if (ax < acc.m) {
            const double sc = (double)exp2f(ax - acc.m);
            acc.sf *= sc;
            acc.sg *= sc;
            acc.m = ax;
        }
        acc.sg += (double)dw[j] * (double)exp2f(acc.m - ax);
    }
    acc = ga_block(acc, s_acc);
    if (__syncthreads_or(bad)) acc.sg = CUDART_NAN;
    if (threadIdx.x == 0) L.part[row * L.chunks + blockIdx.x] = acc;
}

__global__ void __launch_bounds__(GL_T) select_grad_apply_kernel(GradLong L) {
    __shared__ GradAcc s_acc[GL_T / 32];
    __shared__ int64_t s_at[2];
    pdl_enter();
    const int64_t row = blockIdx.y;
    const float *r = L.scores + row * L.n;
    const int32_t *idx = L.idx + row * L.k;
    const float *dw = L.dw + row * L.k;
    float *out = L.grad + row * L.n;
    const XForm xf = make_xform(L.b[row], L.inv_t * LOG2E);
    GradAcc acc{AX_MAX, 0.0, 0.0};
    for (int c = threadIdx.x; c < L.chunks; c += GL_T) acc = ga_merge(acc, L.part[row * L.chunks + c]);
    acc = ga_block(acc, s_acc);
    const double lam = acc.sg / acc.sf;
    const GradRow G(lam, L.inv_t);
    const int64_t a0 = (int64_t)blockIdx.x * L.chunk, a1 = min(a0 + L.chunk, L.n);
    for (int64_t i = a0 + threadIdx.x; i < a1; i += GL_T) out[i] = G(ax_of(xf, r[i]), 0.f);
    if (lam != lam) return;
    if (threadIdx.x < 2) {   // the selected scores of this chunk: idx ascends
        const int64_t v = threadIdx.x ? a1 : a0;
        int64_t lo = 0, hi = L.k;
        while (lo < hi) {
            const int64_t mid = (lo + hi) >> 1;
            if (idx[mid] < v) lo = mid + 1; else hi = mid;
        }
        s_at[threadIdx.x] = lo;
    }
    __syncthreads();
    for (int64_t j = s_at[0] + threadIdx.x; j < s_at[1]; j += GL_T) out[idx[j]] = G(ax_of(xf, r[idx[j]]), dw[j]);
}

void grad_chunks(int64_t rows, int64_t n, int64_t *chunk, int *chunks) {
    int64_t c = std::max<int64_t>(1, 1184 / rows);
    c = std::min<int64_t>(c, (n + 4095) / 4096);
    int64_t len = (n + c - 1) / c;
    len = (len + 8 * GL_T - 1) / (8 * GL_T) * (8 * GL_T);
    *chunk = len;
    *chunks = (int)((n + len - 1) / len);
}

constexpr int64_t GRAD_BATCH = 1024;

size_t grad_scratch(int64_t rows, int64_t n) {
    if (n <= SEL_CTA_MAX) return 0;
    int64_t chunk;
    int chunks;
    const int64_t batch = std::min(rows, GRAD_BATCH);
    grad_chunks(batch, n, &chunk, &chunks);
    return (size_t)batch * chunks * sizeof(GradAcc);
}

bool scratch_ok(const void *scratch, int64_t have, size_t need) {
    return need == 0 || (scratch && (reinterpret_cast<uintptr_t>(scratch) & 15) == 0 && have >= (int64_t)need);
}

template <int I>
cudaError_t run_select_warp(const float *s, const float *p, int64_t rows, int64_t n, int64_t k, int32_t *idx, float *w,
                            cudaStream_t st) {
    return launch_k(select_warp_kernel<I>, (unsigned)((rows + 7) / 8), 256, 0, st, s, p, rows, (int)n, (int)k, idx, w);
}
template <int G>
cudaError_t run_grad_ring(const float *s, const double *b, const int32_t *idx, const float *dw, int64_t rows, int64_t n,
                          int64_t k, double inv_t, float *grad, cudaStream_t st) {
    auto kern = select_grad_ring_kernel<G>;
    const void *fn = reinterpret_cast<const void *>(kern);
    cudaError_t e = set_max_dynamic_smem(fn, sizeof(GradShared<G>));
    if (e != cudaSuccess) return e;
    int ctas = 0;
    if ((e = resident_ctas(fn, 32 * G + 32, sizeof(GradShared<G>), &ctas)) != cudaSuccess) return e;
    return launch_k(kern, (unsigned)std::min<int64_t>(rows, ctas), 32 * G + 32, sizeof(GradShared<G>), st, s, b, idx, dw,
                    (int)rows, (int)n, (int)k, inv_t, grad);
}
template <int I>
cudaError_t run_grad(const float *s, const double *b, const int32_t *idx, const float *dw, int64_t rows, int64_t n,
                     int64_t k, double inv_t, float *grad, cudaStream_t st) {
    return launch_k(select_grad_kernel<I>, (unsigned)((rows + 7) / 8), 256, 0, st, s, b, idx, dw, rows, (int)n, (int)k, inv_t,
                    grad);
}

}  // namespace

cudaError_t select_give_up(int kind, int turn) { return set_give_up((GiveUp)kind, turn); }
}  // namespace lapsum

using namespace lapsum;

extern "C" {

// (what a device's launch set-up keeps is host memory: no exception leaves a C entry)
int64_t lapsum_select_scratch(int64_t rows, int64_t n, int64_t k) try {
    return sel_sizes_ok(rows, n, k) ? (int64_t)sel_scratch(rows, n) : LAPSUM_ERR_ARG;
} catch (...) {
    return LAPSUM_ERR_ALLOC;
}

int lapsum_select(const float *scores, const float *p, int64_t rows, int64_t n, int64_t k, int32_t *idx, float *w,
                  void *scratch, int64_t scratch_bytes, struct CUstream_st *stream_in) try {
    if (!scores || !idx || !sel_sizes_ok(rows, n, k) || (p == nullptr) != (w == nullptr)) return LAPSUM_ERR_ARG;
    if (!multiples_of(4, scores, p, idx, w)) return LAPSUM_ERR_ARG;
    if (!scratch_ok(scratch, scratch_bytes, sel_scratch(rows, n))) return LAPSUM_ERR_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream_in);
    if (n <= SEL_CTA_MAX) {
        Launch L("select_topk", st);
        cudaError_t e;
        if (n <= 32) e = run_select_warp<1>(scores, p, rows, n, k, idx, w, st);
        else if (n <= 64) e = run_select_warp<2>(scores, p, rows, n, k, idx, w, st);
        else if (n <= 128) e = run_select_warp<4>(scores, p, rows, n, k, idx, w, st);
        else if (n <= 256) e = run_select_warp<8>(scores, p, rows, n, k, idx, w, st);
        else if (n <= 512) e = run_select_warp<16>(scores, p, rows, n, k, idx, w, st);
        else if (n <= SEL_WARP_MAX) e = run_select_warp<32>(scores, p, rows, n, k, idx, w, st);
        else e = run_select_rows(scores, p, rows, n, k, idx, w, st);
        LAPSUM_TRY(e);
        return LAPSUM_OK;
    }
    const int64_t batch = std::min(rows, SEL_BATCH);
    SelLong A{};
    sel_chunks(batch, n, &A.chunk, &A.chunks);
    A.n = n;
    A.k = k;
    // the sample holds about mu of the k best: a Poisson count, below mu - 4 sqrt(mu), or
    // none at all from mu = 12 on, less than once in 10^5 rows
    const double mu = (double)k * SEL_SAMPLE / (double)n, sd = std::sqrt(mu);
    A.rank_lo = (int)std::ceil(mu + 4.0 * sd + 4.0);
    A.rank_hi = (int)std::floor(mu - 4.0 * sd);
    if (A.rank_hi < 1 && mu >= 12.0) A.rank_hi = 1;
    A.row = static_cast<SelRow *>(scratch);
    A.counts = reinterpret_cast<uint32_t *>(A.row + batch);
    for (int64_t r0 = 0; r0 < rows; r0 += batch) {
        const unsigned m = (unsigned)std::min(batch, rows - r0);
        A.scores = scores + r0 * n;
        A.p = p ? p + r0 * n : nullptr;
        A.idx = idx + r0 * k;
        A.w = w ? w + r0 * k : nullptr;
        const dim3 grid((unsigned)A.chunks, m);
        { Launch L("select_sample", st); LAPSUM_TRY(launch_k(select_sample_kernel, m, 256, 0, st, A)); }
        for (int pass = 0; pass < SEL_PASSES; ++pass) {
            Launch L("select_hist", st);
            // the later passes mostly return at once: few blocks
            const dim3 some((unsigned)(pass ? std::min<int64_t>(A.chunks, std::max<int64_t>(1, device_sm_count() / m)) : A.chunks), m);
            LAPSUM_TRY(launch_k(select_hist_kernel, some, SEL_T, 0, st, A, pass));
        }
        { Launch L("select_count", st); LAPSUM_TRY(launch_k(select_count_kernel, grid, SEL_T, 0, st, A)); }
        { Launch L("select_emit", st); LAPSUM_TRY(launch_k(select_emit_kernel, grid, SEL_T, 0, st, A)); }
    }
    return LAPSUM_OK;
} catch (...) {
    return LAPSUM_ERR_ALLOC;
}

int64_t lapsum_select_backward_scratch(int64_t rows, int64_t n) {
    return sel_sizes_ok(rows, n, 1) ? (int64_t)grad_scratch(rows, n) : LAPSUM_ERR_ARG;
}

int lapsum_select_backward(const float *scores, const double *b, const int32_t *idx, const float *dw, int64_t rows,
                           int64_t n, int64_t k, double t, float *grad, void *scratch, int64_t scratch_bytes,
                           struct CUstream_st *stream_in) try {
    if (!scores || !b || !idx || !dw || !grad || !sel_sizes_ok(rows, n, k)) return LAPSUM_ERR_ARG;
    if (!multiples_of(4, scores, idx, dw, grad) || !multiples_of(8, b)) return LAPSUM_ERR_ARG;
    if (!(t >= LAPSUM_T_MIN && t <= LAPSUM_T_MAX)) return LAPSUM_ERR_ARG;
    if (!scratch_ok(scratch, scratch_bytes, grad_scratch(rows, n))) return LAPSUM_ERR_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream_in);
    const double inv_t = 1.0 / t;
    if (n <= SEL_CTA_MAX) {
        Launch L("select_grad", st);
        cudaError_t e;
        if (n <= 128) e = run_grad<4>(scores, b, idx, dw, rows, n, k, inv_t, grad, st);
        else if (n <= 1024) e = run_grad<32>(scores, b, idx, dw, rows, n, k, inv_t, grad, st);
        else if (n <= 2048) e = run_grad_ring<1>(scores, b, idx, dw, rows, n, k, inv_t, grad, st);
        else if (n <= 4096) e = run_grad_ring<2>(scores, b, idx, dw, rows, n, k, inv_t, grad, st);
        else if (n <= 8192) e = run_grad_ring<4>(scores, b, idx, dw, rows, n, k, inv_t, grad, st);
        else if (n <= 16384) e = run_grad_ring<8>(scores, b, idx, dw, rows, n, k, inv_t, grad, st);
        else e = run_grad_ring<16>(scores, b, idx, dw, rows, n, k, inv_t, grad, st);
        LAPSUM_TRY(e);
        return LAPSUM_OK;
    }
    const int64_t batch = std::min(rows, GRAD_BATCH);
    GradLong A{};
    grad_chunks(batch, n, &A.chunk, &A.chunks);
    A.n = n;
    A.k = k;
    A.inv_t = inv_t;
    A.part = static_cast<GradAcc *>(scratch);
    for (int64_t r0 = 0; r0 < rows; r0 += batch) {
        A.scores = scores + r0 * n;
        A.b = b + r0;
        A.idx = idx + r0 * k;
        A.dw = dw + r0 * k;
        A.grad = grad + r0 * n;
        const dim3 grid((unsigned)A.chunks, (unsigned)std::min(batch, rows - r0));
        { Launch L("select_grad_sum", st); LAPSUM_TRY(launch_k(select_grad_sum_kernel, grid, GL_T, 0, st, A)); }
        { Launch L("select_grad_apply", st); LAPSUM_TRY(launch_k(select_grad_apply_kernel, grid, GL_T, 0, st, A)); }
    }
    return LAPSUM_OK;
} catch (...) {
    return LAPSUM_ERR_ALLOC;
}

}  // extern "C"
