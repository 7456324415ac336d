// k_tokens.cu -- token rows to the experts' slots and back, and their gradients.
//
// All four passes are bound by memory: each row is read or written once, with
// fp32 sums in registers and one rounding.
//   dispatch           copies: walks the tokens' places, so that the slots of one
//                      token follow one another and its row is read once
//   combine,           sums over a token's places: warps own stretches of one
//   dispatch_backward  token's row and add the slots in order
//   combine_backward   walks the tokens' places as dispatch does: per place one
//                      product row and one dot product
// Rows are moved in vectors of VB bytes, the widest that divides a row and suits
// every pointer.  Where that is two bytes (an odd number of 16-bit values) and the row
// is not short, it is stored in the 16-byte granules of the OUTPUT row instead, and an input row that lies
// differently is read by its own granules, two a vector, and shifted into place (the
// second one is the next lane's first: a hit in L1); only the values before and behind
// the granules go one by one.  At 8192 x 4 rows of 2047 bf16: dispatch 41 -> 34 us,
// combine_backward 101 -> 68 us.  (With four- or eight-byte vectors at hand those are
// faster: 131 against 141 us at 4002 bf16.)
//
// Loads are never conditional: past a row's end the last granule is read again, for
// a place that is none slot 0, and the value not used.  (A condition each is a
// branch each, and the loads of a batch then follow one another: measured 667 us
// instead of 240 at 9999 tokens x 1001 fp32 values.)
#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "give_up.cuh"
#include "lapsum_kernels.h"
#include "lapsum_launch.h"
#include "route_common.cuh"

namespace lapsum {
namespace {

// A tensor's 16-byte granules that lie wholly in it start at lo .. hi.
struct Span {
    uintptr_t lo, hi;
};
struct Rows {
    const unsigned char *a, *b;   // inputs (combine_backward: h and g)
    unsigned char *out;
    const float *w;
    float *dw;
    Span sa, sb;                  // of the inputs
    int64_t row_bytes;
    int64_t tokens, slots;
    const int32_t *slot_token, *token_offsets, *token_slots, *token_entries;
};

// Bytes of a vector; SHIFTED: granules of 16, shifted into place.
constexpr int SHIFTED = 0;

// 16 bytes out of two granules, from byte `shift` (0 .. 15) on.
__device__ __forceinline__ uint4 shifted(const uint4 &a, const uint4 &b, int shift) {
    uint32_t x0 = a.x, x1 = a.y, x2 = a.z, x3 = a.w, x4 = b.x, x5 = b.y;
    if (shift & 8) { x0 = a.z; x1 = a.w; x2 = b.x; x3 = b.y; x4 = b.z; x5 = b.w; }
    if (shift & 4) { x0 = x1; x1 = x2; x2 = x3; x3 = x4; x4 = x5; }
    const int bits = (shift & 3) * 8;
    return uint4{__funnelshift_r(x0, x1, bits), __funnelshift_r(x1, x2, bits), __funnelshift_r(x2, x3, bits),
                 __funnelshift_r(x3, x4, bits)};
}

// A vector of N values of a row on its way: load() asks for it, get() has it.
template <typename T, int VB>
struct Vec {
    static constexpr int BYTES = VB == SHIFTED ? 16 : VB, N = BYTES / (int)sizeof(T);
    using P = Pack<T, BYTES>;
    using V = typename VecOf<BYTES>::type;
    V a, b;
    // vector c of the row at p (past `last`: that one)
    __device__ __forceinline__ void load(const unsigned char *p, int c, int last, const Span &s) {
        if (VB != SHIFTED) {
            a = reinterpret_cast<const V *>(p)[min(c, last)];
        } else {
            const uintptr_t g = (reinterpret_cast<uintptr_t>(p) & ~uintptr_t(15)) + 16 * (int64_t)c;
            a = *reinterpret_cast<const V *>(min(max(g, s.lo), s.hi));
            b = *reinterpret_cast<const V *>(min(max(g + 16, s.lo), s.hi));
        }
    }
    __device__ __forceinline__ P get(const unsigned char *p, int c, const Span &s) const {
        P x;
        if constexpr (VB != SHIFTED) {
            x.raw = a;
        } else {
            const int shift = (int)(reinterpret_cast<uintptr_t>(p) & 15);
            const uintptr_t g = reinterpret_cast<uintptr_t>(p) - shift + 16 * (int64_t)c;
            if (g < s.lo || g + (shift ? 16 : 0) > s.hi) {   // the tensor's outermost granules
#pragma unroll
                for (int i = 0; i < N; ++i) x.v[i] = reinterpret_cast<const T *>(p)[(int64_t)c * N + i];
            } else {
                x.raw = shifted(a, b, shift);
            }
        }
        return x;
    }
};

// An output row's vectors: `head` bytes before the first, `vecs` of them; then the rest.
template <typename T, int VB>
struct Cut {
    int head, vecs;
    __device__ __forceinline__ Cut(const unsigned char *out, int64_t row_bytes) {
        head = VB == SHIFTED ? (int)((16 - (reinterpret_cast<uintptr_t>(out) & 15)) & 15) : 0;
        vecs = (int)((row_bytes - head) / Vec<T, VB>::BYTES);
    }
    // The value before or behind the vectors that this lane takes; -1: none.
    __device__ __forceinline__ int64_t single(int lane, int64_t row_bytes) const {
        if (VB != SHIFTED) return -1;
        const int64_t first = head / (int)sizeof(T), from = first + (int64_t)vecs * Vec<T, VB>::N;
        const int64_t i = lane < 16 ? lane : from + lane - 16;
        return (lane < 16 ? lane < first : i < row_bytes / (int64_t)sizeof(T)) ? i : -1;
    }
};

// A warp takes `per` places and a stretch of 32 U vectors of their rows.
template <typename T, int VB, int U>
__global__ void __launch_bounds__(256) dispatch_kernel(Rows R, int per, int64_t stretches) {
    using X = Vec<T, VB>;
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int64_t p0 = item / stretches * per;
    if (p0 >= R.slots) return;
    const int c0 = (int)(item % stretches) * 32 * U + lane;
    const int64_t used = R.token_offsets[R.tokens];
    int32_t slot = -1, token = -1;
    if (lane < per && p0 + lane < R.slots) {
        slot = p0 + lane < used ? R.token_slots[p0 + lane] : (int32_t)(p0 + lane);   // behind the last slot: zero
        if (p0 + lane < used && slot >= 0 && slot < R.slots) token = R.slot_token[slot];
    }
    X v[U];
    int32_t have = -2;
    for (int q = 0; q < per; ++q) {
        const int32_t s = __shfl_sync(FULL, slot, q), t = __shfl_sync(FULL, token, q);
        if (s < 0 || s >= R.slots) continue;
        const bool real = t >= 0 && t < R.tokens;
        unsigned char *dst = R.out + s * R.row_bytes;
        const Cut<T, VB> cut(dst, R.row_bytes);
        const unsigned char *src = R.a + (real ? t : 0) * R.row_bytes + cut.head;
        if (VB == SHIFTED || t != have) {  // (shifted, the slots of a token lie differently: from L1)
            have = t;
#pragma unroll
            for (int u = 0; u < U; ++u) v[u].load(src, c0 + u * 32, cut.vecs - 1, R.sa);
        }
        auto *to = reinterpret_cast<typename X::V *>(dst + cut.head);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c0 + u * 32 < cut.vecs) to[c0 + u * 32] = real ? v[u].get(src, c0 + u * 32, R.sa).raw : typename X::V{};
        if (VB == SHIFTED && c0 == lane) {
            const int64_t i = cut.single(lane, R.row_bytes);
            if (i >= 0) reinterpret_cast<T *>(dst)[i] = real ? reinterpret_cast<const T *>(src - cut.head)[i] : T{};
        }
    }
}

// `parts` warps sum a token's row over its slots, each every parts-th stretch of 32 U
// vectors; B slots' vectors are in flight together.
template <typename T, int VB, int U, int B, bool WEIGHTED>
__global__ void __launch_bounds__(256) to_tokens_kernel(Rows R, int parts) {
    using X = Vec<T, VB>;
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int64_t token = item / parts;
    if (token >= R.tokens) return;
    const int64_t o0 = max(R.token_offsets[token], 0), o1 = min((int64_t)R.token_offsets[token + 1], R.slots);
    // 32 places' slots and weights, one a lane
    int32_t slot = -1;
    float w = 0.f;
    auto places = [&](int64_t p0) {
        slot = -1;
        w = 0.f;
        if (p0 + lane < o1) {
            slot = R.token_slots[p0 + lane];
            if (slot >= R.slots) slot = -1;
            if (WEIGHTED) {
                const int32_t e = R.token_entries[p0 + lane];
                if (e >= 0 && e < R.slots) w = R.w[e]; else slot = -1;
            }
        }
    };
    places(o0);
    unsigned char *dst = R.out + token * R.row_bytes;
    const Cut<T, VB> cut(dst, R.row_bytes);
    const int64_t single = cut.single(lane, R.row_bytes);
    for (int64_t b0 = (item % parts) * 32 * U; b0 < max(cut.vecs, 1); b0 += (int64_t)parts * 32 * U) {
        const int c0 = (int)b0 + lane;
        float acc[U][X::N], one = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < X::N; ++i) acc[u][i] = 0.f;
        for (int64_t p0 = o0; p0 < o1; p0 += 32) {
            if (o1 - o0 > 32) places(p0);
            const int cnt = (int)min(o1 - p0, (int64_t)32);
            for (int q = 0; q < cnt; q += B) {
                X v[B][U];
                T e[B];
                int32_t s[B];
#pragma unroll
                for (int z = 0; z < B; ++z) {
                    s[z] = __shfl_sync(FULL, slot, (q + z) & 31);
                    if (q + z >= cnt) s[z] = -1;
                    const unsigned char *src = R.a + max(s[z], 0) * R.row_bytes;
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        v[z][u].load(src + cut.head, c0 + u * 32, cut.vecs - 1, R.sa);
                    if (VB == SHIFTED) e[z] = reinterpret_cast<const T *>(src)[max(single, int64_t(0))];
                }
#pragma unroll
                for (int z = 0; z < B; ++z) {
                    const float ws = WEIGHTED ? __shfl_sync(FULL, w, (q + z) & 31) : 1.f;
                    if (s[z] < 0) continue;
                    const unsigned char *src = R.a + s[z] * R.row_bytes + cut.head;
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        if (VB == SHIFTED && c0 + u * 32 >= cut.vecs) continue;
                        const typename X::P x = v[z][u].get(src, c0 + u * 32, R.sa);
#pragma unroll
                        for (int i = 0; i < X::N; ++i) acc[u][i] = fmaf(ws, to_f32(x.v[i]), acc[u][i]);
                    }
                    if (VB == SHIFTED) one = fmaf(ws, to_f32(e[z]), one);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (c0 + u * 32 >= cut.vecs) continue;
            typename X::P o;
#pragma unroll
            for (int i = 0; i < X::N; ++i) o.v[i] = from_f32<T>(acc[u][i]);
            reinterpret_cast<typename X::V *>(dst + cut.head)[c0 + u * 32] = o.raw;
        }
        if (VB == SHIFTED && b0 == 0 && single >= 0) reinterpret_cast<T *>(dst)[single] = from_f32<T>(one);
    }
}

// The same for long rows, through shared memory: one warp walks ahead over the
// places of its CTA's tokens and keeps a ring of row segments full (one bulk copy
// each), four or eight warps add them up.  The loads in flight do not hang on registers or on
// the chain offsets -> slot -> row, and a token with many slots streams like many
// tokens.  A row need not start on 16 bytes: the copy takes the granules around it,
// those that reach past the tensor excepted, whose values are read from memory.
constexpr int TS_RING = 5;
constexpr int TS_VP = 2;                   // vectors a thread holds of a segment
template <int TS_T>                        // threads that add
struct TokensShared {
    static constexpr int SEG = TS_T * 16 * TS_VP;
    unsigned char seg[TS_RING][SEG + 16];
    uint4 note[TS_RING];                   // what the adding warps need to know of a segment: see Note
    uint64_t full[TS_RING], empty[TS_RING];
};
// A segment's note: where its first value is in memory, its weight, and packed: the
// bytes of the stage that are there end at `hi` (16 bits) and start at `lo` (8), the
// first value's place in the stage (4), flags (4).
constexpr uint32_t NOTE_FIRST = 1u, NOTE_LAST = 2u, NOTE_NONE = 4u;   // of a token's segments; no slot at all

template <typename T, bool EVEN, bool WEIGHTED, int TS_T>
__global__ void __launch_bounds__(TS_T + 32)
to_tokens_ring_kernel(const __grid_constant__ Rows R, int seg_bytes, int segs) {   // (copied, R costs 2 us of 61 at 16384 x 4 x 2048 bf16)
    constexpr int VP = TS_VP, N = 16 / (int)sizeof(T), PER = VP * N;   // values of a vector, of a thread
    extern __shared__ __align__(16) unsigned char smem[];
    TokensShared<TS_T> &S = *reinterpret_cast<TokensShared<TS_T> *>(smem);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < TS_RING; ++i) {
            mbar_init(&S.full[i], 1);
            mbar_init(&S.empty[i], TS_T / 32);
        }
        mbar_init_fence();
    }
    pdl_enter();
    __syncthreads();
    const int64_t items = R.tokens * segs;
    const unsigned char *base = R.a;
    if (warp == TS_T / 32) {               // ---- the warp that walks ahead, one place a lane
        const uintptr_t first_granule = (reinterpret_cast<uintptr_t>(base) + 15) & ~uintptr_t(15);
        const uintptr_t end_granule = (reinterpret_cast<uintptr_t>(base) + (uintptr_t)(R.slots * R.row_bytes)) & ~uintptr_t(15);
        // ahead: the item after next's offsets; the next one's slots and entries
        auto offsets = [&](int64_t item, int64_t &a, int64_t &b) {
            a = b = 0;
            if (item < items) {
                const int64_t t = item / segs;
                a = max(R.token_offsets[t], 0);
                b = min((int64_t)R.token_offsets[t + 1], R.slots);
            }
        };
        auto places = [&](int64_t p0, int64_t end, int32_t &s, int32_t &e) {
            s = e = -1;
            if (p0 + lane < end) {
                s = R.token_slots[p0 + lane];
                if (WEIGHTED) e = R.token_entries[p0 + lane];
            }
        };
        uint4 note{};
        uintptr_t from = 0;                // of this lane's copy
        uint32_t bytes = 0, into = 0;
        auto prepare = [&](int32_t s, int32_t e, int64_t seg) {
            if (s >= R.slots || (WEIGHTED && (e < 0 || e >= R.slots))) s = -1;
            const int64_t off = seg * seg_bytes;
            const uintptr_t u = reinterpret_cast<uintptr_t>(base + (s < 0 ? 0 : (int64_t)s * R.row_bytes) + off);
            const uintptr_t len = (uintptr_t)min((int64_t)seg_bytes, R.row_bytes - off);
            const uintptr_t g0 = u & ~uintptr_t(15), end = min((u + len + 15) & ~uintptr_t(15), end_granule);
            from = max(g0, first_granule);
            bytes = s >= 0 && end > from ? (uint32_t)(end - from) : 0u;
            into = (uint32_t)(from - g0);
            note.x = (uint32_t)u;
            note.y = (uint32_t)(u >> 32);
            note.z = __float_as_uint(WEIGHTED && s >= 0 ? R.w[e] : 1.f);
            note.w = (bytes ? (uint32_t)(end - g0) << 16 | into << 8 : 0u) | (uint32_t)(u - g0) << 4 | (s < 0 ? NOTE_NONE : 0u);
        };
        int stage = 0, phase = 1;
        uint32_t sent = 0;
        bool ok = true;
        int64_t item = blockIdx.x, o0, o1, n0, n1;
        int32_t slot, entry;
        offsets(item, o0, o1);
        offsets(item + gridDim.x, n0, n1);
        places(o0, o1, slot, entry);
        prepare(slot, entry, item % segs);
        for (; item < items; item += gridDim.x) {
            int64_t f0, f1;
            places(n0, n1, slot, entry);
            offsets(item + 2 * (int64_t)gridDim.x, f0, f1);
            const int64_t count = max(o1 - o0, int64_t(1));   // a token without slots: one note of none
            for (int64_t p0 = 0; p0 < count; p0 += 32) {
                if (p0) {
                    int32_t s, e;
                    places(o0 + p0, o1, s, e);
                    prepare(s, e, item % segs);
                }
                const int cnt = (int)min(count - p0, (int64_t)32);
                for (int q = 0; q < cnt; ++q) {
                    if (lane == q && ok) {
                        ok = mbar_wait(&S.empty[stage], phase, RING_WAIT_CAP);
                        if (ok) {
                            uint4 x = note;
                            x.w |= (p0 + q == 0 ? NOTE_FIRST : 0u) | (p0 + q + 1 == count ? NOTE_LAST : 0u);
                            S.note[stage] = x;
                            fence_proxy_async_smem();   // the stage was read
                            mbar_expect_tx(&S.full[stage], bytes);
                            if (bytes) bulk_load(S.seg[stage] + into, reinterpret_cast<const void *>(from), bytes, &S.full[stage]);
                        }
                    }
                    ++sent;
                    if (++stage == TS_RING) { stage = 0; phase ^= 1; }
                }
                if (!__all_sync(FULL, ok)) break;
            }
            ok = __all_sync(FULL, ok);
            if (!ok) break;
            o0 = n0;
            o1 = n1;
            n0 = f0;
            n1 = f1;
            prepare(slot, entry, (item + gridDim.x) % segs);
        }
        // no CTA ends with copies in flight: the last of every stage
        if (lane == 0)
            for (uint32_t z = 0; z < min(sent, (uint32_t)TS_RING); ++z) {
                const uint32_t q = sent - 1 - z;
                mbar_wait(&S.full[q % TS_RING], (q / TS_RING) & 1, RING_WAIT_CAP);
            }
        return;
    }
    // ---- the warps that add: vectors t + v TS_T of a segment (EVEN), or values t + j TS_T
    const int tid = threadIdx.x;
    int stage = 0, phase = 0, turn = 0;
    bool ok = true;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x, ++turn) {
        const int64_t token = item / segs, off = item % segs * seg_bytes;
        const int len = (int)min((int64_t)seg_bytes, R.row_bytes - off);
        float acc[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] = 0.f;
        for (bool last = false; !last;) {
            ok = ok && waited(mbar_wait(&S.full[stage], phase, RING_WAIT_CAP), GIVE_UP_READ, turn);
            if (!ok) break;
            const uint4 note = S.note[stage];
            const float w = __uint_as_float(note.z);
            last = note.w & NOTE_LAST;
            if (!(note.w & NOTE_NONE)) {
                const unsigned char *seg = S.seg[stage];
                if (EVEN) {
                    Pack<T, 16> x[VP];
#pragma unroll
                    for (int v = 0; v < VP; ++v)   // past the segment's end: of the stage still, and not stored
                        x[v].raw = *reinterpret_cast<const uint4 *>(seg + (tid + v * TS_T) * 16);
#pragma unroll
                    for (int v = 0; v < VP; ++v)
#pragma unroll
                        for (int i = 0; i < N; ++i) acc[v * N + i] = fmaf(w, to_f32(x[v].v[i]), acc[v * N + i]);
                } else {
                    const int at = (note.w >> 4) & 15, lo = (note.w >> 8) & 255, hi = note.w >> 16;
                    if (lo == 0 && at + len <= hi) {
                        T x[PER];
#pragma unroll
                        for (int j = 0; j < PER; ++j) x[j] = *reinterpret_cast<const T *>(seg + at + (tid + j * TS_T) * (int)sizeof(T));
#pragma unroll
                        for (int j = 0; j < PER; ++j) acc[j] = fmaf(w, to_f32(x[j]), acc[j]);
                    } else {               // the tensor's first or last granule: some values from memory
                        const unsigned char *src = reinterpret_cast<const unsigned char *>((uintptr_t)note.x | (uintptr_t)note.y << 32);
#pragma unroll
                        for (int j = 0; j < PER; ++j) {
                            const int o = (tid + j * TS_T) * (int)sizeof(T), b = at + o;
                            if (o >= len) break;
                            const T x = b >= lo && b + (int)sizeof(T) <= hi ? *reinterpret_cast<const T *>(seg + b)
                                                                           : *reinterpret_cast<const T *>(src + o);
                            acc[j] = fmaf(w, to_f32(x), acc[j]);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.empty[stage]);
            if (++stage == TS_RING) { stage = 0; phase ^= 1; }
        }
        unsigned char *dst = R.out + token * R.row_bytes + off;
        if (!ok)                           // a wait gave up: no stale row is left
#pragma unroll
            for (int i = 0; i < PER; ++i) acc[i] = CUDART_NAN_F;
        if (EVEN) {
#pragma unroll
            for (int v = 0; v < VP; ++v) {
                const int o = (tid + v * TS_T) * 16;
                if (o >= len) break;
                Pack<T, 16> x;
#pragma unroll
                for (int i = 0; i < N; ++i) x.v[i] = from_f32<T>(acc[v * N + i]);
                *reinterpret_cast<uint4 *>(dst + o) = x.raw;
            }
        } else {
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const int o = (tid + j * TS_T) * (int)sizeof(T);
                if (o >= len) break;
                *reinterpret_cast<T *>(dst + o) = from_f32<T>(acc[j]);
            }
        }
    }
}

// G warps (of one CTA) take P places together: grad_h of their slots and grad_w of
// their entries.  The places follow one another in the tokens' lists, so the rows of
// g that they share are read once (the loads meet in L1), stretch by stretch: place
// by place, 32 KB rows fell out of the caches between two places of a token (8192 x 4
// rows of 8192 fp32: 494 us, the time of reading g four times).
template <typename T, int VB, int G, int P>
__global__ void __launch_bounds__(256) combine_grad_kernel(Rows R) {
    using X = Vec<T, VB>;
    constexpr int U = VB == SHIFTED || VB >= 8 ? 2 : 4;
    __shared__ float s_dot[8][P];
    pdl_enter();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int part = warp % G;
    const int64_t p0 = ((int64_t)blockIdx.x * (8 / G) + warp / G) * P;
    const int64_t used = R.token_offsets[R.tokens];
    // the places' slots, entries, tokens and weights, one a lane
    int32_t slots = -1, entries = -1, tokens = -1;
    float ws = 0.f;
    if (lane < P && p0 + lane < R.slots) {
        if (p0 + lane < used) {
            slots = R.token_slots[p0 + lane];
            entries = R.token_entries[p0 + lane];
            if (slots < 0 || slots >= R.slots || entries < 0 || entries >= R.slots) {
                slots = -1;
            } else {
                tokens = R.slot_token[slots];
                ws = R.w[entries];
                if (tokens < 0 || tokens >= R.tokens) slots = -1;
            }
        } else {
            slots = (int32_t)(p0 + lane);  // behind the last slot: zero
        }
    }
    int32_t s[P], t[P];
    float w[P], dot[P];
#pragma unroll
    for (int q = 0; q < P; ++q) {
        s[q] = __shfl_sync(FULL, slots, q);
        t[q] = __shfl_sync(FULL, tokens, q);
        w[q] = __shfl_sync(FULL, ws, q);
        dot[q] = 0.f;
    }
    const int most = (int)(R.row_bytes / X::BYTES);   // vectors of a row at most
    for (int b = part * 32 * U; b < most; b += G * 32 * U) {
        X hv[P][U], gv[P][U];
        const int c = b + lane;
#pragma unroll
        for (int q = 0; q < P; ++q) {
            const Cut<T, VB> cut(R.out + max(s[q], 0) * R.row_bytes, R.row_bytes);
            const unsigned char *h = R.a + max(s[q], 0) * R.row_bytes + cut.head, *g = R.b + max(t[q], 0) * R.row_bytes + cut.head;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                hv[q][u].load(h, c + u * 32, cut.vecs - 1, R.sa);
                gv[q][u].load(g, c + u * 32, cut.vecs - 1, R.sb);
            }
        }
#pragma unroll
        for (int q = 0; q < P; ++q) {
            if (s[q] < 0) continue;
            unsigned char *dst = R.out + s[q] * R.row_bytes;
            const Cut<T, VB> cut(dst, R.row_bytes);
            const unsigned char *h = R.a + s[q] * R.row_bytes + cut.head, *g = R.b + max(t[q], 0) * R.row_bytes + cut.head;
            auto *to = reinterpret_cast<typename X::V *>(dst + cut.head);
            if (t[q] < 0) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (c + u * 32 < cut.vecs) to[c + u * 32] = typename X::V{};
                continue;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (c + u * 32 >= cut.vecs) continue;
                const typename X::P hx = hv[q][u].get(h, c + u * 32, R.sa), gx = gv[q][u].get(g, c + u * 32, R.sb);
                typename X::P o;
#pragma unroll
                for (int i = 0; i < X::N; ++i) {
                    const float gf = to_f32(gx.v[i]);
                    dot[q] = fmaf(to_f32(hx.v[i]), gf, dot[q]);
                    o.v[i] = from_f32<T>(w[q] * gf);
                }
                to[c + u * 32] = o.raw;
            }
        }
    }
    if (VB == SHIFTED && part == 0) {
#pragma unroll
        for (int q = 0; q < P; ++q) {
            if (s[q] < 0) continue;
            unsigned char *dst = R.out + s[q] * R.row_bytes;
            const int64_t i = Cut<T, VB>(dst, R.row_bytes).single(lane, R.row_bytes);
            if (i < 0) continue;
            const float gf = t[q] < 0 ? 0.f : to_f32(reinterpret_cast<const T *>(R.b + t[q] * R.row_bytes)[i]);
            if (t[q] >= 0) dot[q] = fmaf(to_f32(reinterpret_cast<const T *>(R.a + s[q] * R.row_bytes)[i]), gf, dot[q]);
            reinterpret_cast<T *>(dst)[i] = from_f32<T>(w[q] * gf);
        }
    }
#pragma unroll
    for (int q = 0; q < P; ++q) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) dot[q] += __shfl_xor_sync(FULL, dot[q], d);
        if (G > 1) {
            if (lane == 0) s_dot[warp][q] = dot[q];
            __syncthreads();
            dot[q] = 0.f;
            for (int i = 0; i < G; ++i) dot[q] += s_dot[warp - part + i][q];
        }
        const int32_t e = __shfl_sync(FULL, entries, q);
        if (s[q] >= 0 && t[q] >= 0 && part == 0 && lane == 0) R.dw[e] = dot[q];
    }
}

// ------------------------------------------------------------------ host --
bool route_ok(const lapsum_route *R) {
    const int64_t lim = int64_t(1) << 31;
    return R && R->tokens >= 1 && R->tokens < lim && R->slots >= 1 && R->slots < lim && R->slot_token &&
           R->token_offsets && R->token_slots && R->token_entries &&
           multiples_of(4, R->slot_token, R->token_offsets, R->token_slots, R->token_entries);
}
int type_size(int32_t type) {
    return type == LAPSUM_TYPE_F32 ? 4 : type == LAPSUM_TYPE_F16 || type == LAPSUM_TYPE_BF16 ? 2 : 0;
}
bool rows_ok(int32_t type, int64_t d, const lapsum_route *R) {
    return type_size(type) && d >= 1 && d < (int64_t(1) << 30) && route_ok(R);   // (vectors are counted in 32 bits)
}
uintptr_t bits_of(std::initializer_list<const void *> ps) {
    uintptr_t u = 0;
    for (const void *p : ps) u |= reinterpret_cast<uintptr_t>(p);
    return u;
}
bool aligned(int32_t type, std::initializer_list<const void *> ps) {
    return (bits_of(ps) & (uintptr_t)(type_size(type) - 1)) == 0;
}
// The widest vector that divides a row and suits every pointer; SHIFTED instead of
// one 16-bit value at a time, but for short rows, which are all edges (dispatch, its
// gradient, combine, its gradients in us, a value at a time and shifted: 301 experts of
// 603 tokens at d = 77, 24, 41, 38, 40 and 58, 66, 68, 101; 64 experts, 3e7 values at
// d = 257, 41, 89, 82, 56 and 40, 96, 110, 73; at d = 1025, 36, 33, 34, 50 and 29, 33, 34, 39).
int vec_bytes(int64_t row_bytes, std::initializer_list<const void *> ps) {
    const uintptr_t u = bits_of(ps) | (uintptr_t)row_bytes;
    if (u & 2) return row_bytes < 640 ? 2 : SHIFTED;
    return u & 4 ? 4 : u & 8 ? 8 : 16;
}
// f(std::integral_constant<int, VB>) for the VB at hand (no SHIFTED and no 2 for
// four-byte values).
template <typename T, typename F>
cudaError_t with_vec(int vb, F &&f) {
    switch (vb) {
        case 16: return f(std::integral_constant<int, 16>());
        case 8: return f(std::integral_constant<int, 8>());
        case 4: return f(std::integral_constant<int, 4>());
        default:
            if constexpr (sizeof(T) == 2) {
                return vb == 2 ? f(std::integral_constant<int, 2>()) : f(std::integral_constant<int, SHIFTED>());
            }
            return cudaErrorInvalidValue;
    }
}
Span span_of(const void *p, int64_t bytes) {
    const uintptr_t u = reinterpret_cast<uintptr_t>(p);
    return {(u + 15) & ~uintptr_t(15), ((u + (uintptr_t)bytes) & ~uintptr_t(15)) - 16};
}

Rows make_rows(const lapsum_route *R, int64_t row_bytes, const void *a, int64_t a_rows, void *out) {
    Rows A{};
    A.a = static_cast<const unsigned char *>(a);
    A.out = static_cast<unsigned char *>(out);
    A.sa = span_of(a, a_rows * row_bytes);
    A.row_bytes = row_bytes;
    A.tokens = R->tokens;
    A.slots = R->slots;
    A.slot_token = R->slot_token;
    A.token_offsets = R->token_offsets;
    A.token_slots = R->token_slots;
    A.token_entries = R->token_entries;
    return A;
}

constexpr int64_t GRID_MAX = 0x7fffffff;

template <typename T, int VB>
int64_t vectors(const Rows &A) { return (A.row_bytes + Vec<T, VB>::BYTES - 1) / Vec<T, VB>::BYTES; }   // of a row

template <typename T>
cudaError_t run_dispatch(const Rows &A, int vb, cudaStream_t st) {
    return with_vec<T>(vb, [&](auto v) {
        constexpr int VB = v, U = VB == SHIFTED || VB == 4 ? 4 : 2;
        // few places: one each, so that every SM has some; many: eight in a row, so
        // that a token's row is read once for all of its slots
        const int per = A.slots >= 8192 ? 8 : 1;
        const int64_t stretches = (vectors<T, VB>(A) + 32 * U - 1) / (32 * U);
        const int64_t blocks = ((A.slots + per - 1) / per * stretches + 7) / 8;
        if (blocks > GRID_MAX) return cudaErrorInvalidConfiguration;
        return launch_k(dispatch_kernel<T, VB, U>, (unsigned)blocks, 256, 0, st, A, per, stretches);
    });
}

template <typename T, int VB, int B, bool WEIGHTED>
cudaError_t run_to_tokens(const Rows &A, cudaStream_t st) {
    // vectors in flight over the B slots: about 128 bytes a lane, so narrow vectors
    // come in larger numbers
    constexpr int U = VB == SHIFTED ? 4 / B : VB == 16 ? (B == 1 ? 4 : 8 / B) : VB == 8 ? 4 : 8;
    const int64_t stretches = (vectors<T, VB>(A) + 32 * U - 1) / (32 * U);
    // a warp a token, which reads the token's places once, unless that leaves SMs
    // without work: then the row is shared by several
    const int64_t want = 32 * (int64_t)device_sm_count();
    const int parts = (int)std::min(stretches, std::max<int64_t>(1, (want + A.tokens - 1) / A.tokens));
    const int64_t blocks = (A.tokens * parts + 7) / 8;
    if (blocks > GRID_MAX) return cudaErrorInvalidConfiguration;
    return launch_k(to_tokens_kernel<T, VB, U, B, WEIGHTED>, (unsigned)blocks, 256, 0, st, A, parts);
}
template <typename T, bool EVEN, bool WEIGHTED, int TS_T>
cudaError_t run_to_tokens_ring(const Rows &A, cudaStream_t st) {
    auto kern = to_tokens_ring_kernel<T, EVEN, WEIGHTED, TS_T>;
    const void *fn = reinterpret_cast<const void *>(kern);
    constexpr size_t smem = sizeof(TokensShared<TS_T>);
    cudaError_t e = set_max_dynamic_smem(fn, smem);
    if (e != cudaSuccess) return e;
    int ctas = 0;
    if ((e = resident_ctas(fn, TS_T + 32, smem, &ctas)) != cudaSuccess) return e;
    const int segs = (int)((A.row_bytes + TokensShared<TS_T>::SEG - 1) / TokensShared<TS_T>::SEG);
    // even segments, whole vectors of every type
    const int seg = (int)(((A.row_bytes + segs - 1) / segs + 15) / 16 * 16);
    const int64_t items = A.tokens * segs;
    return launch_k(kern, (unsigned)std::min<int64_t>(items, ctas), TS_T + 32, smem, st, A, seg, segs);
}
template <typename T, bool EVEN, bool WEIGHTED>
cudaError_t run_to_tokens_vp(const Rows &A, cudaStream_t st) {
    return A.row_bytes > TokensShared<128>::SEG ? run_to_tokens_ring<T, EVEN, WEIGHTED, 256>(A, st)
                                              : run_to_tokens_ring<T, EVEN, WEIGHTED, 128>(A, st);
}
template <typename T, bool WEIGHTED>
cudaError_t run_to_tokens_vb(const Rows &A, int vb, cudaStream_t st) {
    // long rows, and enough of them to fill the SMs' rings: see the two kernels
    if (A.row_bytes >= 1024 && A.slots * A.row_bytes >= (int64_t(4) << 20) && A.row_bytes < (int64_t(1) << 30))
        return vb == 16 ? run_to_tokens_vp<T, true, WEIGHTED>(A, st) : run_to_tokens_vp<T, false, WEIGHTED>(A, st);
    return with_vec<T>(vb, [&](auto v) {
        constexpr int VB = v;
        // slots of a token on average
        if (A.slots <= A.tokens) return run_to_tokens<T, VB, 1, WEIGHTED>(A, st);
        if (A.slots <= 2 * A.tokens) return run_to_tokens<T, VB, 2, WEIGHTED>(A, st);
        return run_to_tokens<T, VB, 4, WEIGHTED>(A, st);
    });
}
template <bool WEIGHTED>
cudaError_t run_to_tokens_type(const Rows &A, int32_t type, int vb, cudaStream_t st) {
    if (type == LAPSUM_TYPE_F32) return run_to_tokens_vb<float, WEIGHTED>(A, vb, st);
    if (type == LAPSUM_TYPE_F16) return run_to_tokens_vb<__half, WEIGHTED>(A, vb, st);
    return run_to_tokens_vb<__nv_bfloat16, WEIGHTED>(A, vb, st);
}

template <typename T>
cudaError_t run_combine_grad(const Rows &A, int vb, cudaStream_t st) {
    return with_vec<T>(vb, [&](auto v) {
        constexpr int VB = v;
        // places are many: a warp four of them (one, shifted: the granules in flight fill
        // the registers); they are few: a CTA each
        constexpr int P = VB == SHIFTED ? 1 : 4;
        if (A.slots >= 4096)
            return launch_k(combine_grad_kernel<T, VB, 1, P>, (unsigned)((A.slots + 8 * P - 1) / (8 * P)), 256, 0, st, A);
        return launch_k(combine_grad_kernel<T, VB, 8, 1>, (unsigned)A.slots, 256, 0, st, A);
    });
}

}  // namespace

cudaError_t tokens_give_up(int kind, int turn) { return set_give_up((GiveUp)kind, turn); }
}  // namespace lapsum

using namespace lapsum;

extern "C" {

// (what a device's launch set-up keeps is host memory: no exception leaves a C entry)
int lapsum_dispatch(const void *x, int32_t type, int64_t d, const lapsum_route *R, void *out,
                    struct CUstream_st *stream_in) try {
    if (!x || !out || !rows_ok(type, d, R) || !aligned(type, {x, out})) return LAPSUM_ERR_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream_in);
    const int64_t rb = d * type_size(type);
    const Rows A = make_rows(R, rb, x, R->tokens, out);
    const int vb = vec_bytes(rb, {x, out});
    Launch L("dispatch", st);
    if (type == LAPSUM_TYPE_F32) LAPSUM_TRY(run_dispatch<uint32_t>(A, vb, st));
    else LAPSUM_TRY(run_dispatch<uint16_t>(A, vb, st));
    return LAPSUM_OK;
} catch (...) {
    return LAPSUM_ERR_ALLOC;
}

int lapsum_dispatch_backward(const void *g, int32_t type, int64_t d, const lapsum_route *R, void *grad_x,
                             struct CUstream_st *stream_in) try {
    if (!g || !grad_x || !rows_ok(type, d, R) || !aligned(type, {g, grad_x})) return LAPSUM_ERR_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream_in);
    const int64_t rb = d * type_size(type);
    const Rows A = make_rows(R, rb, g, R->slots, grad_x);
    Launch L("dispatch_grad", st);
    LAPSUM_TRY(run_to_tokens_type<false>(A, type, vec_bytes(rb, {g, grad_x}), st));
    return LAPSUM_OK;
} catch (...) {
    return LAPSUM_ERR_ALLOC;
}

int lapsum_combine(const void *h, const float *w, int32_t type, int64_t d, const lapsum_route *R, void *y,
                   struct CUstream_st *stream_in) try {
    if (!h || !w || !y || !rows_ok(type, d, R) || !aligned(type, {h, y}) || !multiples_of(4, w)) return LAPSUM_ERR_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream_in);
    const int64_t rb = d * type_size(type);
    Rows A = make_rows(R, rb, h, R->slots, y);
    A.w = w;
    Launch L("combine", st);
    LAPSUM_TRY(run_to_tokens_type<true>(A, type, vec_bytes(rb, {h, y}), st));
    return LAPSUM_OK;
} catch (...) {
    return LAPSUM_ERR_ALLOC;
}

int lapsum_combine_backward(const void *h, const float *w, const void *g, int32_t type, int64_t d,
                            const lapsum_route *R, void *grad_h, float *grad_w, struct CUstream_st *stream_in) try {
    if (!h || !w || !g || !grad_h || !grad_w || !rows_ok(type, d, R) || !aligned(type, {h, g, grad_h}) ||
        !multiples_of(4, w, grad_w))
        return LAPSUM_ERR_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream_in);
    const int64_t rb = d * type_size(type);
    Rows A = make_rows(R, rb, h, R->slots, grad_h);
    A.b = static_cast<const unsigned char *>(g);
    A.sb = span_of(g, R->tokens * rb);
    A.w = w;
    A.dw = grad_w;
    const int vb = vec_bytes(rb, {h, g, grad_h});
    // entries that went nowhere have no place to be reached from: zero first
    LAPSUM_TRY(cudaMemsetAsync(grad_w, 0, sizeof(float) * (size_t)R->slots, st));
    Launch L("combine_grad", st);
    if (type == LAPSUM_TYPE_F32) LAPSUM_TRY(run_combine_grad<float>(A, vb, st));
    else if (type == LAPSUM_TYPE_F16) LAPSUM_TRY(run_combine_grad<__half>(A, vb, st));
    else LAPSUM_TRY(run_combine_grad<__nv_bfloat16>(A, vb, st));
    return LAPSUM_OK;
} catch (...) {
    return LAPSUM_ERR_ALLOC;
}

}  // extern "C"
