// k_clip.cu -- the global norm over many gradient tensors, and clipping to it.
//
//   norm = sqrt(sum_i g_i^2),  out_i = g_i min(1, max_norm / (norm + 1e-6)).
//
// Two launches per group of up to CLIP_GROUP tensors: the first leaves one fp64
// partial sum a block, the second adds the partials up in a fixed order (every
// block the same sum), forms the scale and writes.  The scale is rounded to fp32, half
// a step of an fp32 output and far below a 16-bit one's: products and values then stay
// in 32 bits.  An output carries that rounding, the product's and its type's.  The tensors' addresses and
// sizes travel as kernel parameters: nothing is copied to the device, and a
// captured graph holds them.  Tensors are cut into chunks of CLIP_VECS 16-byte
// vectors; a block takes an even share of consecutive chunks, the second launch each
// share from its end, where the first has left the caches filled.
#include <algorithm>
#include <cmath>
#include <vector>

#include "lapsum_kernels.h"
#include "lapsum_launch.h"
#include "route_common.cuh"

namespace lapsum {
namespace {

constexpr int CT = 256;
constexpr int CLIP_GROUP = 512;
constexpr int CLIP_SMALL = 48;
constexpr int CLIP_VECS = 2048;            // 32 KB a chunk
constexpr int CLIP_BLOCKS = 1184;          // eight blocks an SM
constexpr double CLIP_EPS = 1e-6;

struct ClipTensor {
    const void *in;
    void *out;
    int64_t n;
    uint32_t first;                        // its first chunk
    int32_t type;
};
template <int N>
struct ClipTable {
    ClipTensor t[N];
    int count;
    uint32_t chunks;
};

// A tensor's values: `head` up to the first 16-byte boundary of the input, then
// whole vectors, then the rest.
struct ClipSpan {
    int64_t head, vecs, tail;
};
__host__ __device__ inline ClipSpan clip_span(const void *in, int64_t n, int size) {
    ClipSpan s;
    s.head = ((16 - (reinterpret_cast<uintptr_t>(in) & 15)) & 15) / size;
    if (s.head > n) s.head = n;
    const int per = 16 / size;
    s.vecs = (n - s.head) / per;
    s.tail = n - s.head - s.vecs * per;
    return s;
}
__host__ __device__ inline int clip_size(int32_t type) { return type == LAPSUM_TYPE_F32 ? 4 : 2; }

template <int N>
__device__ __forceinline__ int clip_find(const ClipTable<N> &T, uint32_t chunk) {
    int lo = 0, hi = T.count - 1;          // the last tensor whose first chunk is <= chunk
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (T.t[mid].first <= chunk) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// A block's chunks: an even share of consecutive ones.
struct ClipShare {
    uint32_t from, to;
    __device__ __forceinline__ explicit ClipShare(uint32_t chunks) {
        from = (uint32_t)((uint64_t)chunks * blockIdx.x / gridDim.x);
        to = (uint32_t)((uint64_t)chunks * (blockIdx.x + 1) / gridDim.x);
    }
};

__device__ __forceinline__ double sum_block(double v, double *s) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    v = warp_sum(v);
    if (lane == 0) s[warp] = v;
    __syncthreads();
    double t = 0.0;
    for (int w = 0; w < CT / 32; ++w) t += s[w];
    __syncthreads();
    return t;
}

// Squares of one vector: in fp32 where that neither overflows nor loses small
// values (each product rounds once; the sum goes on in fp64), else in fp64.
template <typename T>
__device__ __forceinline__ double square_sum(const Pack<T, 16> &v) {
    constexpr int N = 16 / (int)sizeof(T);
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float x = to_f32(v.v[i]);
        q = fmaf(x, x, q);
    }
    if (q > 1e-28f && q < 1e38f) return (double)q;
    double d = 0.0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const double x = (double)to_f32(v.v[i]);
        d = fma(x, x, d);
    }
    return d;
}

template <typename T>
__device__ __forceinline__ double norm_chunk(const ClipTensor &t, uint32_t c) {
    constexpr int U = 8;
    const ClipSpan s = clip_span(t.in, t.n, (int)sizeof(T));
    const T *in = static_cast<const T *>(t.in);
    const uint4 *v = reinterpret_cast<const uint4 *>(in + s.head);
    const int64_t a = (int64_t)c * CLIP_VECS, b = min(a + CLIP_VECS, s.vecs);
    double acc = 0.0;
    for (int64_t i = a + threadIdx.x; i < b; i += CT * U) {
        Pack<T, 16> p[U];
#pragma unroll
        for (int u = 0; u < U; ++u) p[u].raw = i + u * CT < b ? v[i + u * CT] : uint4{};
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + u * CT < b) acc += square_sum<T>(p[u]);
    }
    if (c == 0) {
        double x = 0.0;
        if (threadIdx.x < s.head) x = (double)to_f32(in[threadIdx.x]);
        else if (threadIdx.x >= 32 && threadIdx.x - 32 < s.tail) x = (double)to_f32(in[t.n - s.tail + threadIdx.x - 32]);
        acc = fma(x, x, acc);
    }
    return acc;
}

template <int N>
__global__ void __launch_bounds__(CT) clip_norm_kernel(const __grid_constant__ ClipTable<N> T, double *part) {
    __shared__ double s_red[CT / 32];
    pdl_enter();
    double acc = 0.0;
    const ClipShare share(T.chunks);
    int at = clip_find(T, share.from);
    for (uint32_t c = share.from; c < share.to; ++c) {
        while (at + 1 < T.count && T.t[at + 1].first <= c) ++at;
        const ClipTensor &t = T.t[at];
        const uint32_t lc = c - t.first;
        if (t.type == LAPSUM_TYPE_F32) acc += norm_chunk<float>(t, lc);
        else if (t.type == LAPSUM_TYPE_F16) acc += norm_chunk<__half>(t, lc);
        else acc += norm_chunk<__nv_bfloat16>(t, lc);
    }
    acc = sum_block(acc, s_red);
    if (threadIdx.x == 0) part[blockIdx.x] = acc;
}

template <typename T>
__device__ __forceinline__ void scale_chunk(const ClipTensor &t, uint32_t c, float scale) {
    constexpr int U = 4, N = 16 / (int)sizeof(T);
    const ClipSpan s = clip_span(t.in, t.n, (int)sizeof(T));
    const T *in = static_cast<const T *>(t.in);
    T *out = static_cast<T *>(t.out);
    const uint4 *v = reinterpret_cast<const uint4 *>(in + s.head);
    const bool wide = (reinterpret_cast<uintptr_t>(out + s.head) & 15) == 0;
    const int64_t a = (int64_t)c * CLIP_VECS, b = min(a + CLIP_VECS, s.vecs);
    for (int64_t i = a + threadIdx.x; i < b; i += CT * U) {
        Pack<T, 16> p[U];
#pragma unroll
        for (int u = 0; u < U; ++u) p[u].raw = i + u * CT < b ? v[i + u * CT] : uint4{};
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i + u * CT >= b) continue;
#pragma unroll
            for (int j = 0; j < N; ++j) p[u].v[j] = from_f32<T>(to_f32(p[u].v[j]) * scale);
            if (wide) {
                reinterpret_cast<uint4 *>(out + s.head)[i + u * CT] = p[u].raw;
            } else {
#pragma unroll
                for (int j = 0; j < N; ++j) out[s.head + (i + u * CT) * N + j] = p[u].v[j];
            }
        }
    }
    if (c == 0) {
        if (threadIdx.x < s.head) out[threadIdx.x] = from_f32<T>(to_f32(in[threadIdx.x]) * scale);
        else if (threadIdx.x >= 32 && threadIdx.x - 32 < s.tail) {
            const int64_t i = t.n - s.tail + threadIdx.x - 32;
            out[i] = from_f32<T>(to_f32(in[i]) * scale);
        }
    }
}

template <int N>
__global__ void __launch_bounds__(CT)
clip_scale_kernel(const __grid_constant__ ClipTable<N> T, const double *part, int parts, double max_norm, float *norm_out) {
    __shared__ double s_red[CT / 32];
    pdl_enter();
    double acc = 0.0;
    for (int i = threadIdx.x; i < parts; i += CT) acc += part[i];
    const double norm = sqrt(sum_block(acc, s_red));
    if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
    float scale = 1.0f;
    if (!isinf(max_norm)) {
        const double s = max_norm / (norm + CLIP_EPS);
        if (!(s >= 1.0)) scale = (float)s;           // a NaN norm makes the scale NaN
    }
    const ClipShare share(T.chunks);
    if (share.from >= share.to) return;
    int at = clip_find(T, share.to - 1);
    for (uint32_t c = share.to; c-- > share.from;) {
        while (T.t[at].first > c) --at;
        const ClipTensor &t = T.t[at];
        if (scale == 1.0f && t.in == t.out) continue;   // in place, nothing changes
        const uint32_t lc = c - t.first;
        if (t.type == LAPSUM_TYPE_F32) scale_chunk<float>(t, lc, scale);
        else if (t.type == LAPSUM_TYPE_F16) scale_chunk<__half>(t, lc, scale);
        else scale_chunk<__nv_bfloat16>(t, lc, scale);
    }
}

int64_t clip_groups(int64_t count) { return (count + CLIP_GROUP - 1) / CLIP_GROUP; }

// No output overlaps another tensor, except its own input where they are equal.
bool clip_disjoint(int64_t count, const void *const *in, const int64_t *n, const int32_t *type, void *const *out,
                   const float *norm) {
    struct Item {
        uintptr_t a, b;
        bool written;
    };
    std::vector<Item> v;
    v.reserve((size_t)(2 * count + 1));
    v.push_back({reinterpret_cast<uintptr_t>(norm), reinterpret_cast<uintptr_t>(norm) + 4, true});
    for (int64_t i = 0; i < count; ++i) {
        if (n[i] == 0) continue;
        const uintptr_t bytes = (uintptr_t)n[i] * clip_size(type[i]);
        const uintptr_t a = reinterpret_cast<uintptr_t>(in[i]), o = reinterpret_cast<uintptr_t>(out[i]);
        if (a != o) v.push_back({a, a + bytes, false});
        v.push_back({o, o + bytes, true});
    }
    auto before = [](const Item &x, const Item &y) { return x.a < y.a; };
    if (!std::is_sorted(v.begin(), v.end(), before)) std::sort(v.begin(), v.end(), before);
    uintptr_t any = 0, written = 0;
    for (const Item &x : v) {
        if ((x.written ? any : written) > x.a) return false;
        any = std::max(any, x.b);
        if (x.written) written = std::max(written, x.b);
    }
    return true;
}

template <int N>
uint32_t fill_table(ClipTable<N> &T, int64_t a, int64_t b, const void *const *in, const int64_t *n, const int32_t *type,
                    void *const *out) {
    T.count = 0;
    T.chunks = 0;
    for (int64_t i = a; i < b; ++i) {
        if (n[i] == 0) continue;
        const ClipSpan s = clip_span(in[i], n[i], clip_size(type[i]));
        const int64_t c = std::max<int64_t>(1, (s.vecs + CLIP_VECS - 1) / CLIP_VECS);
        T.t[T.count++] = ClipTensor{in[i], out[i], n[i], T.chunks, type[i]};
        T.chunks += (uint32_t)c;
    }
    return T.chunks;
}

template <int N>
int run_clip(int64_t count, const void *const *in, const int64_t *n, const int32_t *type, double max_norm,
             void *const *out, float *norm, double *part, cudaStream_t st) {
    std::vector<ClipTable<N>> tables((size_t)((count + N - 1) / N));
    int parts = 0;
    for (size_t g = 0; g < tables.size(); ++g) {
        const int64_t a = (int64_t)g * N, b = std::min<int64_t>(a + N, count);
        const uint32_t chunks = fill_table(tables[g], a, b, in, n, type, out);
        if (!chunks) continue;
        const unsigned grid = std::min<uint32_t>(chunks, CLIP_BLOCKS);
        Launch L("clip_norm", st);
        LAPSUM_TRY(launch_k(clip_norm_kernel<N>, grid, CT, 0, st, tables[g], part + parts));
        parts += (int)grid;
    }
    for (size_t g = 0; g < tables.size(); ++g) {
        const unsigned grid = std::min<uint32_t>(std::max<uint32_t>(tables[g].chunks, 1), CLIP_BLOCKS);
        Launch L("clip_scale", st);
        LAPSUM_TRY(launch_k(clip_scale_kernel<N>, grid, CT, 0, st, tables[g], part, parts, max_norm, g ? nullptr : norm));
    }
    return LAPSUM_OK;
}

}  // namespace
}  // namespace lapsum

using namespace lapsum;

extern "C" {

int64_t lapsum_clip_scratch(int64_t count) {
    if (count < 1 || count > (int64_t(1) << 20)) return LAPSUM_ERR_ARG;
    return clip_groups(count) * CLIP_BLOCKS * (int64_t)sizeof(double);
}

int lapsum_clip_grads(int64_t count, const void *const *grads, const int64_t *sizes, const int32_t *types,
                      double max_norm, void *const *outs, float *norm_out, void *scratch, int64_t scratch_bytes,
                      struct CUstream_st *stream_in) try {
    const int64_t need = lapsum_clip_scratch(count);
    if (need < 0 || !grads || !sizes || !types || !outs || !norm_out || !(max_norm >= 0.0)) return LAPSUM_ERR_ARG;
    if (!scratch || (reinterpret_cast<uintptr_t>(scratch) & 15) || scratch_bytes < need) return LAPSUM_ERR_ARG;
    if (reinterpret_cast<uintptr_t>(norm_out) & 3) return LAPSUM_ERR_ARG;
    int64_t total = 0;
    for (int64_t i = 0; i < count; ++i) {
        if (types[i] != LAPSUM_TYPE_F32 && types[i] != LAPSUM_TYPE_F16 && types[i] != LAPSUM_TYPE_BF16) return LAPSUM_ERR_ARG;
        if (sizes[i] < 0 || sizes[i] >= (int64_t(1) << 40)) return LAPSUM_ERR_ARG;
        if (sizes[i] == 0) continue;
        const uintptr_t u = reinterpret_cast<uintptr_t>(grads[i]) | reinterpret_cast<uintptr_t>(outs[i]);
        if (!grads[i] || !outs[i] || (u & (uintptr_t)(clip_size(types[i]) - 1))) return LAPSUM_ERR_ARG;
        total += sizes[i];
        if (total >= (int64_t(1) << 42)) return LAPSUM_ERR_ARG;
    }
    if (!clip_disjoint(count, grads, sizes, types, outs, norm_out)) return LAPSUM_ERR_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream_in);
    double *part = static_cast<double *>(scratch);
    // a short list travels in a short parameter block: the launch copies it
    if (count <= CLIP_SMALL) return run_clip<CLIP_SMALL>(count, grads, sizes, types, max_norm, outs, norm_out, part, st);
    return run_clip<CLIP_GROUP>(count, grads, sizes, types, max_norm, outs, norm_out, part, st);
} catch (...) {   // host memory for the tables: no exception leaves a C entry
    return LAPSUM_ERR_ALLOC;
}

}  // extern "C"
