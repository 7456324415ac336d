// route_common.cuh -- building blocks of the routing and clipping kernels.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "lapsum_device.cuh"
#include "select_keys.cuh"

namespace lapsum {

__device__ __forceinline__ unsigned lanes_below(int lane) { return (1u << lane) - 1u; }

// Sum of one value per thread over the CTA, the same in every thread; one
// barrier a call (two buffers in turn: a buffer is written again only after the
// barrier of the call between).
template <int NW>
struct BlockAdd {
    unsigned *buf;   // 2 * NW words of shared memory
    int flip = 0;
    __device__ explicit BlockAdd(unsigned *b) : buf(b) {}
    __device__ __forceinline__ unsigned operator()(unsigned v) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        unsigned *s = buf + flip * NW;
        flip ^= 1;
        v = __reduce_add_sync(FULL, v);
        if (lane == 0) s[warp] = v;
        __syncthreads();
        return __reduce_add_sync(FULL, lane < NW ? s[lane] : 0u);
    }
};

__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// ------------------------------------------------------- typed vectors --
// VB bytes moved by one load or store, and their values in fp32.
template <int VB> struct VecOf;
template <> struct VecOf<16> { using type = uint4; };
template <> struct VecOf<8> { using type = uint2; };
template <> struct VecOf<4> { using type = uint32_t; };
template <> struct VecOf<2> { using type = uint16_t; };

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <typename T, int VB>
union Pack {
    typename VecOf<VB>::type raw;
    T v[VB / sizeof(T)];
    __device__ __forceinline__ Pack() {}
};

}  // namespace lapsum
