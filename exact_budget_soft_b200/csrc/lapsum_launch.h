// lapsum_launch.h -- what every entry point shares on the host: the launch
// record, and the mapping of CUDA errors to return codes (internal).
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/lapsum.h"

namespace lapsum {

// RAII: counts one kernel launch, names it for tracing tools (an NVTX range
// around the host-side launch, named after the step: free when no tool is
// attached) and, when profiling, brackets it with events.
struct Launch {
    const char *name;
    cudaStream_t st;
    cudaEvent_t e0 = nullptr;
    Launch(const char *nm, cudaStream_t s);
    ~Launch();
    Launch(const Launch &) = delete;
    Launch &operator=(const Launch &) = delete;
};

inline int map_err(cudaError_t e) {
    if (e == cudaSuccess) return LAPSUM_OK;
    if (e == cudaErrorMemoryAllocation) return LAPSUM_ERR_ALLOC;
    return LAPSUM_ERR_CUDA;
}

// Addresses that are multiples of `to`, a power of two (null is one).
template <typename... P>
inline bool multiples_of(uintptr_t to, P... p) {
    return ((reinterpret_cast<uintptr_t>(p) | ...) & (to - 1)) == 0;
}

// checked build: waits of a kind (GiveUp) report that they gave up from a block's row `turn` on
cudaError_t select_give_up(int kind, int turn);   // k_select.cu
cudaError_t tokens_give_up(int kind, int turn);   // k_tokens.cu

#define LAPSUM_TRY(expr)                                    \
    do {                                                    \
        cudaError_t _e = (expr);                            \
        if (_e != cudaSuccess) return lapsum::map_err(_e);  \
    } while (0)

}  // namespace lapsum
