// give_up.cuh -- what a ring's reader sees of its wait; the checked build can have it
// say that a wait gave up which did not, so that what follows can be tested: the copy
// has landed all the same, and every wait behind it is bounded.
#pragma once
#include <climits>

#include "lapsum_device.cuh"

namespace lapsum {

// Polls of a ring's wait before it gives up: seconds (a poll that finds nothing takes about
// 1.5 us), 0.1 s in the checked build, whose tests let waits run out.
#ifdef LAPSUM_CHECKED
constexpr int RING_WAIT_CAP = 1 << 16;
#else
constexpr int RING_WAIT_CAP = BULK_WAIT_CAP;
#endif

enum GiveUp { GIVE_UP_READ = 0, GIVE_UP_WRITE = 1, GIVE_UP_AGAIN = 2, GIVE_UP_KINDS = 3 };   // LAPSUM_GIVE_UP_*

#ifdef LAPSUM_CHECKED
static __device__ int g_give_up_from[GIVE_UP_KINDS] = {INT_MAX, INT_MAX, INT_MAX};   // a block's row from which on its waits give up
__device__ __forceinline__ bool waited(bool ok, GiveUp kind, int turn) { return ok && turn < g_give_up_from[kind]; }
static inline cudaError_t set_give_up(GiveUp kind, int turn) {
    return cudaMemcpyToSymbol(g_give_up_from, &turn, sizeof(int), sizeof(int) * kind);
}
#else
__device__ __forceinline__ bool waited(bool ok, GiveUp, int) { return ok; }
static inline cudaError_t set_give_up(GiveUp, int) { return cudaErrorNotSupported; }
#endif

}  // namespace lapsum
