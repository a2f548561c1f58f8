// How long a block waits for its own copies and products before it ends, apart from what it polls, so that the loop
// also compiles for the host.
#pragma once

#ifdef __CUDACC__
#define GS_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define GS_HOST_DEVICE inline
#endif

namespace gs {

constexpr unsigned kDrainLimit = 1u << 22;

// Polls done() until it is true, kDrainLimit times at most; whether it was. Nothing shortens it: neither the caller's spin
// limit nor a wait elsewhere that gave up. A block drains mostly after a wait that did, and one that ended sooner would
// leave copies running into the shared memory, or products into the tensor memory, of the block that follows it.
template <class Done>
GS_HOST_DEVICE bool poll_drain(Done done) {
    for (unsigned i = 0; i < kDrainLimit; ++i)
        if (done()) return true;
    return false;
}

}  // namespace gs
