// q4_wait.cuh -- a bounded wait that a whole warp makes as one.  No CUDA
// header is needed: the tests compile it for the host, lanes being threads.
#pragma once

#ifdef __CUDACC__
#define Q4_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define Q4_HOST_DEVICE inline
#endif

namespace q4 {

// True once `ready`, false once `expired`, both votes of the warp: whether the
// phase is complete for every lane, and whether the wait is over for any.  One
// lane may see an error flag or the time limit while another sees the phase
// complete, and what follows a wait are instructions of the whole warp
// (elect.sync, tcgen05.ld, __syncwarp), so lanes must not part here.
template <typename Ready, typename Expired>
Q4_HOST_DEVICE bool wait_together(Ready ready, Expired expired) {
    while (true) {
        for (int i = 0; i < 64; ++i)
            if (ready()) return true;
        if (expired()) return false;
    }
}

}  // namespace q4
