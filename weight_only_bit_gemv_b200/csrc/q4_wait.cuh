// q4_wait.cuh -- a bounded wait that a whole warp makes as one.  No CUDA
// header is needed: the tests compile it for the host, lanes being threads.
#pragma once

#ifdef __CUDACC__
#define Q4_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define Q4_HOST_DEVICE inline
#endif

namespace q4 {

// True once `ready` is true in every lane, false once `expired` is in any: the
// same in all lanes.  One lane may see an error flag or the time limit while
// another sees the phase complete, and what follows a wait are instructions of
// the whole warp (elect.sync, tcgen05.ld, __syncwarp), so lanes must not part
// here.  all(b): whether b is true in every lane, a vote of the warp.
template <typename Ready, typename Expired, typename All>
Q4_HOST_DEVICE bool wait_together(Ready ready, Expired expired, All all) {
    while (true) {
        for (int i = 0; i < 64; ++i)
            if (all(ready())) return true;
        if (!all(!expired())) return false;
    }
}

}  // namespace q4
