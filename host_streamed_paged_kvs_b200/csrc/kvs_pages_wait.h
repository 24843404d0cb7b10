// kvs_pages_wait.h -- when a wait inside the page attention kernels gives up.
// Plain C++ too, so that the rule can be tested on the host.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define KVS_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define KVS_HOST_DEVICE inline
#endif

namespace kvs {

// Time without completion after which a wait gives up.  While other warps of the
// block recompute rows from their definition (`busy`) the time does not run:
// that work is long (seconds for millions of keys and an infinity among the
// values that every row sees) but ends, and it waits for nothing itself.
constexpr uint64_t kPagesWaitNs = 10000000000ull;
struct WaitClock {
    uint64_t since = 0;  // 0: not looked yet
    KVS_HOST_DEVICE bool expired(uint64_t now_ns, bool busy) {
        if (since == 0 || busy) since = now_ns;
        return now_ns - since > kPagesWaitNs;
    }
};

}  // namespace kvs
