// launch_evict (csrc/evict.cu) with launches that are only written down and may be refused, for tests without a GPU.

#include <cuda_runtime.h>

#include "cache_plan.h"

namespace {

int g_refused = -1, g_launches = 0;   // number of the launch that is refused; launches so far

}  // namespace

extern "C" {

cudaError_t CUDARTAPI cudaLaunchKernelExC(const cudaLaunchConfig_t*, const void*, void**) {
    return g_launches++ == g_refused ? cudaErrorLaunchOutOfResources : cudaSuccess;
}

// The launches that an eviction of 100 rows of two heads to 40 makes.
int evict_host_launches(int refused) {
    g_refused = refused;
    g_launches = 0;
    fq::EvictArgs a = {};
    a.n_seq = 1;
    a.Hkv = 2;
    a.s[0].len = 100;
    a.s[0].n = 40;
    fq::launch_evict(a, 100, 4, nullptr);
    return g_launches;
}

}  // extern "C"
