// Error reporting shared by the host files of the C ABI.
#pragma once

#include <cuda_runtime.h>

#include "fq.h"

namespace fq {

// Set the thread's fq_last_error message and return s.
fq_status fail(fq_status s, const char* fmt, ...);

}  // namespace fq

#define CK(call)                                                                                       \
    do {                                                                                               \
        cudaError_t e_ = (call);                                                                       \
        if (e_ != cudaSuccess)                                                                         \
            return fail(e_ == cudaErrorMemoryAllocation ? FQ_ERR_OUT_OF_MEMORY : FQ_ERR_CUDA, "%s: %s", \
                        #call, cudaGetErrorString(e_));                                                \
    } while (0)

#define TRY(call)                  \
    do {                           \
        fq_status s_ = (call);     \
        if (s_ != FQ_OK) return s_; \
    } while (0)
