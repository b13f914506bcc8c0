// host.cuh -- argument checks and launch helpers shared by the entry points
// of the embedding, log-probability and gated-delta-rule operators.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/liblstm.h"
#include "common.cuh"

namespace lstm {

// First kernel of a call: clear the workspace's control block (the status
// word reports the call that this kernel begins).
__device__ __forceinline__ void clear_ctrl(Ctrl *ctrl) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < sizeof(Ctrl) / 4)
        reinterpret_cast<unsigned int *>(ctrl)[threadIdx.x] = 0u;
}

namespace host {

#define LSTM_CUDA_TRY(expr)                               \
    do {                                                  \
        cudaError_t e_ = (expr);                          \
        if (e_ != cudaSuccess) return LSTM_ERR_CUDA;      \
    } while (0)

// A pointer argument: aligned (to 16 bytes, or to its elements where the
// kernels read them one by one), and not NULL where it is needed.
inline bool ptr_ok(const void *p, bool needed, size_t align = 16) {
    return (p != nullptr || !needed) && ((uintptr_t)p & (align - 1)) == 0;
}

inline bool dtype_ok(int dtype) {
    return dtype == LSTM_F32 || dtype == LSTM_BF16 || dtype == LSTM_F16;
}

inline size_t elem_bytes(int dtype) { return dtype == LSTM_F32 ? 4 : 2; }

inline int ws_check(const void *ws, size_t ws_bytes, size_t need) {
    return (!ws || ws_bytes < need || ((uintptr_t)ws & 255u) != 0) ? LSTM_ERR_WORKSPACE : LSTM_OK;
}

// SMs of the current device (a B200's 148 where there is no device to ask).
inline int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
        (void)cudaGetLastError();
        n = 148;
    }
    return n;
}

// After a <<<>>> launch: count it, return its launch error.
inline cudaError_t launched() {
    note_launch();
    return cudaGetLastError();
}

}  // namespace host
}  // namespace lstm
