// Host-side helpers that the library's translation units share; defined in
// pa_api.cu.
#pragma once

#include <cuda_runtime.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "pa.h"

// Records the text pa_last_error() returns.
void pa_internal_set_last_error(const char *msg);

// Counts one kernel launch of this thread (pa_launch_count).
void pa_internal_count_launch();

// The current device's index and number of SMs.
pa_status pa_internal_device(int *dev, int *sms);

// The driver's cuTensorMapEncodeTiled (a PFN_cuTensorMapEncodeTiled).
pa_status pa_internal_tensor_map_encoder(void **fn);

// Device address of the current device's error word. Looked up on every call
// (host side once the module is loaded), so it survives a device reset.
pa_status pa_internal_error_word(unsigned int **word);

namespace pa_host {

inline pa_status fail(pa_status st, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    pa_internal_set_last_error(buf);
    return st;
}

inline pa_status cuda_fail(cudaError_t e, const char *what) {
    return fail(PA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline bool block_size_supported(int bs) { return bs == 16 || bs == 32 || bs == 64; }

}  // namespace pa_host
