// tfa_internal.h -- what the library's translation units share on the host:
// error reporting (tfa_last_error) and the per-device state of tfa.cu.
#pragma once

#include <cuda_runtime.h>

namespace tfa {

constexpr int kMaxDevices = 64;  // device_info refuses others

// Record which CUDA call failed (readable through tfa_last_error); TFA_ERR_CUDA.
int report_cuda(const char *what, cudaError_t e);

// The current device's status word and SM count, created on first use like any
// call's (TFA_ERR_CAPTURE if that would happen inside a graph capture).
int device_info(cudaStream_t stream, unsigned **status, int *sm_count);

}  // namespace tfa
