// tfa_internal.h -- what the library's translation units share on the host:
// error reporting (tfa_last_error) and the per-device state of tfa.cu.
#pragma once

#include <cuda_runtime.h>

namespace tfa {

constexpr int kMaxDevices = 64;  // device_info refuses others
constexpr int kSms = 148;        // of a B200, for rules that choose between variants without a device

// Record which CUDA call failed (readable through tfa_last_error); TFA_ERR_CUDA.
int report_cuda(const char *what, cudaError_t e);

// The current device's status word and SM count, created on first use like any
// call's (TFA_ERR_CAPTURE if that would happen inside a graph capture).
int device_info(cudaStream_t stream, unsigned **status, int *sm_count);

// Launches a kernel that may be set up while the stream's previous one still ends: it
// calls grid_dep_wait before it touches memory, and grid_dep_launch only then, so that
// a kernel after it never starts before the one before it has ended.  Inputs are not
// read through the read-only path (load_input).  (kv4::join_kernel reads the lengths
// before its wait: the kernel before it, its own call's, neither writes them nor
// launches it before its own wait.)
template <typename... Args, typename... Given>
cudaError_t launch_after(void (*kernel)(Args...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                         Given... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, Args(args)...);
}

}  // namespace tfa
