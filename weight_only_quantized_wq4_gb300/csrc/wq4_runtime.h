// What the entry points outside wq4_api.cu share with it: the device's properties and status word,
// the process-wide options that apply to every kernel, and a launch with the library's attributes.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "wq4.h"

namespace wq4 {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

constexpr int kMaxDevices = 64;

struct Runtime {
    int device;                 // the current device's ordinal, below kMaxDevices
    int sm_count;
    unsigned int* status;       // device status word
    long long timeout_cycles;   // bound of every pipeline wait
    int test_stall;             // (tests) one wait per CTA that nothing ends
    bool pdl;                   // programmatic dependent launch
    bool trace;
    EncodeTiledFn encode;       // cuTensorMapEncodeTiled
};

// The current device's runtime under the current options (WQ4_ERR_CUDA without a device).
int runtime(Runtime* out);

// A positive number that belongs to a device (a kernel's attributes once they are set, its occupancy), found out by the first
// call there. Threads may find it out twice; they find the same. What is not positive, a failure, is not kept.
class PerDevice {
public:
    template <typename F>
    int get(int device, F find) {
        int n = v_[device].load(std::memory_order_acquire);
        if (n == 0 && (n = find()) > 0) v_[device].store(n, std::memory_order_release);
        return n;
    }

private:
    std::atomic<int> v_[kMaxDevices] = {};
};

inline bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Launches `kern` on `st`, in clusters of `cluster` CTAs, with programmatic dependent launch when
// the options ask for it: every kernel launched so waits (griddepcontrol.wait) before it touches
// global memory, and reads it by ordinary loads and copies: a read-only load (ld.global.nc) is for data that
// nothing writes while the kernel is there, and it is there while the kernels ahead may still write.
template <typename... P, typename... A>
int launch(const Runtime& rt, void (*kern)(P...), dim3 grid, int threads, int smem, int cluster, wq4_stream_t st,
           A&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (rt.pdl) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = cluster;
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    if (cudaLaunchKernelEx(&cfg, kern, P(args)...) != cudaSuccess) {
        cudaGetLastError();   // reported here, not by a later call
        return WQ4_ERR_CUDA;
    }
    return WQ4_OK;
}

}  // namespace wq4
