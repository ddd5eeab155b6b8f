// Host-side helpers that the files of the C ABI share: pointer checks, the current
// device, the tensor map encoder, NVTX ranges.  Internal; not installed.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>
#include <stdint.h>

#include <mutex>

#include "../../include/moe.h"

namespace moe {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct DevInfo {
    int sm_count = 0;
    int major = 0;
};

inline DevInfo dev_info() {
    static std::mutex mu;
    static DevInfo cache[64];
    static bool have[64] = {};
    int dev = 0;
    DevInfo info;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return info;
    std::lock_guard<std::mutex> g(mu);
    if (dev < 64 && have[dev]) return cache[dev];
    cudaDeviceGetAttribute(&info.sm_count, cudaDevAttrMultiProcessorCount, dev);
    cudaDeviceGetAttribute(&info.major, cudaDevAttrComputeCapabilityMajor, dev);
    if (dev < 64) {
        cache[dev] = info;
        have[dev] = true;
    }
    return info;
}

inline moe_status check_device(DevInfo* out) {
    DevInfo i = dev_info();
    if (i.major != 10 || i.sm_count <= 0) return MOE_ERR_UNSUPPORTED;
    *out = i;
    return MOE_OK;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

inline moe_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// NVTX ranges around the host-side enqueue of each stage (names "moe.<stage>"),
// nested in one range per entry point: a profiler's timeline groups the kernels
// by stage, and ncu can select them with --nvtx-include.  Header-only NVTX: with
// no tool attached each push/pop is a call through a null stub.
struct NvtxRange {
    explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange&) = delete;
    NvtxRange& operator=(const NvtxRange&) = delete;
};

}  // namespace moe
