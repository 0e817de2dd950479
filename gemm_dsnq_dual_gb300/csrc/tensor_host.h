// Host helpers of the tensor-core kernels: the driver's tensor-map encoder and
// the shared-memory attribute of a kernel.
#pragma once

#include <mutex>
#include <tuple>
#include <vector>

#include <cuda.h>
#include <cuda_runtime.h>

#include "dsnq_internal.h"

namespace dsnq {

constexpr uint64_t kDefaultTimeoutNs = 2000000000ull;   // bound of every device wait

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// cudaFuncSetAttribute once per (kernel, device, size): it is host work on
// every call otherwise.
inline bool set_smem_attr(const void* kern, size_t smem) {
    static std::mutex mu;
    static std::vector<std::tuple<const void*, int, size_t>> done;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    try {
        std::lock_guard<std::mutex> lock(mu);
        for (const auto& d : done)
            if (std::get<0>(d) == kern && std::get<1>(d) == dev && std::get<2>(d) >= smem) return true;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) !=
            cudaSuccess) {
            cudaGetLastError();
            return false;
        }
        done.emplace_back(kern, dev, smem);
        return true;
    } catch (...) {                                        // no exception leaves a C entry point
        return false;
    }
}

}  // namespace dsnq
