// smla_host.cuh -- host helpers of the C ABI: the device check, argument alignment and the TMA
// descriptor of Q.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <mutex>

#include "../../include/smla.h"

namespace smla {
namespace host {

constexpr int kMaxDevices = 64;

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// SMLA_OK and the current device's SM count, SMLA_ERR_DEVICE if it is not sm_100.  The answer
// is kept per device.
inline int current_device(int &dev, int &sms) {
    static std::mutex mutex;
    static int known[kMaxDevices] = {};  // 0 unknown, -1 other, else the SM count of an sm_100
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return SMLA_ERR_CUDA;
    std::lock_guard<std::mutex> lock(mutex);
    if (known[dev] == 0) {
        int major = 0, minor = 0, n = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return SMLA_ERR_CUDA;
        known[dev] = (major == 10 && minor == 0) ? n : -1;
    }
    sms = known[dev];
    return sms > 0 ? SMLA_OK : SMLA_ERR_DEVICE;
}

// cuTensorMapEncodeTiled from the driver, looked up once through the runtime.
inline int tensor_map_encoder(PFN_cuTensorMapEncodeTiled_v12000 &fn) {
    static std::mutex mutex;
    static PFN_cuTensorMapEncodeTiled_v12000 encode_tiled = nullptr;
    std::lock_guard<std::mutex> lock(mutex);
    if (encode_tiled == nullptr) {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess || f == nullptr)
            return SMLA_ERR_CUDA;
        encode_tiled = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }
    fn = encode_tiled;
    return SMLA_OK;
}

// Q [B*64 rows, 512 bf16] as a 2-D tensor; a box of 64 dims x 64 heads with the
// 128-byte swizzle lands as one K-block of the shared-memory Q operand.
inline int encode_q_map(CUtensorMap *map, const void *q, int B) {
    PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    const int rc = tensor_map_encoder(fn);
    if (rc != SMLA_OK) return rc;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(SMLA_DIM), static_cast<cuuint64_t>(B) * SMLA_HEADS};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(SMLA_DIM) * 2};
    cuuint32_t box[2] = {64, 64};
    cuuint32_t estr[2] = {1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(q), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? SMLA_OK : SMLA_ERR_INVALID;
}

// Launches a kernel that may be scheduled while the one before it in the stream drains, or still runs if that
// one allows it.  Every block of it has to call wait_for_prior_kernel(), before it touches memory
// that an earlier kernel writes or reads.
template <class Kernel, class... Args>
cudaError_t launch_after(Kernel kernel, dim3 grid, unsigned threads, size_t smem, cudaStream_t stream, const Args &...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace host
}  // namespace smla
