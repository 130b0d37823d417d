// Per-device launch preparation and the tensor-map encoder, shared by every
// translation unit that launches kernels.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace fftconv {

// A value per device: kernel attribute opt-ins belong to the context of the
// device that is current when they are made, so launch preparations are kept
// per device ordinal (0: not prepared on that device yet).
constexpr int kDevSlots = 64;
struct PerDevice {
    int v[kDevSlots] = {};
    int* slot() {
        int d = 0;
        if (cudaGetDevice(&d) != cudaSuccess || d < 0 || d >= kDevSlots) return nullptr;
        return &v[d];
    }
};

// cuTensorMapEncodeTiled, reached through the runtime (once per process;
// null if the driver does not provide it).
using TensorMapEncoder = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                      const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                      CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline TensorMapEncoder tensor_map_encoder() {
    static TensorMapEncoder fn = [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            return TensorMapEncoder(nullptr);
        }
        return reinterpret_cast<TensorMapEncoder>(ptr);
    }();
    return fn;
}

}  // namespace fftconv
