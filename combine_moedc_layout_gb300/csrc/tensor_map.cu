// The driver's encoder of tensor maps, looked up once.
#include "tensor_map.cuh"

#include <cudaTypedefs.h>

namespace moedc_host {

bool tensor_map(CUtensorMap* map, CUtensorMapDataType type, CUtensorMapSwizzle swizzle, const void* base, int dims,
                const cuuint64_t* size, const cuuint64_t* stride, const cuuint32_t* box)
{
    static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &found) != cudaSuccess || found != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    if (!encode) return false;
    const cuuint32_t elem[5] = {1, 1, 1, 1, 1};
    return encode(map, type, dims, const_cast<void*>(base), size, stride, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace moedc_host
