// TMA tensor maps for the latent-attention kernels.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "sm100_pipe.cuh"

namespace rda {

bool make_map_3d(CUtensorMap *map, const void *base, uint64_t d0, uint64_t d1, uint64_t d2, uint64_t stride1,
                 uint64_t stride2, uint32_t box1, uint32_t box2) {
    static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p) : nullptr;
    }();
    const cuuint64_t dims[3] = {d0, d1, d2}, strides[2] = {stride1 * 2, stride2 * 2};
    const cuuint32_t box[3] = {64, box1, box2}, step[3] = {1, 1, 1};
    return encode && encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
                            step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_map_heads(CUtensorMap *map, const void *base, int D, int H, long rows, uint32_t box, const void *any) {
    return make_map_3d(map, rows ? base : any, D, H, rows ? rows : 1, D, (uint64_t)H * D, 1, box);
}

}  // namespace rda
