// tma.cu -- the tensor maps of the paged-cache kernels.
#include "tma.cuh"

namespace tsa {

static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> g_page_encode{nullptr};

cudaError_t page_map(CUtensorMap* map, const Pages& c, void* base, int rows) {
    PFN_cuTensorMapEncodeTiled_v12000 encode = g_page_encode.load(std::memory_order_acquire);
    if (!encode) {
        cudaDriverEntryPointQueryResult q;
        void* fn = nullptr;
        const cudaError_t e = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q);
        if (e != cudaSuccess) return e;
        if (q != cudaDriverEntryPointSuccess || fn == nullptr) return cudaErrorNotSupported;
        encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
        g_page_encode.store(encode, std::memory_order_release);
    }
    const cuuint64_t dims[4] = {(cuuint64_t)kDHead, (cuuint64_t)c.page_size, (cuuint64_t)c.Hkv, (cuuint64_t)c.num_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)c.row_stride * 2, (cuuint64_t)c.head_stride * 2, (cuuint64_t)c.page_stride * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1};
    const cuuint32_t step[4] = {1, 1, 1, 1};
    const CUresult r = encode(map, c.half ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base,
                              dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace tsa
