// Host side of the tensor-core kernels: tensor maps of paged caches.
#include <mutex>

#include "kv_tensor.cuh"

namespace pkv {

namespace {

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                              const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder, looked up once (the library links the runtime alone).
EncodeFn encoder()
{
    static std::mutex mu;
    static EncodeFn fn = nullptr;
    std::lock_guard<std::mutex> lock(mu);
    if (fn == nullptr) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cuda_status(cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found)) == KV_OK &&
            found == cudaDriverEntryPointSuccess)
            fn = (EncodeFn)p;
    }
    return fn;
}

}  // namespace

int make_map(CUtensorMap *map, uint64_t base, int rank, const uint64_t *dims, const uint64_t *strides, const uint32_t *box)
{
    const EncodeFn fn = encoder();
    if (fn == nullptr) return KV_ERR_CUDA;
    cuuint64_t d[5], st[4];
    cuuint32_t b[5], one[5];
    for (int i = 0; i < rank; i++) {
        d[i] = dims[i];
        b[i] = box[i];
        one[i] = 1;
        if (i) st[i - 1] = strides[i - 1];
    }
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, (cuuint32_t)rank, (void *)base, d, st, b, one,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? KV_OK : KV_ERR_UNSUPPORTED;
}

int make_cache_map(CUtensorMap *map, const kv_cache_desc *c, int tensor, int plane, int heads, int head_dim, int rows)
{
    const uint64_t dims[4] = {(uint64_t)head_dim, (uint64_t)heads, (uint64_t)c->block_size, (uint64_t)c->num_blocks};
    const uint64_t strides[3] = {(uint64_t)head_dim * 2, (uint64_t)c->token_stride, (uint64_t)c->block_stride};
    const uint32_t box[4] = {64, 1, (uint32_t)rows, 1};
    return make_map(map, c->base[tensor] + (plane ? (uint64_t)c->plane_stride : 0), 4, dims, strides, box);
}

}  // namespace pkv
