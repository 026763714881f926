// kv_attention_q4 for few rows: heads of up to 128 elements.
#include "kv_attention_q4_few.cuh"

namespace pkv {

int run_q4_few128(bool bf16, const Q4Params &q, int rows, const DeviceInfo &dev, cudaStream_t s)
{
    FewParams p = {};
    static_cast<Q4Params &>(p) = q;
    p.bf16 = bf16;
    return rows <= 8 ? launch_few<128, 1>(p, &dev, s) : launch_few<128, 2>(p, &dev, s);
}

int preload_q4_few128_kernels()
{
    FewParams p = {};
    const int st = launch_few<128, 1>(p, nullptr, nullptr);
    return st != KV_OK ? st : launch_few<128, 2>(p, nullptr, nullptr);
}

}  // namespace pkv
