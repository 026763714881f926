// What the two kernels of kv_attention_q4 share.
#pragma once

#include "kv_attention.cuh"
#include "kv_q4.cuh"

namespace pkv {

// A plane of 4-bit rows.
struct Q4Plane {
    uint64_t base;
    const kv_cache_desc *desc;  // host
    int32_t dim;
};

struct Q4Params {
    Batch b;
    Q4Plane k, v;
    const int32_t *table;
    int64_t table_stride;
    int32_t num_blocks;  // pages that both planes have
    int32_t no_page;     // a page that neither has: its loads bring zeros
    FastDiv block;       // slots of a page
    const char *q;
    int64_t q_token, q_head;
    int32_t heads_all;   // key heads of a row
    Output o;            // o.scale: of the products, with the keys' tensor scale
    float v_scale;
    float *ws;
    int *counters;
};

// Bytes that the barrier's phase waits for, without an arrival.
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// An untiled copy: addresses and size multiples of 16.
__device__ __forceinline__ void bulk_load(uint32_t dst, uint64_t src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// Units of `rows` rows, 8 or 16, of heads of at most 64 and of 128 elements (kv_attention_q4_few64.cu, kv_attention_q4_few128.cu).
int run_q4_few64(bool bf16, const Q4Params &p, int rows, const DeviceInfo &dev, cudaStream_t s);
int run_q4_few128(bool bf16, const Q4Params &p, int rows, const DeviceInfo &dev, cudaStream_t s);
int preload_q4_few64_kernels();
int preload_q4_few128_kernels();
// Units of whole tokens of up to 256 rows, key tiles of 2^q4_tile_shift() (kv_attention_q4_many.cu).
int q4_unit_rows(int group);
int q4_tile_shift();
int run_q4_many(bool bf16, const Q4Params &p, const kv_attn_batch *batch, const DeviceInfo &dev, cudaStream_t s);
int preload_q4_many_kernels();
int preload_q4_kernels();      // kv_attention_q4.cu

}  // namespace pkv
