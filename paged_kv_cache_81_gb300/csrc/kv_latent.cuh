// What the two latent attention kernels share (kv_latent.cu, kv_latent_few.cu).
#pragma once

#include "kv_attention.cuh"

namespace pkv {

constexpr int kLatentDim = 576, kLatentRank = 512;  // of a row, and of its values

struct LatentParams {
    Batch b;
    const int32_t *table;
    int64_t table_stride;
    int32_t num_blocks;
    FastDiv block;
    int32_t piece_rows;
    int32_t q_rows;  // rows one TMA brings of q
    Output o;
    float *ws;
    int *counters;
};

// Panels (64 elements of each key) of one tile of Keys rows into their slot: a TMA per (run of slots inside a page, panel), spread over the
// lanes; column(h) is the first element of panel h.  The first page a lane needs is looked up before
// `ready` waits for the slot.
template <int Keys, int Panels, typename Column, typename Ready>
__device__ __forceinline__ bool load_latent_tile(const LatentParams &p, const Walk &w, int kb, uint32_t to, uint32_t bar, const CUtensorMap *map, const Column &column,
                                          const Ready &ready)
{
    const int lane = threadIdx.x & 31, pr = p.piece_rows;
    const int p0 = max(0, w.u.lo - kb) / pr, p1 = (min(w.u.hi - kb, Keys) + pr - 1) / pr;
    const int32_t *row = p.table + (int64_t)w.at.req * p.table_stride;
    int page = 0, slot = 0;
    const auto find = [&](int i) {
        const uint32_t key = (uint32_t)(kb + i * pr), col = fdiv(key, p.block);
        slot = (int)(key - col * p.block.d);
        page = __ldg(row + col);
        if (page < 0 || page >= p.num_blocks) {
            set_error(p.b.err, KV_DERR_TABLE);
            page = p.num_blocks;  // outside the map: reads zeros
        }
    };
    if (p0 + lane < p1) find(p0 + lane);
    if (!ready()) return false;
    if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)((p1 - p0) * pr) * Panels * 128);
    __syncwarp();
    for (int i = p0 + lane; i < p1; i += 32) {
        if (i >= p0 + 32) find(i);
#pragma unroll
        for (int h = 0; h < Panels; h++) tma_load_4d(to + h * Keys * 128 + i * pr * 128, map, bar, column(h), 0, slot, page);
    }
    __syncwarp();
    return true;
}

// Up to 64 rows a unit, tiles of 32 keys (kv_latent_few.cu).
constexpr int kLatentFewRows = 64, kLatentFewKeyShift = 5;
int run_latent_few(bool bf16, const CUtensorMap &map, const CUtensorMap &q_map, const LatentParams &p, int parts, cudaStream_t s);
int preload_latent_few_kernels();

}  // namespace pkv
