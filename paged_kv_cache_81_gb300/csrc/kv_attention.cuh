// What the attention kernels' host sides share: argument checks, the batch they pass on, the workspace.
#pragma once

#include <cmath>

#include "kv_plan.cuh"
#include "kv_tensor.cuh"

namespace pkv {

constexpr int64_t kPlaceBytes = 16384;  // where each CTA's piece begins: 16 bytes a CTA

// Two fragments a CTA: of 256 rows x (128 values + maximum + sum) for kv_attention, of 128 rows x (256
// values + maximum + sum) for each CTA of kv_latent_attention.
inline int64_t attention_workspace(int num_sms) { return kPlaceBytes + (int64_t)num_sms * 2 * 256 * (128 + 2) * 4; }

int check_batch(const kv_attn_batch *t);
int fill_batch(Batch *b, const kv_attn_batch *t, int heads, int kv_heads, int block_size, int unit_rows, int tile, int causal, int window);
int check_plane(const kv_cache_desc *c, int tensor, int plane, int heads, int dim);
int check_rows(const void *p, int64_t token_stride, int64_t head_stride);
// A map of q [tokens, heads, head_dim]; a load brings 64 elements of `group` heads of box_tokens tokens.
int make_q_map(CUtensorMap *map, const void *q, int64_t token_stride, int64_t head_stride, int head_dim, int heads, int64_t tokens, int group,
               int box_tokens);
// Slots that one TMA brings: the largest power of two that divides the block, at most a tile, so that a
// piece never leaves its page.
int piece_rows(int block_size, int tile);

// Joins the fragments of the units that were cut.  Every CTA writes at most two: slot 2x + 1 for one that
// begins its unit, 2x for one that does not; x = part * halves + half, where `halves` CTAs of a part
// hold DV values of a row each.
struct Join {
    Batch b;
    const Place *places;
    const float *ws;
    char *out;
    int64_t out_token, out_head;
    float *lse;
    int32_t heads, dv, rows, halves, parts;
    float scale, c;
};

// Block (c, y, half) looks whether the cut before part c + 1 is the first one inside its unit, and joins
// rows y, y + gridDim.y, ... of it.  A row's fragments are read in the order of their keys, so the
// result does not depend on timing.
template <int DV, bool Bf16>
__global__ void __launch_bounds__(256) join_kernel(const Join p)
{
    grid_dep_entry();
    const Batch &b = p.b;
    const int c = blockIdx.x + 1, half = blockIdx.z;
    const Place pl = p.places[c];
    if (pl.req < 0 || pl.off == 0) return;
    const Place before = p.places[c - 1];
    const auto same = [&](const Place &o) { return o.req == pl.req && o.head == pl.head && o.unit == pl.unit; };
    if (same(before) && before.off != 0) return;  // an earlier cut of the unit joins it
    int last = c;
    while (last + 1 < p.parts) {
        const Place nx = p.places[last + 1];
        if (!same(nx) || nx.off == 0) break;
        last++;
    }
    const Request q = load_request(b, pl.req);
    const Unit u = make_unit(b, q, pl.unit);
    const int64_t stride = (int64_t)p.rows * (DV + 2);
    const auto fragment = [&](int x) { return p.ws + (2 * (x * p.halves + half) + (x == c - 1)) * stride; };
    constexpr int kLanes = DV / 8, kRowsPerPass = 256 / kLanes;
    const int col = (threadIdx.x % kLanes) * 8;
    for (int row = blockIdx.y * kRowsPerPass + threadIdx.x / kLanes; row < u.rows; row += gridDim.y * kRowsPerPass) {
        float top = -INFINITY;
        for (int x = c - 1; x <= last; x++) top = fmaxf(top, fragment(x)[(int64_t)p.rows * DV + row]);
        float o[8] = {0, 0, 0, 0, 0, 0, 0, 0}, l = 0.0f;
        if (top > -INFINITY) {
#pragma unroll 4
            for (int x = c - 1; x <= last; x++) {
                const float *part = fragment(x);
                const float a = exp2_fast((part[(int64_t)p.rows * DV + row] - top) * p.c);
                l += part[(int64_t)p.rows * (DV + 1) + row] * a;
                const float4 v0 = *reinterpret_cast<const float4 *>(part + (int64_t)row * DV + col);
                const float4 v1 = *reinterpret_cast<const float4 *>(part + (int64_t)row * DV + col + 4);
                o[0] += v0.x * a, o[1] += v0.y * a, o[2] += v0.z * a, o[3] += v0.w * a;
                o[4] += v1.x * a, o[5] += v1.y * a, o[6] += v1.z * a, o[7] += v1.w * a;
            }
        }
        const int r = u.row0 + row, tok = (int)fdiv((uint32_t)r, b.group);
        const int head = pl.head * (int)b.group.d + r - tok * (int)b.group.d;
        const int64_t out_row = (int64_t)(q.q0 + tok);
        const float inv = l > 0.0f ? 1.0f / l : 0.0f;
        if (half * DV + col < p.dv) {
            uint4 v;
            v.x = pack2<Bf16>(o[0] * inv, o[1] * inv);
            v.y = pack2<Bf16>(o[2] * inv, o[3] * inv);
            v.z = pack2<Bf16>(o[4] * inv, o[5] * inv);
            v.w = pack2<Bf16>(o[6] * inv, o[7] * inv);
            *reinterpret_cast<uint4 *>(p.out + out_row * p.out_token + (int64_t)head * p.out_head + (half * DV + col) * 2) = v;
        }
        if (half == 0 && col == 0 && p.lse) p.lse[out_row * p.heads + head] = l > 0.0f ? fmaf(top, p.scale, logf(l)) : -INFINITY;
    }
}

template <int DV, bool Bf16>
int join_fragments(const Join &p, cudaStream_t s)
{
    return cuda_status(launch(join_kernel<DV, Bf16>, dim3(p.parts - 1, 8, p.halves), dim3(256), 0, s, p));
}

// 32 accumulator columns of a row to the output, scaled.
template <bool Bf16>
__device__ __forceinline__ void store_row32(char *to, const float (&o)[32], float inv, int col, int dv)
{
#pragma unroll
    for (int i = 0; i < 4; i++) {
        if (col + 8 * i < dv) {
            uint4 v;
            v.x = pack2<Bf16>(o[8 * i] * inv, o[8 * i + 1] * inv);
            v.y = pack2<Bf16>(o[8 * i + 2] * inv, o[8 * i + 3] * inv);
            v.z = pack2<Bf16>(o[8 * i + 4] * inv, o[8 * i + 5] * inv);
            v.w = pack2<Bf16>(o[8 * i + 6] * inv, o[8 * i + 7] * inv);
            *reinterpret_cast<uint4 *>(to + (col + 8 * i) * 2) = v;
        }
    }
}

// Launch attributes of every attention kernel, set once per device (kv_runtime.cu).
int prepare_attention(const DeviceInfo &dev);
int preload_attention_kernels();  // kv_attention.cu
int preload_latent_kernels();     // kv_latent.cu
int preload_expand_kernels();     // kv_expand.cu
int preload_mass_kernels();       // kv_mass.cu
int preload_evict_kernels();      // kv_evict.cu

}  // namespace pkv
