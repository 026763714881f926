// What the attention kernels' host sides share: argument checks, the batch they pass on, the workspace.
#pragma once

#include <cmath>

#include "kv_plan.cuh"
#include "kv_tensor.cuh"

namespace pkv {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int64_t kCounterBytes = 16384;  // arrival counts of cut units, zero between calls

// Two fragments a CTA: of 256 rows x (128 values + maximum + sum) for kv_attention, of 128 rows x (256
// values + maximum + sum) for each CTA of kv_latent_attention.
inline int64_t attention_workspace(int num_sms) { return kCounterBytes + (int64_t)num_sms * 2 * 256 * (128 + 2) * 4; }

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

// A unit that was cut: parts c0 .. c1 hold a fragment each, the first in slot 2 c0 + 1 of the workspace
// and the others in slot 2 c (a CTA has at most one fragment that begins its unit and one that does not).
struct Cut {
    int c0, count;
    __device__ __forceinline__ Cut(const Line &line, long long begin, int cost)
        : c0(line.part_of(begin)), count(line.part_of(begin + cost - 1) - c0 + 1)
    {
    }
    __device__ __forceinline__ int slot(int i) const { return 2 * (c0 + i) + (i == 0); }
};

// Called by the 128 threads of a group once they have written a fragment: true in the group that wrote
// the last of the `count` fragments, which then sees them all.  bar: a barrier of four (warp) arrivals that
// the group keeps for this; answer: a word of shared memory.  ok becomes false if a wait runs out.
__device__ __forceinline__ bool last_of(int *counter, int count, uint32_t bar, int &phase, volatile int *answer, const Waiter &wait, bool &ok)
{
    __threadfence();
    warp_arrive(bar);
    if (!(ok = wait.warp(bar, phase++ & 1))) return false;
    if ((threadIdx.x & 127) == 0) {
        const bool last = atomicAdd(counter, 1) == count - 1;
        if (last) atomicExch(counter, 0);  // as the next call wants it
        __threadfence();
        *answer = last;
    }
    warp_arrive(bar);
    if (!(ok = wait.warp(bar, phase++ & 1))) return false;
    return *answer != 0;
}

struct Output {
    char *out;
    int64_t out_token, out_head;
    float *lse;
    int32_t heads, dv;
    float scale, c;
};

// Joins rows [row0, row0 + rows) of a cut unit from `count` fragments, `stride` floats a slot: accumulators
// [.., DV], then maxima and sums `stat` apart.  128 threads; a row's fragments are read in the order of
// their keys, so the result does not depend on which CTA came last.  Row r is (first + r) / group of the
// request's tokens from q0 on, head head0 + the rest.  Not inlined: its registers would crowd the loop
// over the key tiles.
template <int DV, bool Bf16>
__device__ __noinline__ void join_rows(const Output p, const float *ws, int c0, int count, int halves, int half, int stride, int row0, int rows, int stat,
                                       int first, int q0, int head0, const FastDiv group)
{
    const int out_col = half * DV;
    const bool with_lse = half == 0;
    constexpr int kLanes = DV / 8, kRowsPerPass = 128 / kLanes, kBatch = 4;
    const int t = threadIdx.x & 127, col = (t % kLanes) * 8;
    for (int r0 = row0 + t / kLanes; r0 < row0 + rows; r0 += kRowsPerPass * kBatch) {
        // four rows at a time: the loads, not the arithmetic, take the time
        float o[kBatch][8], m[kBatch], l[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; k++) {
            m[k] = -INFINITY, l[k] = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; j++) o[k][j] = 0.0f;
        }
#pragma unroll 1
        for (int i = 0; i < count; i++) {
            const float *part = ws + (2 * ((c0 + i) * halves + half) + (i == 0)) * (int64_t)stride;
            float pm[kBatch], pl[kBatch];
            float4 v[kBatch][2];
#pragma unroll
            for (int k = 0; k < kBatch; k++) {
                const int row = min(r0 + k * kRowsPerPass, row0 + rows - 1);
                pm[k] = __ldcg(part + stat * DV + row);
                pl[k] = __ldcg(part + stat * (DV + 1) + row);
                v[k][0] = __ldcg(reinterpret_cast<const float4 *>(part + row * DV + col));
                v[k][1] = __ldcg(reinterpret_cast<const float4 *>(part + row * DV + col + 4));
            }
#pragma unroll
            for (int k = 0; k < kBatch; k++) {
                const float top = fmaxf(m[k], pm[k]), z = top == -INFINITY ? 0.0f : top;
                const float a = exp2_fast((m[k] - z) * p.c), b = exp2_fast((pm[k] - z) * p.c);
                m[k] = top;
                l[k] = l[k] * a + pl[k] * b;
                o[k][0] = o[k][0] * a + v[k][0].x * b, o[k][1] = o[k][1] * a + v[k][0].y * b;
                o[k][2] = o[k][2] * a + v[k][0].z * b, o[k][3] = o[k][3] * a + v[k][0].w * b;
                o[k][4] = o[k][4] * a + v[k][1].x * b, o[k][5] = o[k][5] * a + v[k][1].y * b;
                o[k][6] = o[k][6] * a + v[k][1].z * b, o[k][7] = o[k][7] * a + v[k][1].w * b;
            }
        }
#pragma unroll
        for (int k = 0; k < kBatch; k++) {
            const int row = r0 + k * kRowsPerPass;
            if (row >= row0 + rows) break;
            const int tok = (int)fdiv((uint32_t)(first + row), group), head = head0 + first + row - tok * (int)group.d;
            const int64_t token = (int64_t)q0 + tok;
            const float inv = l[k] > 0.0f ? 1.0f / l[k] : 0.0f;
            if (out_col + col < p.dv) {
                uint4 v;
                v.x = pack2<Bf16>(o[k][0] * inv, o[k][1] * inv);
                v.y = pack2<Bf16>(o[k][2] * inv, o[k][3] * inv);
                v.z = pack2<Bf16>(o[k][4] * inv, o[k][5] * inv);
                v.w = pack2<Bf16>(o[k][6] * inv, o[k][7] * inv);
                *reinterpret_cast<uint4 *>(p.out + token * p.out_token + (int64_t)head * p.out_head + (out_col + col) * 2) = v;
            }
            if (with_lse && col == 0 && p.lse) p.lse[token * p.heads + head] = l[k] > 0.0f ? fmaf(m[k], p.scale, logf(l[k])) : -INFINITY;
        }
    }
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
