// What the attention kernels' host sides share: argument checks, the batch they pass on, the workspace.
#pragma once

#include <cmath>
#include <type_traits>

#include "kv_plan.cuh"
#include "kv_tensor.cuh"

namespace pkv {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int64_t kCounterBytes = 16384;  // arrival counts of cut units, zero between calls

// Two fragments a CTA: of 256 rows x (128 values + maximum + sum) for kv_attention, of 128 rows x (256
// values + maximum + sum) for each CTA of kv_latent_attention.
inline int64_t attention_workspace(int num_sms) { return kCounterBytes + (int64_t)num_sms * 2 * 256 * (128 + 2) * 4; }

int check_batch(const kv_attn_batch *t);
// A factor of the products that the kernels take: 8 / (scale log2 e), by which the maximum may grow before an
// accumulator is rescaled, and its reciprocal stay finite.
inline bool good_scale(float scale) { return scale >= 1e-30f && scale <= 1e30f; }
int fill_batch(Batch *b, const kv_attn_batch *t, int heads, int kv_heads, int block_size, int unit_rows, int tile_shift, int causal, int window);
int check_plane(const kv_cache_desc *c, int tensor, int plane, int heads, int dim);
int check_rows(const void *p, int64_t token_stride, int64_t head_stride);
// Tokens of a TMA of q: the smallest divisor of `most` (a group's tokens in 128 rows) that holds a request's
// new tokens on average, so that decoding brings no other request's rows and a chunk takes few boxes; a
// divisor, so that the last box of 128 rows ends with them.
int box_tokens(int most, const kv_attn_batch *t);
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
    __device__ __forceinline__ Cut(const Line &line, int begin, int cost)
    {
        if (line.nth >= 0) {
            c0 = line.part - line.nth;
            count = ceil_div(cost, line.each);
        } else {
            c0 = line.part_of(begin);
            count = line.part_of(begin + cost - 1) - c0 + 1;
        }
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

// Joins rows [row0, row0 + rows) of a cut unit from `count` fragments, `stride` floats a slot.  A fragment
// holds its accumulators four columns at a time, [DV / 4][stat rows][4], so that writing (a thread a row)
// and reading (a thread a row and some columns) are both coalesced, then the rows' maxima and sums.  128
// threads; a row's fragments are added in the order of their keys, so the result does not depend on which
// CTA came last.  Row r is (first + r) / group of the request's tokens from q0 on, head head0 + the
// rest.  Not inlined: its registers would crowd the loop over the key tiles.
template <int DV, bool Bf16>
__device__ __noinline__ void join_rows(const Output p, const float *ws, int c0, int count, int halves, int half, int stride, int row0, int rows, int stat,
                                       int first, int q0, int head0, const FastDiv group)
{
    // rows rounded up to a power of two; the other threads share out the columns (at least one quad each)
    int shift = DV == 64 ? 3 : DV == 128 ? 2 : 1;
    while ((1 << shift) < rows) shift++;
    const int t = threadIdx.x & 127, row = row0 + (t & ((1 << shift) - 1)), parts = 128 >> shift, quads = DV / 4 / parts;
    const int quad0 = (t >> shift) * quads;
    if (row >= row0 + rows) return;
    const auto fragment = [&](int i) { return ws + (2 * ((c0 + i) * halves + half) + (i == 0)) * (int64_t)stride; };
    float top = -INFINITY;
#pragma unroll 8
    for (int i = 0; i < count; i++) top = fmaxf(top, __ldcg(fragment(i) + stat * DV + row));
    const float z = top == -INFINITY ? 0.0f : top;
    const int tok = (int)fdiv((uint32_t)(first + row), group), head = head0 + first + row - tok * (int)group.d;
    const int64_t token = (int64_t)q0 + tok;
    char *to = p.out + token * p.out_token + (int64_t)head * p.out_head;
    // `Batch` column quads of `Ahead` fragments in flight: the loads take the time
    const auto columns = [&](auto batch, auto ahead) {
        constexpr int kBatch = batch(), kAhead = ahead();
#pragma unroll 1
        for (int q = quad0; q < quad0 + quads; q += kBatch) {
            float4 o[kBatch];
            float l = 0.0f;
#pragma unroll
            for (int k = 0; k < kBatch; k++) o[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll kAhead
            for (int i = 0; i < count; i++) {
                const float *part = fragment(i);
                const float pm = __ldcg(part + stat * DV + row), pl = __ldcg(part + stat * (DV + 1) + row);
                float4 v[kBatch];
#pragma unroll
                for (int k = 0; k < kBatch; k++)
                    if (k < quads) v[k] = __ldcg(reinterpret_cast<const float4 *>(part) + (q + k) * stat + row);
                const float a = exp2_fast((pm - z) * p.c);
                l += pl * a;
#pragma unroll
                for (int k = 0; k < kBatch; k++)
                    if (k < quads) o[k].x += v[k].x * a, o[k].y += v[k].y * a, o[k].z += v[k].z * a, o[k].w += v[k].w * a;
            }
            const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
            for (int k = 0; k < kBatch; k++)
                if (k < quads && half * DV + (q + k) * 4 < p.dv) {
                    uint2 v;
                    v.x = pack2<Bf16>(o[k].x * inv, o[k].y * inv);
                    v.y = pack2<Bf16>(o[k].z * inv, o[k].w * inv);
                    *reinterpret_cast<uint2 *>(to + (half * DV + (q + k) * 4) * 2) = v;
                }
            if (half == 0 && q == 0 && p.lse) p.lse[token * p.heads + head] = l > 0.0f ? fmaf(top, p.scale, logf(l)) : -INFINITY;
        }
    };
    if (quads <= 4)
        columns(std::integral_constant<int, 4>(), std::integral_constant<int, 6>());
    else
        columns(std::integral_constant<int, 8>(), std::integral_constant<int, 3>());
}

// 32 accumulator columns of a row into its fragment, as join_rows reads them.
__device__ __forceinline__ void store_fragment32(float *part, int rows, int row, int q, const float (&f)[32])
{
    float4 *d = reinterpret_cast<float4 *>(part) + q * 8 * rows + row;
#pragma unroll
    for (int i = 0; i < 8; i++) __stcg(d + i * rows, make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]));
}

// 32 accumulator columns of every lane's row to global memory, scaled and rounded.  A thread holds a whole
// row, and 16-byte stores a row apart would each take a cache line to themselves: four lanes first exchange
// their 16-byte pieces, so that a store instruction writes 64 consecutive bytes of eight rows.  Called by
// whole warps; `to` is the lane's row, nullptr where there is nothing to write; columns from `end` on do not exist.
template <bool Bf16>
__device__ __forceinline__ void store_rows32(char *to, const float (&o)[32], float inv, int col, int end)
{
    const int lane = threadIdx.x & 31, a = lane & 3;
    uint32_t v[4][4];
#pragma unroll
    for (int i = 0; i < 16; i++) v[i / 4][i % 4] = pack2<Bf16>(o[2 * i] * inv, o[2 * i + 1] * inv);
#pragma unroll
    for (int s = 1; s <= 2; s *= 2)  // piece j of lane a's row <-> piece a of lane j's row
#pragma unroll
        for (int j = 0; j < 4; j++)
            if (!(j & s))
#pragma unroll
                for (int w = 0; w < 4; w++) {
                    const uint32_t got = __shfl_xor_sync(0xffffffffu, a & s ? v[j][w] : v[j | s][w], s);
                    if (a & s)
                        v[j][w] = got;
                    else
                        v[j | s][w] = got;
                }
    const unsigned long long mine = (unsigned long long)to;
#pragma unroll
    for (int j = 0; j < 4; j++) {
        char *row = (char *)__shfl_sync(0xffffffffu, mine, (lane & 28) | j);
        if (row != nullptr && col + 8 * a < end)
            *reinterpret_cast<uint4 *>(row + (col + 8 * a) * 2) = make_uint4(v[j][0], v[j][1], v[j][2], v[j][3]);
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
