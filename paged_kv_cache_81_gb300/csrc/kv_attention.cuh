// What the attention kernels' host sides share: argument checks, the batch they pass on, the workspace.
#pragma once

#include <cmath>
#include <type_traits>

#include "kv_plan.cuh"
#include "kv_tensor.cuh"

namespace pkv {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int64_t kCounterBytes = KV_ATTENTION_ZEROED_BYTES;  // arrival counts of cut units, zero between calls

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

// A unit that was cut: parts c0 .. c0 + count - 1 hold a fragment each, the first in slot 2 c0 + 1 of the workspace
// and the others in slot 2 c (a part has at most one fragment that begins its unit and one that does not).
// Slot 2 c + 1 and the counter of an inner part belong to this unit too.
struct Cut {
    int c0, count, nth;  // nth: this part's
    __device__ __forceinline__ Cut(const Line &line, int begin, int cost)
    {
        if (line.nth >= 0) {
            c0 = line.part - line.nth;
            count = ceil_div(cost, line.each);
        } else {
            c0 = line.part_of(begin);
            int c1 = line.part_of(begin + cost - 1);
            if (line.snap && c0 < c1) {  // as Walk moves the ends of its pieces
                const int x = line.begin_of(c0 + 1) - begin;
                if (x <= line.snap && x <= cost - x) c0++;
            }
            if (line.snap && c0 < c1) {
                const int y = begin + cost - line.begin_of(c1);
                if (y <= line.snap && y < cost - y) c1--;
            }
            count = c1 - c0 + 1;
        }
        nth = line.part - c0;
    }
    __device__ __forceinline__ int slot(int i) const { return 2 * (c0 + i) + (i == 0); }
};

// Fragments that one group of threads adds up, for one half of the columns: `count` of them, `pitch` floats apart, the
// first `head` further on; sum: where a sum goes.
struct Pieces {
    float *at, *sum;
    int count, pitch, head;
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

// Joins rows [row0, row0 + rows) of a cut unit from fragments of `stride` floats, or (at.sum) adds fragments up to a
// new one, in an inner part's odd slot.  A fragment
// holds its accumulators four columns at a time, [DV / 4][stat rows][4], so that writing (a thread a row)
// and reading (a thread a row and some columns) are both coalesced, then the rows' maxima and sums.  128
// threads; a row's fragments are added in the order of their keys, so the result does not depend on which
// CTA came last.  Row r is (first + r) / group of the request's tokens from q0 on, head head0 + the
// rest.  Not inlined: its registers would crowd the loop over the key tiles.
template <int DV, bool Bf16>
__device__ __noinline__ void join_rows(const Output p, const Pieces at, int half, int row0, int rows, int stat, int first, int q0, int head0,
                                       const FastDiv group)
{
    // rows rounded up to a power of two; the other threads share out the columns (at least one quad each)
    int shift = DV == 64 ? 3 : DV == 128 ? 2 : 1;
    while ((1 << shift) < rows) shift++;
    const int t = threadIdx.x & 127, row = row0 + (t & ((1 << shift) - 1)), parts = 128 >> shift, quads = DV / 4 / parts;
    const int quad0 = (t >> shift) * quads;
    if (row >= row0 + rows) return;
    const int count = at.count;
    const auto fragment = [&](int i) { return at.at + (i * at.pitch + (i == 0 ? at.head : 0)); };
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
#pragma unroll 1
            for (int i0 = 0; i0 < count; i0 += kAhead) {
                float4 v[kAhead][kBatch];
                float pm[kAhead], pl[kAhead];
#pragma unroll
                for (int j = 0; j < kAhead; j++) {
                    const float *part = fragment(i0 + j);
                    pm[j] = -INFINITY;
                    pl[j] = 0.0f;
                    if (i0 + j < count) {
                        pm[j] = __ldcg(part + stat * DV + row);
                        pl[j] = __ldcg(part + stat * (DV + 1) + row);
                    }
#pragma unroll
                    for (int k = 0; k < kBatch; k++) {
                        v[j][k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        if (k < quads && i0 + j < count) v[j][k] = __ldcg(reinterpret_cast<const float4 *>(part) + (q + k) * stat + row);
                    }
                }
#pragma unroll
                for (int j = 0; j < kAhead; j++) {
                    const float a = exp2_fast((pm[j] - z) * p.c);
                    l += pl[j] * a;
#pragma unroll
                    for (int k = 0; k < kBatch; k++)
                        o[k].x += v[j][k].x * a, o[k].y += v[j][k].y * a, o[k].z += v[j][k].z * a, o[k].w += v[j][k].w * a;
                }
            }
            if (at.sum) {
#pragma unroll
                for (int k = 0; k < kBatch; k++)
                    if (k < quads) __stcg(reinterpret_cast<float4 *>(at.sum) + (q + k) * stat + row, o[k]);
                if (q == 0) {
                    at.sum[stat * DV + row] = top;
                    at.sum[stat * (DV + 1) + row] = l;
                }
                continue;
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
            if (half == 0 && q == 0 && p.lse) p.lse[token * p.heads + head] = l > 0.0f ? fmaf(top, p.scale, weight_log<Bf16>(l)) : -INFINITY;
        }
    };
    // what the registers beside the tile loop hold; two fragments (a long unit's usual cut) in four trips a row instead
    // of eight: three prefill chunks of 500 to 2000 tokens 117 us, so 114.5
    if (quads <= 4)
        columns(std::integral_constant<int, 4>(), std::integral_constant<int, 6>());
    else if (DV == 256)
        columns(std::integral_constant<int, 8>(), std::integral_constant<int, 3>());
    else if (count <= 2)
        columns(std::integral_constant<int, 8>(), std::integral_constant<int, 2>());
    else
        columns(std::integral_constant<int, 4>(), std::integral_constant<int, 4>());
}

// Called by the 128 threads of a group once they have written their fragment: rows [row0, row0 + rows) of
// halves [half0, half1) of the unit are joined by the group that wrote the last one.  Of many pieces the last of
// every kSum (3 to 10 at the unit's end) adds those up first, into the odd slot of the second of them: a group has
// some 40 KB of loads in flight, so a fragment takes it 0.3 (8 rows of 128) to 0.9 us (64 rows of 256).  One
// request of 16000 tokens, 8 heads over one key head: 30 us with one join of all pieces, 20 us so; of 60000 tokens,
// 128 heads: 164 and 55 us; latent, 32000 tokens, 64 heads: 81 and 40 us; 16 pieces of 128 rows 44 and 39 us.
// counter: the first part's; those of the parts are `apart`.
constexpr int kSum = 8;

template <int DV, bool Bf16>
__device__ __forceinline__ void join_unit(const Output &p, float *ws, const Cut &cut, int *counter, int apart, int halves, int half0, int half1,
                                          int stride, int row0, int rows, int stat, int first, int q0, int head0, const FastDiv &group, uint32_t bar,
                                          int &phase, volatile int *answer, const Waiter &wait, bool &ok)
{
    const bool many = cut.count > kSum + kSum / 2;
    const int sums = (cut.count - 3) / kSum + 1, mine = min(cut.nth / kSum, sums - 1);
    bool sum = many;
    for (;; sum = false) {
        const int from = sum ? mine * kSum : 0, n = sum ? (mine + 1 < sums ? kSum : cut.count - from) : many ? sums : cut.count;
        if (!last_of(counter + (sum ? (1 + mine) * apart : 0), n, bar, phase, answer, wait, ok)) return;
        const bool sums_of = many && !sum;
#pragma unroll 1
        for (int h = half0; h < half1; h++) {
            const auto slot = [&](int piece, int odd) { return ws + (2 * ((cut.c0 + piece) * halves + h) + odd) * stride; };
            const Pieces at{sums_of ? slot(1, 1) : slot(from, 0), sum ? slot(from + 1, 1) : nullptr, n, (sums_of ? kSum : 1) * 2 * halves * stride,
                            from == 0 && !sums_of ? stride : 0};
            join_rows<DV, Bf16>(p, at, h, row0, rows, stat, first, q0, head0, group);
        }
        if (!sum) return;
    }
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
