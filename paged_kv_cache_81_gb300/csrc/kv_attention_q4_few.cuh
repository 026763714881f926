// kv_attention_q4 for few rows: decoding, with at most 16 query rows (tokens x heads of a key head's group) a unit.
//
// The same one-pass softmax as kv_attention.cu.  What bounds it is memory, at 4.5 bits an element, so the work a
// byte is 3.5 times that of a 16-bit cache: an SM gets 41 elements a cycle, and can issue about three instructions for
// each.  So a code is touched once: it goes from shared memory to the registers of the warp that multiplies it, where
// one conversion and one product with its scale make two fp16 values of it, exact (six significant bits), in the place that a
// warp-wide product's operand wants (mma.sync with 8 query rows as its N: keys are the rows of S^T = K Q^T, and O^T = V^T P^T;
// the dimensions' order within a thread's part is free in the first product, the keys' order in the second).  A
// tcgen05 product would want them written to shared memory, twice the bytes of the cache's 16-bit rows a cycle
// (82 in and 82 out of 128), or both operands in 4 bits, which queries and weights are not.
//
// Measured: 64 requests of 4096 to 12288 tokens, 32 heads over 8 of 128, pages of 16: 114 us, 81% of the copy rate: about 98% between the
// first tile and the last, 8 us before and 5 to 12 after (ends of pieces, joins); with 16 key heads 212 us, 87%.  The integer pipe is half
// taken, by codes.  12 rows over 64 requests of 8000: 150 us, 59%: two products of 8 rows, twice the exponentials.
//
// Queries are brought to [1, 2) by a power of two a row and held in fp16, weights are fp16, 2^7 times as large (kv_tensor.cuh,
// weight_offset); sums are in 32 bits.  fp16 since a product's operands have one type, and codes times scales are exact in it but not in bf16; a
// second product for what the rounding of weights leaves would double the second half of the work.  The reference m of a row's weights is one of its scores, as the product left them, and is taken off
// before the product with c: 2^(c (s - m) + 7) with s - m <= 8 / c, which stays below fp16's 2^16 whatever the size of s.  (With c s and c m rounded
// by themselves it did not from scaled scores of 10^7 on; the long decode batch takes 1 us more so, twelve rows 2 us less.)
//
// One persistent CTA per SM; a unit is one request's rows of as many key heads as there are warps for, or fewer (launch_few).
//   warps 0, 1 (to 3)  bring rows of keys and of values by TMA, one for each run of slots inside a page, into rings of tiles
//   other warps        each one key head and every n-th 16 keys of a tile: scores, weights, values, with a running maximum and sum of
//                      its own; at the unit's end the warps of a head join through shared memory, while those that are done go on
//                      with the next unit; pieces of cut units are joined through the workspace at the CTA's end
// The 16 keys of a step are taken in an order (order_of) in which the keys' 16-byte reads do not meet in a bank, and the values'
// 8-byte reads at most in pairs.
#pragma once

#include <algorithm>

#include "kv_attention_q4.cuh"

namespace pkv {

namespace {

constexpr int kLeast = 2;     // tiles of a piece of a unit, at least
constexpr int kMaxSlots = 8;
constexpr float kNothing = -3e38f;  // the reference of a row that has seen no key yet: a number, so that a hidden score less it is -inf still
constexpr int kMany = 12;     // pieces of a unit from which on they are joined in two stages
// The key of row r of 8 (hexadecimal digit r) by how far rows lie apart: in pairs that are 64 bytes off one another, modulo 128.
constexpr uint32_t order_of(uint32_t pitch)
{
    return pitch % 128 == 64 ? 0x76543210u : 2 * pitch % 128 == 64 ? 0x57463120u : 0x73516240u;
}

// H: see attention_q4_few_kernel.
template <int D, int NT, int H>
struct Few {
    static constexpr int kWarps = NT == 1 ? 16 : 8;  // that compute
    // Warps that load.  Rows of one or two heads come in short runs, and two warps do not issue them fast enough (152 requests of 20480
    // tokens, two heads: 167 us, with four 151); where they do, two more cost a call 2 us.
    static constexpr int kLoaders = H == 1 || H == 2 ? 4 : 2;
    static constexpr int kThreads = 32 * (kWarps + kLoaders);
    // Groups of 16 keys that a warp takes of a tile; of one head's rows half as many leave room for more than one tile.
    static constexpr int kSteps = (NT == 1 ? 2 : 4) / (H == 1 ? 2 : 1);
    static constexpr uint32_t kQ = NT * (D / 32) * 512;  // bytes of a warp's queries
};

// Where a unit's heads of a tile lie in shared memory: rows of codes and of scales, `codes` and `scales` bytes apart.  All heads of
// a row come together, the scales behind the codes; some of them in two loads, the scales behind all codes of the tile.
struct Place4 {
    int32_t codes, scales;
    int32_t first;  // of the first row's scales
    int32_t bytes;  // of a tile
    int32_t apart;  // two loads
    // rows follow one another in the page too: a run is one untiled copy (a tiled one takes 8 cycles a row, and more a load)
    int32_t dense;
    uint64_t base;
    int64_t block_stride;
};

struct FewParams : Q4Params {
    int32_t bf16;
    uint32_t order;
    int32_t unit_heads;        // key heads of a unit
    int32_t split;             // warps of a key head
    int32_t tile;              // keys
    int32_t slots;             // tiles of each ring
    int32_t piece_rows;        // slots that one TMA brings: they never leave a page
    Place4 kl, vl;
};

// A unit's rows.
struct HeadRows {
    int row0, rows;  // of the request
    int64_t q0;      // its first token
};

// Counts a piece whose writes come before this; true for the last of `count`, which sees what the others wrote.
__device__ __forceinline__ bool count_in(int *counter, int count)
{
    int before;
    asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
    if (before != count - 1) return false;
    atomicExch(counter, 0);  // as the next call wants it
    return true;
}

// A cut unit of which this CTA has a piece (at most one that ends in its part of the line, and one that begins there).
struct CutUnit {
    int c0, count, nth;  // Cut
    int head0;           // the first key head
    HeadRows rows;
    int stored;          // heads whose pieces are in the workspace
    int last;            // every part's are: this CTA joins them
};

// Pieces of a group, so that both stages have as many.
__device__ __forceinline__ int group_of(int count)
{
    int n = 3;
#pragma unroll 1
    while (n * n < count) n++;
    return n;
}

// Whether all heads of a row come together and rows follow one another, in runs that end on a multiple of 128 bytes.
inline bool dense_rows(const FewParams &p, const Q4Plane &plane)
{
    const kv_cache_desc &d = *plane.desc;
    return p.unit_heads == p.heads_all && d.token_stride == d.row_bytes && (int64_t)d.row_bytes * p.piece_rows % 128 == 0;
}

struct Aux {
    uint64_t k_full[kMaxSlots], k_empty[kMaxSlots], v_full[kMaxSlots], v_empty[kMaxSlots];
    uint64_t join_first[8], join_full[8], join_free[8];  // a place of the join: filled in the first round, in a later one; free
    uint64_t sync;
    CutUnit cut[2];  // that end in its part, that begin there
    int scan[4 * 20];
    Place place;
    Walk walk[20];  // of each warp: held in registers it would crowd the loop over the tiles
    unsigned char size[16][16];  // of each computing warp's rows: the exponent of the power of two that was taken off
    int gave_up;
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The 8 x 8 matrix of 16-bit elements that the warp holds, a row in four lanes, transposed.
__device__ __forceinline__ uint32_t transposed8(uint32_t v)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t s)
{
    uint32_t v;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(v) : "r"(a), "r"(b), "r"(s));
    return v;
}

__device__ __forceinline__ uint32_t ld_smem4(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 ld_smem8(uint32_t a)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld_smem2(uint32_t a)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld_smem1(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

// Steps to the next unit through registers: each lane's read of the shared walk comes before any lane's write.
__device__ __forceinline__ bool next_of(Walk &shared, const Batch &b)
{
    Walk w = shared;
    const bool more = w.next(b);
    __syncwarp();
    shared = w;
    return more;
}

// A tile as a loading warp sees it, one of Warps that share it: every Warps-th run of slots inside a page, one a lane (and every 32nd
// after it), and the page of the lane's first one, asked for a tile ahead: a trip to the block table takes as long as half a tile's work.
template <int Warps>
struct Tile {
    const int32_t *row;
    int kb, h0, p0, p1;  // this warp's runs: p0, p0 + Warps, .. below p1
    int page, slot;

    __device__ __forceinline__ void look(const FewParams &p, int i)
    {
        const uint32_t key = (uint32_t)(kb + i * p.piece_rows), col = fdiv(key, p.block);
        slot = (int)(key - col * p.block.d);
        page = __ldg(row + col);
    }
    __device__ __forceinline__ void start(const FewParams &p, const Walk &w, int t, int tile_keys, int heads, int which)
    {
        row = p.table + (int64_t)w.at.req * p.table_stride;
        kb = (w.u.tile0 + w.at.off + t) * tile_keys;
        h0 = w.at.head * heads;
        p0 = max(0, w.u.lo - kb) / p.piece_rows + which;
        p1 = (min(w.u.hi - kb, tile_keys) + p.piece_rows - 1) / p.piece_rows;
        const int i = p0 + Warps * (threadIdx.x & 31);
        if (i < p1) look(p, i);
    }
    // Its rows of keys or values: a TMA (two where heads are apart) a run.
    __device__ __forceinline__ void load(const FewParams &p, const CUtensorMap *map, const CUtensorMap *scale_map, int dim, const Place4 &place, uint32_t to,
                                         uint32_t bar, bool report)
    {
        const int lane = threadIdx.x & 31, pr = p.piece_rows, runs = max(p1 - p0 + Warps - 1, 0) / Warps;
        if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(runs * pr) * (place.codes + (place.apart ? place.scales : 0)));
        __syncwarp();
        for (int j = lane; j < runs; j += 32) {
            const int i = p0 + Warps * j;
            if (j >= 32) look(p, i);
            int from = page;
            if (from < 0 || from >= p.num_blocks) {
                if (report) set_error(p.b.err, KV_DERR_TABLE);
                from = p.no_page;
            } else if (place.dense) {
                bulk_load(to + i * pr * place.codes, place.base + (uint64_t)from * place.block_stride + (uint32_t)(slot * place.codes), pr * place.codes, bar);
                continue;
            }
            tma_load_3d(to + i * pr * place.codes, map, bar, h0 * dim / 2 >> row_map_shift(place.codes), slot, from);
            if (place.apart)
                tma_load_3d(to + place.first + i * pr * place.scales, scale_map, bar, ((p.heads_all * dim / 2 + h0 * dim / 16) & ~15) / 4, slot, from);
        }
        __syncwarp();
    }
};

// One warp's sums over some keys, as its threads hold them.  A piece of them in memory: O [row][D], then a maximum and a sum a row.
template <int D, int NT>
struct Sums {
    static constexpr int kPitch = D + 4;                    // floats of a row in shared memory
    static constexpr int kShared = 8 * NT * (kPitch + 2);   // of a piece there
    static constexpr int kFloats = 8 * NT * (D + 2);        // of a piece in the workspace
    float o[D / 16][NT][4];
    float m[NT][2], l[NT][2];

    // The columns of rows below `rows` to a place in shared or global memory.
    template <bool Shared>
    __device__ __forceinline__ void store(float *at, int rows) const
    {
        const int lane = threadIdx.x & 31, n = lane >> 2, t = lane & 3;
#pragma unroll
        for (int x = 0; x < NT; x++)
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const int r = 8 * x + 2 * t + i;
                if (r >= rows) continue;
                float4 *const to = reinterpret_cast<float4 *>(at + r * (Shared ? kPitch : D) + n * (D / 8));
#pragma unroll
                for (int k = 0; k < D / 32; k++) {
                    const float4 v = make_float4(o[2 * k][x][i], o[2 * k][x][i + 2], o[2 * k + 1][x][i], o[2 * k + 1][x][i + 2]);
                    if (Shared)
                        to[k] = v;
                    else
                        __stcg(to + k, v);
                }
                if (n == 0) {
                    float2 *const stat = reinterpret_cast<float2 *>(at + 8 * NT * (Shared ? kPitch : D)) + r;
                    if (Shared)
                        *stat = make_float2(m[x][i], l[x][i]);
                    else
                        __stcg(stat, make_float2(m[x][i], l[x][i]));
                }
            }
    }
    // Others from shared memory are added; c: log2 of a weight a unit of the maxima.
    __device__ __forceinline__ void join(const float *from, int rows, const float (&c)[NT][2])
    {
        const int lane = threadIdx.x & 31, n = lane >> 2, t = lane & 3;
#pragma unroll
        for (int x = 0; x < NT; x++)
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const int r = 8 * x + 2 * t + i;
                if (r >= rows) continue;
                const float2 ml = reinterpret_cast<const float2 *>(from + 8 * NT * kPitch)[r];
                const float top = fmaxf(m[x][i], ml.x);
                const float a = exp2_fast((m[x][i] - top) * c[x][i]), f = exp2_fast((ml.x - top) * c[x][i]);
                m[x][i] = top;
                l[x][i] = l[x][i] * a + ml.y * f;
#pragma unroll
                for (int j = 0; j < D / 32; j++) {
                    const float4 v = reinterpret_cast<const float4 *>(from + r * kPitch + n * (D / 8))[j];
                    o[2 * j][x][i] = o[2 * j][x][i] * a + v.x * f, o[2 * j][x][i + 2] = o[2 * j][x][i + 2] * a + v.y * f;
                    o[2 * j + 1][x][i] = o[2 * j + 1][x][i] * a + v.z * f, o[2 * j + 1][x][i + 2] = o[2 * j + 1][x][i + 2] * a + v.w * f;
                }
            }
    }
};
static_assert(16 * Sums<128, 1>::kFloats <= 256 * 130 && 8 * Sums<128, 2>::kFloats <= 256 * 130, "a piece fits its place in the workspace");

// Row r of a unit: where its output begins, and its lse.
__device__ __forceinline__ char *row_out(const FewParams &p, const HeadRows &u, int head0, int r, float *&lse)
{
    const int x = u.row0 + r, tok = (int)fdiv((uint32_t)x, p.b.group), head = head0 + x - tok * (int)p.b.group.d;
    const int64_t token = u.q0 + tok;
    lse = p.o.lse ? p.o.lse + token * p.o.heads + head : nullptr;
    return p.o.out + token * p.o.out_token + (int64_t)head * p.o.out_head;
}
__device__ __forceinline__ float lse_of(const FewParams &p, float m, float l) { return l > 0.0f ? fmaf(m, p.o.scale, weight_log<false>(l)) : -INFINITY; }
__device__ __forceinline__ uint32_t pack_out(const FewParams &p, float a, float b) { return p.bf16 ? pack2<true>(a, b) : pack2<false>(a, b); }

// Joins `count` pieces of one head of a cut unit in the workspace, in their order, by `threads` threads of which this is number `thread`.
// each 0: pieces from, from + 1, ..; else the sums of groups of `each`.  sum: to a new piece, the odd one of piece from + 1, else to the
// output.  A thread takes four values of a row at a time, of four pieces a trip to memory.
template <int D, int NT>
__device__ __forceinline__ void join_pieces(const FewParams &p, const CutUnit &unit, int h, int from, int each, int count, bool sum, int thread, int threads)
{
    const HeadRows u = unit.rows;
    float *const ws = p.ws + (int64_t)(2 * unit.c0) * (256 * 130) + h * Sums<D, NT>::kFloats;
    constexpr int kStats = 8 * NT * D;
    constexpr int kWide = NT == 1 ? 2 : 4;  // values of so many rows at a time
#pragma unroll 1
    for (int i0 = thread; i0 < u.rows * (D / 4); i0 += kWide * threads) {
        int r[kWide], quad[kWide];
        float4 o[kWide];
        float top[kWide], l[kWide];
#pragma unroll
        for (int j = 0; j < kWide; j++) {
            const int i = min(i0 + j * threads, u.rows * (D / 4) - 1);  // the last one again past the end
            r[j] = i / (D / 4), quad[j] = i % (D / 4);
            o[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            top[j] = -INFINITY, l[j] = 0.0f;
        }
#pragma unroll 1
        for (int k0 = 0; k0 < count; k0 += 4) {
            float4 w[kWide][4];
            float2 s[kWide][4];
#pragma unroll
            for (int k = 0; k < 4; k++) {
                // pieces lie in even slots but the unit's first, sums in the odd slot of their second piece
                const int piece = each ? (k0 + k) * each + 1 : from + k0 + k;
                const float *const at = ws + (2 * piece + (each || piece == 0)) * (256 * 130);
#pragma unroll
                for (int j = 0; j < kWide; j++) {
                    w[j][k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f), s[j][k] = make_float2(-INFINITY, 0.0f);
                    if (k0 + k < count) {
                        w[j][k] = __ldcg(reinterpret_cast<const float4 *>(at + r[j] * D) + quad[j]);
                        s[j][k] = __ldcg(reinterpret_cast<const float2 *>(at + kStats) + r[j]);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < kWide; j++) {
                const float now = fmaxf(fmaxf(fmaxf(s[j][0].x, s[j][1].x), fmaxf(s[j][2].x, s[j][3].x)), top[j]), z = now == -INFINITY ? 0.0f : now;
                const float a = exp2_fast((top[j] - z) * p.o.c);
                top[j] = now;
                l[j] *= a, o[j].x *= a, o[j].y *= a, o[j].z *= a, o[j].w *= a;
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    const float f = exp2_fast((s[j][k].x - z) * p.o.c);
                    l[j] += s[j][k].y * f, o[j].x += w[j][k].x * f, o[j].y += w[j][k].y * f, o[j].z += w[j][k].z * f, o[j].w += w[j][k].w * f;
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kWide; j++) {
            if (j > 0 && i0 + j * threads >= u.rows * (D / 4)) break;
            if (sum) {
                float *const to = ws + (2 * (from + 1) + 1) * (256 * 130);
                __stcg(reinterpret_cast<float4 *>(to + r[j] * D) + quad[j], o[j]);
                if (quad[j] == 0) __stcg(reinterpret_cast<float2 *>(to + kStats) + r[j], make_float2(top[j], l[j]));
            } else {
                float *lse;
                char *const to = row_out(p, u, (unit.head0 + h) * (int)p.b.group.d, r[j], lse);
                const float inv = l[j] > 0.0f ? p.v_scale / l[j] : 0.0f;
                if (quad[j] * 4 < p.o.dv)
                    reinterpret_cast<uint2 *>(to)[quad[j]] = make_uint2(pack_out(p, o[j].x * inv, o[j].y * inv), pack_out(p, o[j].z * inv, o[j].w * inv));
                if (quad[j] == 0 && lse) *lse = lse_of(p, top[j], l[j]);
            }
        }
    }
}

// H: the unit's heads where they are all of a row's, fill the widths D, and rows follow one another (they then lie a constant
// distance apart), else 0.
template <int D, int NT, int H>
__global__ void __launch_bounds__(Few<D, NT, H>::kThreads, 1)
attention_q4_few_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map, const __grid_constant__ CUtensorMap ks_map,
                        const __grid_constant__ CUtensorMap vs_map, const __grid_constant__ FewParams p)
{
    using F = Few<D, NT, H>;
    extern __shared__ __align__(128) unsigned char smem[];
    Aux &aux = *reinterpret_cast<Aux *>(smem);
    const bool bf16 = p.bf16;
    const int heads = H ? H : p.unit_heads, split = H ? F::kWarps / H : p.split, users = heads * split;  // warps that compute: users
    const int dk = H ? D : p.k.dim, dv = H ? D : p.v.dim, tile_keys = 16 * split * F::kSteps;
    constexpr uint32_t kPitch = (H * D * 9 + 255) / 256 * 16;
    const uint32_t k_row = H ? kPitch : p.kl.codes, y_row = H ? kPitch : p.kl.scales, v_row = H ? kPitch : p.vl.codes, x_row = H ? kPitch : p.vl.scales;
    const uint32_t k_tile = H ? kPitch * tile_keys : p.kl.bytes, v_tile = H ? kPitch * tile_keys : p.vl.bytes;

    unsigned char *const queries = smem + ((sizeof(Aux) + 127) & ~127u);
    float *const joins = reinterpret_cast<float *>(queries + F::kWarps * F::kQ);
    const uint32_t ring = smem_addr(joins) + (((uint32_t)(users / 2) * Sums<D, NT>::kShared * 4 + 127) & ~127u);
    const uint32_t v_ring = ring + (uint32_t)p.slots * p.kl.bytes;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const Batch &b = p.b;
    const Waiter wait{&aux.gave_up, b.err};
    if (tid == 0) {
        aux.gave_up = 0;
        aux.cut[0].last = aux.cut[1].last = aux.cut[0].stored = aux.cut[1].stored = aux.cut[0].rows.rows = 0;
        mbar_init(smem_addr(&aux.sync), users);
        for (int i = 0; i < p.slots; i++) {
            mbar_init(smem_addr(&aux.k_full[i]), F::kLoaders / 2);
            mbar_init(smem_addr(&aux.v_full[i]), F::kLoaders / 2);
            mbar_init(smem_addr(&aux.k_empty[i]), users);
            mbar_init(smem_addr(&aux.v_empty[i]), users);
        }
        for (int i = 0; i < 8; i++) {
            mbar_init(smem_addr(&aux.join_first[i]), 1);
            mbar_init(smem_addr(&aux.join_full[i]), 1);
            mbar_init(smem_addr(&aux.join_free[i]), 1);
        }
        mbar_init_fence();
        tma_prefetch_map(&k_map);
        tma_prefetch_map(&v_map);
    }
    grid_dep_entry();
    const Line line = find_place<F::kThreads>(b, blockIdx.x, gridDim.x, kLeast, aux.scan, &aux.place, blockIdx.x == 0);
    __syncthreads();
    Walk &w = aux.walk[warp];
    Walk first;
    const bool any = first.start(b, aux.place, line);
    w = first;  // every lane writes the same
    __syncwarp();
    if (!any) {
        // nothing to do: on to the common exit
    } else if (warp < F::kLoaders) {
        // ---- rows of keys, rows of values ----
        const bool v = warp & 1;
        const CUtensorMap *const map = v ? &v_map : &k_map, *const scale_map = v ? &vs_map : &ks_map;
        const Place4 &place = v ? p.vl : p.kl;
        const uint32_t to = v ? v_ring : ring, bytes = v ? v_tile : k_tile;
        const uint64_t *const full = v ? aux.v_full : aux.k_full, *const empty = v ? aux.v_empty : aux.k_empty;
        int it = 0, s = 0, at = 0;
        uint32_t phase = 1;
        Tile<F::kLoaders / 2> tile, next;
        // the tile after the one that it was called for last
        const auto ahead = [&](Tile<F::kLoaders / 2> &t) {
            while (at >= first.n || first.u.tiles == 0) {
                at = 0;
                if (!first.next(b)) return false;
            }
            t.start(p, first, at++, tile_keys, heads, warp >> 1);
            return true;
        };
        bool more = ahead(next);
        while (more) {
            tile = next;
            more = ahead(next);
            if (it++ >= p.slots && !wait.warp(smem_addr(&empty[s]), phase)) break;
            tile.load(p, map, scale_map, v ? dv : dk, place, to + s * bytes, smem_addr(&full[s]), !v);
            if (++s == p.slots) s = 0, phase ^= 1;
        }
    } else if (warp < users + F::kLoaders) {
        const int me = warp - F::kLoaders, h = me / split, part = me - h * split;
        bool ok = true;
        const int n = lane >> 2, t = lane & 3;
        const uint32_t order = H ? order_of(kPitch) : p.order;
        const uint32_t rk = (order >> (4 * n)) & 7;                                    // keys of score rows n, n + 8
        const uint32_t ra = (order >> (8 * t)) & 7, rb = (order >> (8 * t + 4)) & 7;  // keys of product columns 2 t, 2 t + 1
        const uint32_t g0 = 16u * part;
        // this thread's scales in a word of them; dimensions that heads do not have count as zeros
        const uint32_t k_mask = t * (D / 4) >= dk ? 0u : D == 128 && t * (D / 4) + 16 < dk ? 0xffffu : 0xffu;
        const uint32_t v_mask = n * (D / 8) < dv ? 0xffu : 0u;
        int s = 0, joined = 0;
        uint32_t phase = 0;
        Sums<D, NT> sums;
        auto &o = sums.o;
        auto &m = sums.m;
        auto &l = sums.l;
        const auto next_unit = [&] {
            __syncwarp();
            const bool more = next_of(w, b);
            __syncwarp();
            return more;
        };
        do {
            const int rows = w.u.rows, head0 = w.at.head * heads;
            // row r of a key head: its token and query head
            const auto token_of = [&](int r, int &head_in) {
                const int x = w.u.row0 + r, tok = (int)fdiv((uint32_t)x, b.group);
                head_in = x - tok * (int)b.group.d;
                return (int64_t)w.q.q0 + tok;
            };
            if (w.u.tiles == 0) {  // nothing is seen
                for (int i = me * 32 + lane; i < heads * rows; i += users * 32) {
                    int g;
                    const int hh = i / rows;
                    const int64_t token = token_of(i - hh * rows, g);
                    const int head = (head0 + hh) * (int)b.group.d + g;
                    char *to = p.o.out + token * p.o.out_token + (int64_t)head * p.o.out_head;
                    for (int col = 0; col < p.o.dv; col += 8) *reinterpret_cast<uint4 *>(to + col * 2) = make_uint4(0, 0, 0, 0);
                    if (p.o.lse) p.o.lse[token * p.o.heads + head] = -INFINITY;
                }
                continue;
            }
            // ---- queries: row n (and n + 8) of the unit, this thread's quarter of the dimensions ----
            // as the products take it, 16 bytes a thread for two of them
            const uint32_t q_at = smem_addr(queries) + me * F::kQ + lane * 16;
            float c[NT][2];  // of the columns 2 t, 2 t + 1: log2 of a weight a unit of the products
#pragma unroll
            for (int x = 0; x < NT; x++) {
                const int r = 8 * x + n;
                uint4 raw[D / 32];
#pragma unroll
                for (int i = 0; i < D / 32; i++) raw[i] = make_uint4(0, 0, 0, 0);
                if (r < rows) {
                    int g;
                    const int64_t token = token_of(r, g);
                    const char *from = p.q + token * p.q_token + (int64_t)((head0 + h) * (int)b.group.d + g) * p.q_head;
#pragma unroll
                    for (int i = 0; i < D / 32; i++)
                        if (t * (D / 4) + 8 * i < dk) raw[i] = __ldg(reinterpret_cast<const uint4 *>(from) + t * (D / 32) + i);
                }
                float to = 1.0f;
                uint32_t e = 127;
                if (bf16) {
                    float most = 0.0f;
#pragma unroll
                    for (int i = 0; i < D / 32; i++) {
                        const uint32_t v[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
                        for (int j = 0; j < 4; j++)
                            most = fmaxf(most, fmaxf(fabsf(__uint_as_float(v[j] << 16)), fabsf(__uint_as_float(v[j] & 0xffff0000u))));
                    }
                    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
                    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
                    e = min(max(__float_as_uint(most) >> 23, 1u), 253u);
                    to = __uint_as_float((254u - e) << 23);
                }
                if (t == 0) aux.size[me][r] = (unsigned char)e;
                const float back = __uint_as_float(e << 23);
#pragma unroll
                for (int i = 0; i < D / 32; i++) {
                    const uint32_t v[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
                    uint32_t f[4];
#pragma unroll
                    for (int j = 0; j < 4; j++) f[j] = bf16 ? pack2<false>(__uint_as_float(v[j] << 16) * to, __uint_as_float(v[j] & 0xffff0000u) * to) : v[j];
                    st_smem16(q_at + (x * (D / 32) + i) * 512, make_uint4(f[0], f[1], f[2], f[3]));
                }
#pragma unroll
                for (int i = 0; i < 2; i++)  // so small a one weighs all alike, and a hidden score, -inf, stays that in the product with it
                    c[x][i] = fminf(fmaxf(p.o.c * __shfl_sync(0xffffffffu, back, (2 * t + i) * 4), 0x1p-120f), 0x1p127f);
            }
#pragma unroll
            for (int x = 0; x < NT; x++) {
#pragma unroll
                for (int i = 0; i < D / 16; i++)
#pragma unroll
                    for (int j = 0; j < 4; j++) o[i][x][j] = 0.0f;
                m[x][0] = m[x][1] = kNothing;
                l[x][0] = l[x][1] = 0.0f;
            }
            // where this thread's codes and scales lie in a tile; scales of heads that come apart begin off a 16-byte boundary
            const auto rest = [&](int dim) { return H ? 0 : (p.heads_all * dim / 2 + head0 * dim / 16) & 15; };
            const uint32_t k_at = ring + (g0 + rk) * k_row + h * dk / 2 + t * (D / 8);
            const uint32_t y_at = ring + (H ? H * D / 2 : p.kl.first) + (g0 + rk) * y_row + rest(dk) + h * dk / 16 + (D == 128 ? 2 * t : t);
            const uint32_t va_at = v_ring + (g0 + ra) * v_row + h * dv / 2 + n * (D / 16), vb_at = va_at + (rb - ra) * v_row;
            const uint32_t xa_at = v_ring + (H ? H * D / 2 : p.vl.first) + (g0 + ra) * x_row + rest(dv) + h * dv / 16 + (D == 128 ? n : n / 2);
            const uint32_t xb_at = xa_at + (rb - ra) * x_row;
            const int tiles = w.n, key0 = (w.u.tile0 + w.at.off) << b.tile_shift, seen_lo = w.u.lo, seen_hi = w.u.hi;
            int clean_lo, clean_hi, other;  // keys that every row sees
            sees(b, w.q, (int)fdiv((uint32_t)(w.u.row0 + rows - 1), b.group), clean_lo, other);
            sees(b, w.q, (int)fdiv((uint32_t)w.u.row0, b.group), other, clean_hi);
            // One tile; Hide: some row does not see all of it.
            const auto work = [&](auto hide, int kb) {
                constexpr bool kHide = decltype(hide)::value;
                const auto unseen = [&](int key) { return key < seen_lo || key >= seen_hi; };
                if (!wait.warp(smem_addr(&aux.k_full[s]), phase)) return false;
                // ---- scores: S^T of 16 keys by 8 rows a step ----
                const uint32_t kp = k_at + s * k_tile, yp = y_at + s * k_tile;
                float sc[F::kSteps][NT][4];
                uint32_t w0[F::kSteps][D / 32], w1[F::kSteps][D / 32], u0[F::kSteps], u1[F::kSteps];
#pragma unroll
                for (int step = 0; step < F::kSteps; step++) {
#pragma unroll
                    for (int x = 0; x < NT; x++)
#pragma unroll
                        for (int j = 0; j < 4; j++) sc[step][x][j] = 0.0f;
                    const uint32_t r0 = kp + step * 16 * split * k_row, r1 = r0 + 8 * k_row;
                    const uint32_t y0 = yp + step * 16 * split * y_row, y1 = y0 + 8 * y_row;
                    if (D == 128) {
                        const uint4 a = ld_smem16(r0), d = ld_smem16(r1);
                        w0[step][0] = a.x, w0[step][1] = a.y, w0[step][D / 32 - 2] = a.z, w0[step][D / 32 - 1] = a.w;
                        w1[step][0] = d.x, w1[step][1] = d.y, w1[step][D / 32 - 2] = d.z, w1[step][D / 32 - 1] = d.w;
                        u0[step] = ld_smem2(y0), u1[step] = ld_smem2(y1);
                    } else {
                        const uint2 a = ld_smem8(r0), d = ld_smem8(r1);
                        w0[step][0] = a.x, w0[step][1] = a.y, w1[step][0] = d.x, w1[step][1] = d.y;
                        u0[step] = ld_smem1(y0), u1[step] = ld_smem1(y1);
                    }
                    if (!H) u0[step] &= k_mask, u1[step] &= k_mask;
                    if (kHide) {  // what no row sees counts as zeros: it may hold anything
                        const int key = kb + (int)(g0 + 16 * split * step + rk);
                        if (unseen(key)) u0[step] = 0;
                        if (unseen(key + 8)) u1[step] = 0;
                    }
                    u0[step] = e4m3x2_to_f16(u0[step]), u1[step] = e4m3x2_to_f16(u1[step]);
                }
#pragma unroll
                for (int i = 0; i < D / 32; i++) {
                    uint4 q[NT];
#pragma unroll
                    for (int x = 0; x < NT; x++) q[x] = ld_smem16(q_at + (x * (D / 32) + i) * 512);
#pragma unroll
                    for (int step = 0; step < F::kSteps; step++) {
                        const uint32_t z0 = prmt(u0[step], u0[step], i < 2 ? 0x1010 : 0x3232), z1 = prmt(u1[step], u1[step], i < 2 ? 0x1010 : 0x3232);
                        uint32_t a[4], d[4];
                        q4_to_f16(w0[step][i], a);
                        q4_to_f16(w1[step][i], d);
#pragma unroll
                        for (int j = 0; j < 4; j++) a[j] = mul_f16x2(a[j], z0), d[j] = mul_f16x2(d[j], z1);
#pragma unroll
                        for (int x = 0; x < NT; x++) {
                            mma16816(sc[step][x], a[0], d[0], a[1], d[1], q[x].x, q[x].y);
                            mma16816(sc[step][x], a[2], d[2], a[3], d[3], q[x].z, q[x].w);
                        }
                    }
                }
                warp_arrive(smem_addr(&aux.k_empty[s]));
                // ---- weights ----
                if (kHide) {
#pragma unroll
                    for (int x = 0; x < NT; x++)
#pragma unroll
                        for (int i = 0; i < 2; i++) {
                            int lo, hi;
                            sees(b, w.q, (int)fdiv((uint32_t)(w.u.row0 + min(8 * x + 2 * t + i, rows - 1)), b.group), lo, hi);
#pragma unroll
                            for (int step = 0; step < F::kSteps; step++)
#pragma unroll
                                for (int j = 0; j < 2; j++) {
                                    const int key = kb + (int)(g0 + 16 * split * step + rk) + 8 * j;
                                    if (key < lo || key >= hi) sc[step][x][i + 2 * j] = -INFINITY;
                                }
                        }
                }
                bool grow = false;
                float top[NT][2];
#pragma unroll
                for (int x = 0; x < NT; x++)
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        float v = -INFINITY;
#pragma unroll
                        for (int step = 0; step < F::kSteps; step++) v = fmaxf(v, fmaxf(sc[step][x][i], sc[step][x][i + 2]));
                        top[x][i] = v;
                        grow |= (v - m[x][i]) * c[x][i] > 8.0f;
                    }
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int x = 0; x < NT; x++)
#pragma unroll
                        for (int i = 0; i < 2; i++) {
                            float v = top[x][i];
#pragma unroll
                            for (int d = 4; d < 32; d *= 2) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
                            const float now = fmaxf(m[x][i], v);
                            const float a = exp2_fast((m[x][i] - now) * c[x][i]);
                            m[x][i] = now;
                            l[x][i] *= a;
#pragma unroll
                            for (int k = 0; k < D / 16; k++) o[k][x][i] *= a, o[k][x][i + 2] *= a;
                        }
                }
                uint32_t pf[F::kSteps][NT][2];
#pragma unroll
                for (int x = 0; x < NT; x++) {
                    const float2 off = make_float2(-m[x][0], -m[x][1]), cc = make_float2(c[x][0], c[x][1]), seven = make_float2(7.0f, 7.0f);
#pragma unroll
                    for (int step = 0; step < F::kSteps; step++) {
                        float e[4];
#pragma unroll
                        for (int j = 0; j < 4; j += 2) {
                            const float2 z = fma2(add2(make_float2(sc[step][x][j], sc[step][x][j + 1]), off), cc, seven);
                            e[j] = exp2_fast(z.x), e[j + 1] = exp2_fast(z.y);
                            l[x][0] += e[j], l[x][1] += e[j + 1];
                        }
                        pf[step][x][0] = transposed8(pack2<false>(e[0], e[1]));
                        pf[step][x][1] = transposed8(pack2<false>(e[2], e[3]));
                    }
                }
                // ---- values: O^T of 16 dimensions by 8 rows a product ----
                if (!wait.warp(smem_addr(&aux.v_full[s]), phase)) return false;
                const uint32_t vp[2] = {va_at + s * v_tile, vb_at + s * v_tile}, xp[2] = {xa_at + s * v_tile, xb_at + s * v_tile};
#pragma unroll
                for (int step = 0; step < F::kSteps; step++) {
                    uint32_t cw[4][D / 64], unit[4];
#pragma unroll
                    for (int j = 0; j < 4; j++) {  // keys 2 t, 2 t + 1 and those eight further on
                        const uint32_t at = vp[j & 1] + (step * 16 * split + (j >> 1) * 8) * v_row;
                        if (D == 128) {
                            const uint2 x = ld_smem8(at);
                            cw[j][0] = x.x, cw[j][D / 64 - 1] = x.y;
                        } else {
                            cw[j][0] = ld_smem4(at);
                        }
                        unit[j] = ld_smem1(xp[j & 1] + (step * 16 * split + (j >> 1) * 8) * x_row);
                        if (!H) unit[j] &= v_mask;
                        if (kHide && unseen(kb + (int)(g0 + 16 * split * step + (j & 1 ? rb : ra) + 8 * (j >> 1)))) unit[j] = 0;
                    }
                    const uint32_t z0 = e4m3x2_to_f16(unit[0] | unit[1] << 8), z1 = e4m3x2_to_f16(unit[2] | unit[3] << 8);
#pragma unroll
                    for (int i = 0; i < D / 64; i++) {
                        // two keys' codes side by side: the even dimensions' and the odd ones'
                        uint32_t a0[4], a1[4], a2[4], a3[4];
                        q4_to_f16((cw[0][i] & 0x0f0f0f0fu) | (cw[1][i] << 4 & 0xf0f0f0f0u), a0);
                        q4_to_f16((cw[0][i] >> 4 & 0x0f0f0f0fu) | (cw[1][i] & 0xf0f0f0f0u), a1);
                        q4_to_f16((cw[2][i] & 0x0f0f0f0fu) | (cw[3][i] << 4 & 0xf0f0f0f0u), a2);
                        q4_to_f16((cw[2][i] >> 4 & 0x0f0f0f0fu) | (cw[3][i] & 0xf0f0f0f0u), a3);
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            a0[j] = mul_f16x2(a0[j], z0), a1[j] = mul_f16x2(a1[j], z0), a2[j] = mul_f16x2(a2[j], z1), a3[j] = mul_f16x2(a3[j], z1);
#pragma unroll
                            for (int x = 0; x < NT; x++) mma16816(o[4 * i + j][x], a0[j], a1[j], a2[j], a3[j], pf[step][x][0], pf[step][x][1]);
                        }
                    }
                }
                warp_arrive(smem_addr(&aux.v_empty[s]));
                return true;
            };
            for (int tile = 0; ok && tile < tiles; tile++) {
                const int kb = key0 + tile * tile_keys;
                if (kb < clean_lo || kb + tile_keys > clean_hi)
                    ok = work(std::true_type(), kb);
                else
                    ok = work(std::false_type(), kb);
                if (++s == p.slots) s = 0, phase ^= 1;
            }
            if (!ok) break;
#pragma unroll
            for (int x = 0; x < NT; x++)
#pragma unroll
                for (int i = 0; i < 2; i++)
#pragma unroll
                    for (int d = 4; d < 32; d *= 2) l[x][i] += __shfl_xor_sync(0xffffffffu, l[x][i], d);
            // ---- the warps of a head join, the upper half of them to the lower one and so on; who has left its sums goes on.  Of the
            // head's split / 2 places warp j reads place j in the first round, and leaves its own sums there in a later one ----
            bool gone = false;
#pragma unroll 1
            for (int half = split / 2; half > 0 && !gone; half /= 2) {
                const bool first_round = half == split / 2;
                gone = part >= half;
                const int j = first_round ? part & (half - 1) : gone ? part : part + half, place = h * (split / 2) + j;
                float *const at = joins + place * Sums<D, NT>::kShared;
                const uint32_t full = smem_addr(first_round ? &aux.join_first[place] : &aux.join_full[place]);
                if (gone) {
                    if (first_round && joined && !wait.warp(smem_addr(&aux.join_free[place]), (joined - 1) & 1)) ok = false;
                    if (!ok) break;
                    sums.template store<true>(at, rows);
                    warp_arrive(full);
                } else {
                    if (!wait.warp(full, joined & 1)) ok = false;
                    if (!ok) break;
                    sums.join(at, rows, c);
                    if (!first_round || part == 0) warp_arrive(smem_addr(&aux.join_free[place]));
                }
            }
            joined++;
            if (!ok) break;
            if (gone) continue;
#pragma unroll
            for (int x = 0; x < NT; x++)
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    // in units of the call's scale from here on.  (The thread's numbers anew: kept in registers over the tiles they spill, and the
                    // long decode batch takes 6 us more.)
                    const uint32_t e = aux.size[(threadIdx.x >> 5) - F::kLoaders][8 * x + 2 * (threadIdx.x & 3) + i];
                    m[x][i] = l[x][i] > 0.0f ? m[x][i] * __uint_as_float(e << 23) : -INFINITY;
                }
            if (!w.whole()) {
                // the last of the CTA's heads to be in the workspace counts the piece; who counts the last one joins them all in the end
                const Cut cut(line, w.pos - w.at.off, unit_cost(w.u));
                sums.template store<false>(p.ws + (int64_t)cut.slot(cut.nth) * (256 * 130) + h * Sums<D, NT>::kFloats, rows);
                CutUnit &mine = aux.cut[cut.nth == 0];
                __threadfence();
                __syncwarp();
                if (lane == 0) {
                    if (h == 0) {
                        mine.c0 = cut.c0, mine.count = cut.count, mine.nth = cut.nth, mine.head0 = head0;
                        mine.rows = HeadRows{w.u.row0, rows, w.q.q0};
                    }
                    if (atomicAdd(&mine.stored, 1) == heads - 1) {
                        __threadfence();
                        const int each = group_of(cut.count), groups = cut.count > kMany ? cut.count / each : 1, group = min(cut.nth / each, groups - 1);
                        const int count = groups == 1 ? cut.count : group + 1 < groups ? each : cut.count - group * each;
                        mine.last = count_in(p.counters + 2 * (cut.c0 + (groups > 1 ? 1 + group : 0)), count);
                    }
                }
                continue;
            }
#pragma unroll
            for (int x = 0; x < NT; x++)
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    const int r = 8 * x + 2 * t + i;
                    if (r >= rows) continue;
                    float *lse;
                    char *const to = row_out(p, HeadRows{w.u.row0, rows, w.q.q0}, (head0 + h) * (int)b.group.d, r, lse);
                    const float inv = l[x][i] > 0.0f ? p.v_scale / l[x][i] : 0.0f;
                    uint32_t z[D / 16];
#pragma unroll
                    for (int k = 0; k < D / 16; k++) z[k] = pack_out(p, o[k][x][i] * inv, o[k][x][i + 2] * inv);
#pragma unroll
                    for (int k = 0; k < D / 64; k++)
                        if (n * (D / 8) < dv) reinterpret_cast<uint4 *>(to)[n * (D / 64) + k] = make_uint4(z[4 * k], z[4 * k + 1], z[4 * k + 2], z[4 * k + 3]);
                    if (n == 0 && lse) *lse = lse_of(p, m[x][i], l[x][i]);
                }
        } while (next_unit());
        // ---- cut units: the CTA that brought the last piece joins them, in the order of the keys; of many pieces the last of every
        // group adds those up first.  Done when the CTA has nothing else to do, by all its warps ----
        int syncs = 0;
        const auto sync_all = [&] {
            warp_arrive(smem_addr(&aux.sync));
            return wait.warp(smem_addr(&aux.sync), syncs++ & 1);
        };
        if (ok && sync_all()) {
#pragma unroll 1
            for (int f = 0; f < 2; f++) {
                const CutUnit &c = aux.cut[f];
                if (!c.last) continue;
                const int each = group_of(c.count), groups = c.count > kMany ? c.count / each : 1, group = min(c.nth / each, groups - 1);
                bool sum = groups > 1;
#pragma unroll 1
                for (;; sum = false) {
                    const bool of_sums = groups > 1 && !sum;
                    const int from = sum ? group * each : 0, count = groups == 1 ? c.count : of_sums ? groups : group + 1 < groups ? each : c.count - from;
                    join_pieces<D, NT>(p, c, h, from, of_sums ? each : 0, count, sum, part * 32 + lane, split * 32);
                    if (!sum) break;
                    __threadfence();
                    if (!sync_all()) break;
                    if (me == 0 && lane == 0) aux.cut[f].last = count_in(p.counters + 2 * c.c0, groups);
                    if (!sync_all() || !c.last) break;
                }
            }
        }
    }
    // common exit
    __syncwarp();
    __syncthreads();
    if (aux.gave_up) {  // let copies in flight land before the shared memory is given back
        const unsigned long long t0 = now_ns();
        while (now_ns() - t0 < 10000000ull) {}
    }
}

// dev: null to prepare the kernel.
template <int D, int NT, int H>
int launch_kernel(FewParams p, const DeviceInfo *dev, cudaStream_t s)
{
    using F = Few<D, NT, H>;
    const auto kernel = attention_q4_few_kernel<D, NT, H>;
    constexpr uint32_t kFixed = ((sizeof(Aux) + 127) & ~127u) + F::kWarps * F::kQ, kAll = 227 * 1024;
    if (dev == nullptr) {
        const int st = cuda_status(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kAll));
        return st != KV_OK ? st : load_kernels(kernel);
    }
    const int all = p.heads_all, heads = p.unit_heads;
    // A run of rows ends on a multiple of 128 bytes, where a TMA may begin; its rows lie 32 or 96 bytes off one where that allows it.
    const auto pitch = [&](int bytes) {
        const int step = p.piece_rows >= 4 ? 64 : 128 / p.piece_rows, off = p.piece_rows >= 4 ? 32 : 0;
        return (bytes - off + step - 1) / step * step + off;
    };
    const auto place = [&](const Q4Plane &plane) {
        Place4 l = {};
        const int codes = heads * plane.dim / 2, row = plane.desc->row_bytes;
        l.apart = heads < all;
        l.dense = dense_rows(p, plane);
        l.base = plane.base;
        l.block_stride = plane.desc->block_stride;
        if (l.apart) {
            l.codes = pitch(codes);
            l.scales = pitch((heads * plane.dim / 16 + 14 + 15) / 16 * 16);
            l.first = p.tile * l.codes;
            l.bytes = p.tile * (l.codes + l.scales);
        } else {
            l.codes = l.scales = l.dense ? row : pitch(row);
            l.first = codes;
            l.bytes = p.tile * l.codes;
        }
        return l;
    };
    uint32_t pair, join;
    const auto fit = [&] {
        p.tile = 16 * p.split * F::kSteps;
        p.piece_rows = piece_rows(p.k.desc->block_size, p.tile < 256 ? p.tile : 256);
        p.kl = place(p.k);
        p.vl = place(p.v);
        pair = (uint32_t)(p.kl.bytes + p.vl.bytes), join = ((uint32_t)(heads * p.split / 2) * Sums<D, NT>::kShared * 4 + 127) & ~127u;
        p.slots = (int)((kAll - kFixed - join - 128) / pair);
    };
    fit();
    // One head of several in pages of an odd size (key heads in a prime number): codes and scales of single rows take 128 bytes each, and the
    // 512 keys of all warps 256 KB.  Half of the warps then.
    while (!H && p.slots < 1 && p.split > 1) p.split /= 2, fit();
    p.order = order_of(p.kl.codes);
    if (p.slots > kMaxSlots) p.slots = kMaxSlots;
    if (p.slots < 1 || dev->num_sms * 2 * 4 > kCounterBytes) return KV_ERR_UNSUPPORTED;
    CUtensorMap map[4];
    int st;
    if ((st = make_row_map(&map[0], p.k.base, p.k.desc, p.kl.codes, p.piece_rows)) != KV_OK) return st;
    if ((st = make_row_map(&map[1], p.v.base, p.v.desc, p.vl.codes, p.piece_rows)) != KV_OK) return st;
    map[2] = map[0], map[3] = map[1];
    if (heads < all && ((st = make_row_map(&map[2], p.k.base, p.k.desc, p.kl.scales, p.piece_rows)) != KV_OK ||
                        (st = make_row_map(&map[3], p.v.base, p.v.desc, p.vl.scales, p.piece_rows)) != KV_OK))
        return st;
    p.b.kv_heads = all / heads;
    p.b.tile_shift = 0;
    while ((1 << p.b.tile_shift) < p.tile) p.b.tile_shift++;
    const uint32_t bytes = kFixed + join + 128 + p.slots * pair;
    return cuda_status(launch(kernel, dim3(dev->num_sms), dim3(F::kThreads), bytes, s, map[0], map[1], map[2], map[3], p));
}

// dev: null to prepare the kernels.
template <int D, int NT>
int launch_few(FewParams &p, const DeviceInfo *dev, cudaStream_t s)
{
    constexpr int kWarps = Few<D, NT, 0>::kWarps;
    // by the logarithm of the heads; those of 8 warps end at 8
    int (*const full[])(FewParams, const DeviceInfo *, cudaStream_t) = {launch_kernel<D, NT, 1>, launch_kernel<D, NT, 2>, launch_kernel<D, NT, 4>,
                                                                       launch_kernel<D, NT, 8>, kWarps > 8 ? launch_kernel<D, NT, kWarps> : nullptr};
    if (dev == nullptr) {
        int st = launch_kernel<D, NT, 0>(p, dev, s);
        for (int i = 0; st == KV_OK && i < 5 && full[i]; i++) st = full[i](p, dev, s);
        return st;
    }
    const int all = p.heads_all;
    int heads = all < kWarps ? all : kWarps;
    while (all % heads) heads--;
    // A unit of few heads lies in fewer pieces, of fewer bytes, when many CTAs share a request: joining them is bound by what one SM reads
    // (45 GB/s).  But rows that come apart into heads cost more to load, so that this pays for short contexts only.  8 key heads of 128
    // and a unit of 8, 4, 2 of them, one request of 120000 and of 8000: 12 rows 72, 61, 56 and 40, 26, 21 us; 8 rows 52, 49, 49 and 29, 22, 20
    // us; eight requests of 15000: 61, 60, 66 and 46, 51, 62; 64 requests of 8000: 12 rows 150, 198, 263, 4 rows 110, 176, 248.
    // The lengths are on the device, so the table's width stands for them: two requests of 8000, 12 rows, take 21 us, under a table for 128000 41.
    constexpr int kPieces = NT == 1 ? 40 : 10;            // of a unit, above which it gets fewer heads
    constexpr int64_t kShort = NT == 1 ? 6144 : 10240;    // keys times heads an SM, up to which (where the two would meet for one request)
    const int64_t seen = p.b.window ? std::min<int64_t>(p.b.max_tokens, (int64_t)p.b.window + p.b.n_tokens) : p.b.max_tokens;
    if (p.b.n_reqs * seen * all <= kShort * dev->num_sms)
        while ((int64_t)dev->num_sms * heads > (int64_t)kPieces * p.b.n_reqs * all) {
            int h = heads - 1;
            while (h > 1 && all % h) h--;
            if (h < 2) break;
            heads = h;
        }
    p.unit_heads = heads;
    p.split = 1;
    while (2 * p.split * heads <= kWarps) p.split *= 2;
    int at = 0;
    while (1 << at < heads) at++;
    // runs of rows as long as the shortest tile allows, in every page
    p.piece_rows = piece_rows(p.k.desc->block_size, 16 * p.split);
    return 1 << at == heads && p.k.dim == D && p.v.dim == D && dense_rows(p, p.k) && dense_rows(p, p.v) ? full[at](p, dev, s)
                                                                                                        : launch_kernel<D, NT, 0>(p, dev, s);
}

}  // namespace

}  // namespace pkv
