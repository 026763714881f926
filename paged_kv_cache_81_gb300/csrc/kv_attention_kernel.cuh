// The kernel of kv_attention and, with rows of another kind than 16-bit ones, of kv_attention_q4: see kv_attention.cu.
#pragma once

#include <cmath>
#include <type_traits>

#include "kv_attention.cuh"

namespace pkv {

namespace {

constexpr int kLeast = 4;  // tiles of a piece of a unit, at least (a join costs as much as three or four more tiles: 3 to 5 us)
constexpr int kThreads = 384, kRowsThreads = 512;
constexpr int kRows = 256;  // rows of a unit, at most: 2 * floor(128 / group) tokens of a group
constexpr int kTileShift = 7, kTile = 1 << kTileShift;  // keys of a tile
constexpr uint32_t kPanel = 128 * 128;  // bytes of a 64-element panel of 128 rows

// Staged: with room for packed rows.
template <int DK, int DV, bool Staged = false>
struct Shape {
    static constexpr uint32_t kQ = 128 * DK * 2, kK = 128 * DK * 2, kV = 128 * DV * 2;
    static constexpr int kNK = Staged ? 2 : DK == 64 ? 5 : DK == 128 ? 3 : 2;  // ring depths: what 227 KB holds
    static constexpr int kNV = Staged ? 2 : DK == 64 ? 5 : DK == 128 ? 2 : 1;  // (192: four single panels of K and two tiles of V ran 7% slower)
    static constexpr uint32_t kOffK = 2 * kQ, kOffV = kOffK + kNK * kK, kOffAux = kOffV + kNV * kV;
    static constexpr uint32_t kOffScales = kOffAux + 2048;  // where Staged: the queries' exponents of two units, a byte a row
    static constexpr uint32_t kBytes = kOffScales + (Staged ? 512 : 0);
    static constexpr uint32_t kOffStage = kBytes, kStage = 227 * 1024 - kOffStage;  // where Staged
};

struct AttentionParams {
    Batch b;
    const int32_t *table;
    int64_t table_stride;
    int32_t num_blocks;  // pages that both caches have
    int32_t no_page;     // a page that neither has: its loads bring zeros
    FastDiv block;       // slots of a page
    int32_t piece_rows;  // slots one TMA brings: gcd(block, 128), so it never leaves a page
    int32_t q_box;       // tokens one TMA brings of q
    Output o;
    float *ws;
    int *counters;
};

// Keys and values of another kind than 16-bit rows: their packed rows come by TMA into a stage of `stages` slots, keys and values in
// turn, and four warps more make tiles of them.
template <typename Rows>
struct RowsParams : AttentionParams {
    Rows k, v;
    int32_t stages;
};
struct NoRows {};
template <typename Rows>
using KernelParams = std::conditional_t<std::is_same_v<Rows, NoRows>, AttentionParams, RowsParams<Rows>>;

// Bookkeeping at the end of shared memory.
struct Aux {
    uint64_t k_full[5], k_empty[5], v_full[5], v_empty[5], stage_full[4], stage_empty[4];
    uint64_t s_full[2], p_ready[2], o_done[2], q_full, q_ready[2], q_empty, merge_ready, merge_free, join[2];
    int scan[64];
    Place place;
    float m[128], l[128];  // the odd tiles' group, for the join
    uint32_t tmem;
    int answer[2];
    int gave_up;
};
static_assert(sizeof(Aux) <= 2048, "bookkeeping");

// Which runs of 32 keys of the tile that begins at key kb some row of the unit sees: [from, to).
__device__ __forceinline__ int seen_from(const Unit &u, int kb) { return max(0, u.lo - kb) >> 5; }
__device__ __forceinline__ int seen_to(const Unit &u, int kb) { return (min(u.hi - kb, kTile) + 31) >> 5; }

// One tile of K or V rows into its slot: a TMA per (run of slots inside a page, panel), spread over the
// lanes.  The first page a lane needs is looked up before `ready` waits for the slot.
template <int Panels, typename Ready>
__device__ __forceinline__ bool load_tile(const AttentionParams &p, const CUtensorMap *map, const int32_t *row, int kb, int lo, int hi, int head,
                                          uint32_t to, uint32_t bar, const Ready &ready)
{
    const int lane = threadIdx.x & 31, pr = p.piece_rows;
    const int p0 = max(0, lo - kb) / pr, p1 = (min(hi - kb, kTile) + pr - 1) / pr;
    int page = 0, slot = 0;
    const auto find = [&](int i) {
        const uint32_t key = (uint32_t)(kb + i * pr), col = fdiv(key, p.block);
        slot = (int)(key - col * p.block.d);
        page = __ldg(row + col);
        if (page < 0 || page >= p.num_blocks) {
            set_error(p.b.err, KV_DERR_TABLE);
            page = p.no_page;
        }
    };
    if (p0 + lane < p1) find(p0 + lane);
    if (!ready()) return false;
    if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)((p1 - p0) * pr) * Panels * 128);
    __syncwarp();
    for (int i = p0 + lane; i < p1; i += 32) {
        if (i >= p0 + 32) find(i);
#pragma unroll
        for (int h = 0; h < Panels; h++) tma_load_4d(to + h * kPanel + i * pr * 128, map, bar, h * 64, head, slot, page);
    }
    __syncwarp();
    return true;
}

// Row `thread` of a set of bf16 queries in shared memory to fp16, brought to [1, 2) by a power of two: returns its exponent.
template <int DK>
__device__ __forceinline__ uint32_t scale_row(uint32_t set, int thread)
{
    const auto at = [&](int c) { return set + (c >> 3) * kPanel + thread * 128 + (((c & 7) ^ (thread & 7)) << 4); };
    uint32_t most = 0;  // magnitudes, two by two
#pragma unroll 4
    for (int c = 0; c < DK / 8; c++) {
        const uint4 v = ld_smem16(at(c));
        most = __vmaxu2(most, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
    }
    const uint32_t e = min(max(max(most & 0xffffu, most >> 16) >> 7, 1u), 253u);
    const float to = __uint_as_float((254u - e) << 23);
#pragma unroll 2
    for (int c = 0; c < DK / 8; c++) {
        const uint4 v = ld_smem16(at(c));
        const auto f16 = [&](uint32_t x) { return pack2<false>(__uint_as_float(x << 16) * to, __uint_as_float(x & 0xffff0000u) * to); };
        st_smem16(at(c), make_uint4(f16(v.x), f16(v.y), f16(v.z), f16(v.w)));
    }
    return e;
}

// Weights of 32 scores as weights32 gives them in fp16, the reference m (0 for none) taken off before the product: 2^(c (s - m) + 7), right at any
// size of s.  weights32 rounds c m - 7 by itself, upwards: weights of different references do not agree then (by 2% at 2^19), and at
// 2^29 every one is lost.
__device__ __forceinline__ void weights32_at_any_size(const uint32_t (&x)[32], float c, float m, float2 (&sum)[2], uint32_t (&pk)[16])
{
    const float2 cc = make_float2(c, c), nn = make_float2(-m, -m), seven = make_float2(7.0f, 7.0f);
#pragma unroll
    for (int i = 0; i < 16; i++) {
        float2 e = fma2(add2(make_float2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), nn), cc, seven);
        e.x = exp2_fast(e.x);
        e.y = exp2_fast(e.y);
        sum[i & 1] = add2(sum[i & 1], e);
        pk[i] = pack2<false>(e.x, e.y);
    }
}

// A unit's queries, `half` rows at `base` and the others at its second panel set, by one warp.
template <int DK>
__device__ __forceinline__ void load_queries(const AttentionParams &p, const CUtensorMap *map, const Walk &w, int half, uint32_t base, uint32_t bar)
{
    const int lane = threadIdx.x & 31;
    const int group = (int)p.b.group.d, tok0 = (int)fdiv((uint32_t)w.u.row0, p.b.group), toks = w.u.rows / group, per_half = half / group;
    // boxes of q_box tokens; a box that begins in the first half ends there
    const int n0 = (min(toks, per_half) + p.q_box - 1) / p.q_box, n1 = toks > per_half ? (toks - per_half + p.q_box - 1) / p.q_box : 0;
    if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)((n0 + n1) * p.q_box * group) * DK * 2);
    __syncwarp();
    for (int i = lane; i < n0 + n1; i += 32) {
        const int g = i >= n0, t = (i - (g ? n0 : 0)) * p.q_box;
#pragma unroll
        for (int h = 0; h < DK / 64; h++)
            tma_load_3d(base + g * Shape<DK, DK>::kQ + h * kPanel + t * group * 128, map, bar, h * 64, w.at.head * group, w.q.q0 + tok0 + g * per_half + t);
    }
    __syncwarp();
}

// Rows: NoRows where tiles of K and V come by TMA.  Otherwise rows of another kind: warps 0 and 2 load them packed (k_scale_map, v_scale_map
// are for them alone), and warps 12 to 15 make the tiles.  Those 512 threads have 128 registers each; the softmax groups take
// 168, the others give theirs away, and as no function can be called then, PKV_APART has to be inline.  Tiles are fp16 ones; bf16 queries
// are brought to fp16 by warps 12 to 15 too, with a power of two a row that the row's softmax takes into its scale.
template <int DK, int DV, bool Bf16, typename Rows>
__global__ void __launch_bounds__(std::is_same_v<Rows, NoRows> ? kThreads : kRowsThreads, 1)
attention_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                 const __grid_constant__ CUtensorMap v_map, const __grid_constant__ KernelParams<Rows> p)
{
    constexpr bool kRowsKind = !std::is_same_v<Rows, NoRows>;
    constexpr int kFull = kRowsKind ? 4 : 1;  // arrivals that fill a tile
    constexpr bool kScaled = kRowsKind && Bf16;    // queries are brought to fp16, as the tiles are: 4-bit codes times their scales are exact in it
    constexpr bool kBfMath = Bf16 && !kScaled;     // the products' type
    using S = Shape<DK, DV, kRowsKind>;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t base = smem_addr(smem);
    Aux &aux = *reinterpret_cast<Aux *>(smem + S::kOffAux);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const Batch &b = p.b;
    const Waiter wait{&aux.gave_up, b.err};

    if (tid == 0) {
        aux.gave_up = 0;
        for (int i = 0; i < S::kNK; i++) mbar_init(smem_addr(&aux.k_full[i]), kFull), mbar_init(smem_addr(&aux.k_empty[i]), 1);
        for (int i = 0; i < S::kNV; i++) mbar_init(smem_addr(&aux.v_full[i]), kFull), mbar_init(smem_addr(&aux.v_empty[i]), 1);
        for (int i = 0; i < 2; i++) {
            mbar_init(smem_addr(&aux.s_full[i]), 1);
            mbar_init(smem_addr(&aux.p_ready[i]), 4);
            mbar_init(smem_addr(&aux.o_done[i]), 1);
            mbar_init(smem_addr(&aux.join[i]), 4);
            mbar_init(smem_addr(&aux.q_ready[i]), 4);
        }
        if (kRowsKind)
            for (int i = 0; i < 4; i++) mbar_init(smem_addr(&aux.stage_full[i]), 1), mbar_init(smem_addr(&aux.stage_empty[i]), 4);
        mbar_init(smem_addr(&aux.q_full), 1);
        mbar_init(smem_addr(&aux.q_empty), 1);
        mbar_init(smem_addr(&aux.merge_ready), 4);
        mbar_init(smem_addr(&aux.merge_free), 4);
        mbar_init_fence();
        tma_prefetch_map(&q_map);
        tma_prefetch_map(&k_map);
        tma_prefetch_map(&v_map);
    }
    if (warp == 3) tmem_alloc(smem_addr(&aux.tmem), 512);
    grid_dep_entry();
    const Line line = find_place<kRowsKind ? kRowsThreads : kThreads>(b, blockIdx.x, gridDim.x, kLeast, aux.scan, &aux.place, blockIdx.x == 0);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, aux.tmem, 0);
    const int half = b.unit_rows / 2;  // rows of a softmax group
    Walk w;
    const bool any = w.start(b, aux.place, line);
    if (!any) {
        // nothing to do: on to the common exit
    } else if (warp >= 4 && warp < 12) {
        if (kRowsKind) asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
        // ---- softmax: group g, a thread per row ----
        const int g = (warp - 4) >> 2, t = tid & 127;
        const uint32_t mine = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_at = tmem + g * 128 + mine, o_at = tmem + 256 + g * 128 + mine;
        float c = p.o.c, slack = 8.0f / c;  // log2 of a weight a unit of the scores; how far the maximum may grow before O is rescaled
        int steps = 0, joins = 0, cuts = 0, units = 0;
        bool owes_free = false;  // the even group may still be reading this (odd) group's O
        bool ok = true;
        do {
            const bool both = w.u.rows > half;
            const int row = (both ? g * half : 0) + t;         // row of the unit
            const bool live = t < half && row < w.u.rows;
            // where the row's output and its lse go (asked for after the key tiles: held over them it would spill)
            const auto place = [&](float *&lse) {
                const int r = w.u.row0 + row, tok = (int)fdiv((uint32_t)r, b.group), head = w.at.head * (int)b.group.d + r - tok * (int)b.group.d;
                const int64_t token = w.q.q0 + tok;
                lse = p.o.lse ? p.o.lse + token * p.o.heads + head : nullptr;
                return p.o.out + token * p.o.out_token + (int64_t)head * p.o.out_head;
            };
            if (w.u.tiles == 0) {  // nothing is seen
                if (live && (both || g == 0)) {
                    float *lse;
                    char *to = place(lse);
                    for (int col = 0; col < p.o.dv; col += 8) *reinterpret_cast<uint4 *>(to + col * 2) = make_uint4(0, 0, 0, 0);
                    if (lse) *lse = -INFINITY;
                }
                continue;
            }
            // key tiles; spare rows see what the last one does
            int lo, hi;
            sees(b, w.q, (int)fdiv((uint32_t)(w.u.row0 + min(row, w.u.rows - 1)), b.group), lo, hi);
            const bool warp_live = __any_sync(0xffffffffu, live);
            float m = -INFINITY, l = 0.0f, back = 1.0f;
            const int first = both ? 0 : g, step = both ? 1 : 2, kt0 = w.u.tile0 + w.at.off;
            if (kScaled) {  // the row's own unit
                // Only a group with a step in the unit waits: its weights hold the products back from the unit after, whose last one
                // lets the queries of the one after that complete this barrier again.  The odd group of a unit of one tile holds
                // nothing back: late (joining a cut unit), it would find the barrier a phase further on and wait for good.
                if (first < w.n) {
                    if (!wait.warp(smem_addr(&aux.q_ready[units & 1]), units >> 1 & 1)) { ok = false; break; }
                    back = __uint_as_float((uint32_t)smem[S::kOffScales + (units & 1) * 256 + (both ? g * 128 : 0) + t] << 23);
                }
                units++;
                c = fminf(fmaxf(p.o.c * back, 0x1p-120f), 0x1p127f);  // so small a one weighs all alike, and leaves slack a number
                slack = 8.0f / c;
            }
            for (int k = first; k < w.n; k += step) {
                const int kb = (kt0 + k) * kTile;
                if (!wait.warp(smem_addr(&aux.s_full[g]), steps & 1)) { ok = false; break; }
                tc_fence_after();
                if (warp_live) {
                    // the maximum over all 128 scores.  A tile that some row sees in part (the first and last of a
                    // request, the diagonal) goes through a short loop (a call of one or two tiles a CTA is bound by
                    // fetching instructions), all others through straight code that reads 32 scores while it works
                    // on 32: more of them in registers at once would spill
                    const int from = lo - kb, to_key = hi - kb;
                    const bool hide = __any_sync(0xffffffffu, from > 0 || to_key < kTile);
                    uint32_t x0[32], x1[32];
                    float top;
                    if (hide) {
                        top = -INFINITY;
#pragma unroll 1
                        for (int q = seen_from(w.u, kb); q < seen_to(w.u, kb); q++) {
                            tmem_ld32(s_at + q * 32, x0);
                            tc_wait_ld();
                            hide32(x0, from - q * 32, to_key - q * 32);
                            top = max32(x0, top);
                        }
                    } else {
                        tmem_ld32(s_at, x0);
                        tc_wait_ld();
                        tmem_ld32(s_at + 32, x1);
                        top = max32(x0, -INFINITY);
                        tc_wait_ld();
                        tmem_ld32(s_at + 64, x0);
                        top = max32(x1, top);
                        tc_wait_ld();
                        tmem_ld32(s_at + 96, x1);
                        top = max32(x0, top);
                        tc_wait_ld();
                        top = max32(x1, top);
                    }
                    const bool grow = top > (kBfMath ? m + slack : __fadd_rd(m, slack));  // -inf + slack: the first finite score
                    if (__any_sync(0xffffffffu, grow)) {
                        const float to_m = grow ? top : m;
                        const float alpha = grow ? exp2_fast((m - to_m) * c) : 1.0f;
                        l *= alpha;
                        m = to_m;
                        if (k > first) {
                            if (!wait.warp(smem_addr(&aux.o_done[g]), (steps - 1) & 1)) { ok = false; break; }
                            tc_fence_after();
#pragma unroll 1
                            for (int q = 0; q < DV / 32; q++) {
                                uint32_t o[32];
                                tmem_ld32(o_at + q * 32, o);
                                tc_wait_ld();
#pragma unroll
                                for (int i = 0; i < 32; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                                tmem_st32(o_at + q * 32, o);
                            }
                        }
                    }
                    const float mc = weight_offset<kBfMath>(m, c);
                    // rows of another kind: large scores take the short loop, whose weights are right at any size.  Up to here the
                    // rounding of c m - 7 is a sixth of a weight's.
                    const bool short_loop = hide || (kRowsKind && __any_sync(0xffffffffu, fabsf(mc) > 0x1p10f));
                    float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                    uint32_t pk[16];
                    // P takes the columns of the upper 64 scores: 32 keys' weights stand in 16 columns from 64 on, so
                    // going down no score is overwritten before it has been read
                    if (short_loop) {
#pragma unroll 1
                        for (int q = seen_to(w.u, kb) - 1; q >= seen_from(w.u, kb); q--) {
                            tmem_ld32(s_at + q * 32, x0);
                            tc_wait_ld();
                            hide32(x0, from - q * 32, to_key - q * 32);
                            if constexpr (kRowsKind)
                                weights32_at_any_size(x0, c, m == -INFINITY ? 0.0f : m, sum, pk);
                            else
                                weights32<kBfMath>(x0, c, mc, sum, pk);
                            tmem_st16(s_at + 64 + q * 16, pk);
                        }
                    } else {
                        tmem_ld32(s_at + 64, x0);  // the last 32 are still in x1
                        weights32<kBfMath>(x1, c, mc, sum, pk);
                        tmem_st16(s_at + 112, pk);
                        tc_wait_ld();
                        tmem_ld32(s_at + 32, x1);
                        weights32<kBfMath>(x0, c, mc, sum, pk);
                        tmem_st16(s_at + 96, pk);
                        tc_wait_ld();
                        tmem_ld32(s_at, x0);
                        weights32<kBfMath>(x1, c, mc, sum, pk);
                        tmem_st16(s_at + 80, pk);
                        tc_wait_ld();
                        weights32<kBfMath>(x0, c, mc, sum, pk);
                        tmem_st16(s_at + 64, pk);
                    }
                    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                    tc_wait_st();
                }
                if (owes_free) {  // this step's product overwrites O
                    if (!wait.warp(smem_addr(&aux.merge_free), (joins - 1) & 1)) { ok = false; break; }
                    owes_free = false;
                }
                tc_fence_before();
                warp_arrive(smem_addr(&aux.p_ready[g]));
                steps++;
            }
            if (!ok) break;
            if (kScaled) m *= back;
            const bool had = first < w.n;
            if (had && !wait.warp(smem_addr(&aux.o_done[g]), (steps - 1) & 1)) { ok = false; break; }
            tc_fence_after();
            if (!both) joins++;
            if (!both && g == 1) {
                // the even tiles' group joins and writes
                if (owes_free) {  // it had no step in this unit: the last join must be over before its m, l go
                    if (!wait.warp(smem_addr(&aux.merge_free), (joins - 2) & 1)) { ok = false; break; }
                }
                aux.m[t] = m;
                aux.l[t] = l;
                tc_fence_before();
                warp_arrive(smem_addr(&aux.merge_ready));
                owes_free = true;
                continue;
            }
            float a0 = 1.0f, a1 = 0.0f;
            const bool join = !both && w.n > 1;
            if (!both) {
                if (!wait.warp(smem_addr(&aux.merge_ready), (joins - 1) & 1)) { ok = false; break; }
                tc_fence_after();
                const float m1 = aux.m[t], l1 = aux.l[t], top = fmaxf(m, m1);
                if (top > -INFINITY) {
                    a0 = exp2_fast((m - top) * p.o.c);
                    a1 = exp2_fast((m1 - top) * p.o.c);
                }
                l = l * a0 + l1 * a1;
                m = top;
            }
            const bool whole = w.whole();
            const float inv = (l > 0.0f ? 1.0f / l : 0.0f) * (kRowsKind ? p.o.values : 1.0f);
            const int slot = 2 * blockIdx.x + (w.at.off == 0 ? 1 : 0);
            float *part = p.ws + (int64_t)slot * (kRows * (DV + 2)), *lse = nullptr;
            char *to = live ? place(lse) : nullptr;
            if (warp_live) {
#pragma unroll 1
                for (int q = 0; q < DV / 32; q++) {
                    uint32_t o[32];
                    tmem_ld32(o_at + q * 32, o);
                    float f[32];
                    if (join) {
                        uint32_t o1[32];
                        tmem_ld32(o_at + 128 + q * 32, o1);
                        tc_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; i++) f[i] = __uint_as_float(o[i]) * a0 + __uint_as_float(o1[i]) * a1;
                    } else {
                        tc_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; i++) f[i] = __uint_as_float(o[i]);
                    }
                    if (l == 0.0f) {
#pragma unroll
                        for (int i = 0; i < 32; i++) f[i] = 0.0f;
                    }
                    if (whole)
                        store_rows32<Bf16>(to, f, inv, q * 32, p.o.dv);
                    else if (live)
                        store_fragment32(part, kRows, row, q, f);
                }
                if (live) {
                    if (whole) {
                        if (lse) *lse = l > 0.0f ? fmaf(m, p.o.scale, weight_log<kBfMath>(l)) : -INFINITY;
                    } else {
                        part[kRows * DV + row] = m;
                        part[kRows * DV + kRows + row] = l;
                    }
                }
            }
            if (!both) {
                tc_fence_before();
                warp_arrive(smem_addr(&aux.merge_free));
            }
            if (!whole) {
                const Cut cut(line, w.pos - w.at.off, unit_cost(w.u));
                const int row0 = both ? g * half : 0;
                join_unit<DV, Bf16, kBfMath>(p.o, p.ws, cut, p.counters + 2 * cut.c0 + g, 2, 1, 0, 1, kRows * (DV + 2), row0, min(half, w.u.rows - row0), kRows,
                                    w.u.row0, w.q.q0, w.at.head * (int)b.group.d, b.group, smem_addr(&aux.join[g]), cuts, &aux.answer[g], wait, ok);
                if (!ok) break;
            }
        } while (w.next(b));
        (void)ok;
    } else {
        if (kRowsKind) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (!kRowsKind && warp == 0) {
        // ---- keys ----
        int it = 0;
        bool ok = true;
        do {
            if (w.u.tiles == 0) continue;
            const int32_t *row = p.table + (int64_t)w.at.req * p.table_stride;
            for (int t = 0; ok && t < w.n; t++, it++) {
                const int s = it % S::kNK;
                ok = load_tile<DK / 64>(p, &k_map, row, (w.u.tile0 + w.at.off + t) * kTile, w.u.lo, w.u.hi, w.at.head, base + S::kOffK + s * S::kK,
                                        smem_addr(&aux.k_full[s]), [&] { return it < S::kNK || wait.warp(smem_addr(&aux.k_empty[s]), ((it / S::kNK) - 1) & 1); });
            }
        } while (ok && w.next(b));
    } else if (!kRowsKind && warp == 2) {
        // ---- values ----
        int it = 0;
        bool ok = true;
        do {
            if (w.u.tiles == 0) continue;
            const int32_t *row = p.table + (int64_t)w.at.req * p.table_stride;
            for (int t = 0; ok && t < w.n; t++, it++) {
                const int s = it % S::kNV;
                ok = load_tile<DV / 64>(p, &v_map, row, (w.u.tile0 + w.at.off + t) * kTile, w.u.lo, w.u.hi, w.at.head, base + S::kOffV + s * S::kV,
                                        smem_addr(&aux.v_full[s]), [&] { return it < S::kNV || wait.warp(smem_addr(&aux.v_empty[s]), ((it / S::kNV) - 1) & 1); });
            }
        } while (ok && w.next(b));
    } else if (warp == 3) {
        // ---- queries: as soon as the last scores of the unit before are out ----
        int units = 0;
        bool ok = true;
        do {
            if (w.u.tiles == 0) continue;
            if (units && !wait.warp(smem_addr(&aux.q_empty), (units - 1) & 1)) break;
            units++;
            load_queries<DK>(p, &q_map, w, half, base, smem_addr(&aux.q_full));
        } while (ok && w.next(b));
    } else if (warp == 1) {
        // ---- matrix products ----
        constexpr uint32_t qk_desc = mma_desc(kBfMath, 128, 128, false), pv_desc = mma_desc(kBfMath, 128, DV, true);
        const uint32_t elected = elect_one();
        const uint64_t qd = smem_desc(base, 16, 1024), kd = smem_desc(base + S::kOffK, 16, 1024), vd = smem_desc(base + S::kOffV, kPanel, 1024);
        int it = 0, steps[2] = {0, 0}, units = 0;
        bool ok = true;
        do {
            if (w.u.tiles == 0) continue;
            const bool both = w.u.rows > half;
            const int n = both ? 2 * w.n : w.n;
            ok = kScaled ? wait.warp(smem_addr(&aux.q_ready[units & 1]), units >> 1 & 1) : wait.warp(smem_addr(&aux.q_full), units & 1);
            units++;
            if (!ok) break;
            tc_fence_after();
            const auto qk = [&](int i) {
                const int s = i & 1, kt = it + (both ? i >> 1 : i), slot = kt % S::kNK;
                if ((!both || s == 0) && !wait.warp(smem_addr(&aux.k_full[slot]), (kt / S::kNK) & 1)) return false;
                const uint64_t qa = qd + (both && s ? S::kQ >> 4 : 0), ka = kd + slot * (S::kK >> 4);
#pragma unroll
                for (int kk = 0; kk < DK / 16; kk++) {
                    const uint32_t o = ((kk / 4) * kPanel + (kk % 4) * 32) >> 4;
                    mma_ss(tmem + s * 128, qa + o, ka + o, qk_desc, kk > 0, elected);
                }
                if (!both || s == 1) tc_commit(smem_addr(&aux.k_empty[slot]), elected);
                if (i == n - 1) tc_commit(smem_addr(&aux.q_empty), elected);
                tc_commit(smem_addr(&aux.s_full[s]), elected);
                return true;
            };
            ok = qk(0) && (n < 2 || qk(1));
            for (int i = 0; ok && i < n; i++) {
                const int s = i & 1, vt = it + (both ? i >> 1 : i), slot = vt % S::kNV;
                ok = wait.warp(smem_addr(&aux.p_ready[s]), steps[s]++ & 1) &&
                     ((both && s) || wait.warp(smem_addr(&aux.v_full[slot]), (vt / S::kNV) & 1));
                if (!ok) break;
                // the tile's runs of 32 keys that some query sees; in them, rows of V that none sees must not reach the
                // product: they may hold anything (rows of another kind were left out when the tile was made)
                const int kb = (w.u.tile0 + w.at.off + vt - it) * kTile, q0 = seen_from(w.u, kb), q1 = seen_to(w.u, kb);
                if (!kRowsKind && !(both && s) && (kb < w.u.lo || kb + kTile > w.u.hi)) {
                    for (int r = 32 * q0 + (lane >> 3); r < 32 * q1; r += 4)
                        if (kb + r < w.u.lo || kb + r >= w.u.hi)
#pragma unroll
                            for (int h = 0; h < DV / 64; h++)
                                st_smem16(base + S::kOffV + slot * S::kV + h * kPanel + r * 128 + (lane & 7) * 16, make_uint4(0, 0, 0, 0));
                    fence_async_smem();
                    __syncwarp();
                }
                tc_fence_after();
                const uint64_t va = vd + slot * (S::kV >> 4);
#pragma unroll
                for (int kk = 0; kk < 8; kk++)
                    mma_ts(tmem + 256 + s * 128, tmem + s * 128 + 64 + kk * 8, va + kk * (2048 >> 4), pv_desc, i >= 2 || kk > 2 * q0,
                           elected && kk >= 2 * q0 && kk < 2 * q1);
                if (!both || s == 1) tc_commit(smem_addr(&aux.v_empty[slot]), elected);
                tc_commit(smem_addr(&aux.o_done[s]), elected);  // last: the groups wait for it before the CTA ends
                if (i + 2 < n) ok = qk(i + 2);
            }
            it += w.n;
        } while (ok && w.next(b));
    } else if (kRowsKind && warp < 12) {
        // ---- packed rows of keys (warp 0) and of values (warp 2) ----
        if constexpr (kRowsKind) {
            const bool v = warp == 2;
            const Rows &rows = v ? p.v : p.k;
            int slot = v ? 1 : 0, turn = 0;
            bool ok = true;
            do {
                if (w.u.tiles == 0) continue;
                const int32_t *row = p.table + (int64_t)w.at.req * p.table_stride;
                for (int t = 0; ok && t < w.n; t++) {
                    ok = rows.load(p, v ? &v_map : &k_map, row, (w.u.tile0 + w.at.off + t) * kTile, w.u.lo, w.u.hi, w.at.head,
                                   base + S::kOffStage + slot * rows.stage_bytes, smem_addr(&aux.stage_full[slot]), !v,
                                   [&] { return turn == 0 || wait.warp(smem_addr(&aux.stage_empty[slot]), (turn - 1) & 1); });
                    if ((slot += 2) >= p.stages) slot -= p.stages, turn++;
                }
            } while (ok && w.next(b));
        }
    } else if (kRowsKind) {
        // ---- tiles of them ----
        if constexpr (kRowsKind) {
            const int thread = tid - 384;
            int slot = 0, turn = 0, it = 0, units = 0;
            bool ok = true;
            do {
                if (w.u.tiles == 0) continue;
                for (int t = 0; ok && t < w.n; t++, it++) {
                    const int kb = (w.u.tile0 + w.at.off + t) * kTile;
#pragma unroll 1
                    for (int v = 0; v < 2; v++) {
                        static_assert(!kRowsKind || S::kNK == S::kNV, "one ring depth");
                        constexpr int depth = S::kNK;
                        const int to = it % depth;
                        const uint32_t full = smem_addr(v ? &aux.v_full[to] : &aux.k_full[to]), empty = smem_addr(v ? &aux.v_empty[to] : &aux.k_empty[to]);
                        const Rows &rows = v ? p.v : p.k;
                        ok = (it < depth || wait.warp(empty, (it / depth - 1) & 1)) && wait.warp(smem_addr(&aux.stage_full[slot]), turn & 1);
                        if (!ok) break;
                        rows.template unpack<DK>(base + S::kOffStage + slot * rows.stage_bytes, base + (v ? S::kOffV + to * S::kV : S::kOffK + to * S::kK),
                                                       w.at.head, w.u.lo - kb, w.u.hi - kb, thread);
                        fence_async_smem();
                        warp_arrive(full);
                        if (lane == 0) mbar_arrive(smem_addr(&aux.stage_empty[slot]));
                        if (++slot == p.stages) slot = 0, turn++;
                    }
                    if (kScaled && t == 0 && ok) {  // behind the first tiles, which can be made before the unit's queries are there
                        ok = wait.warp(smem_addr(&aux.q_full), units & 1);
                        if (!ok) break;
#pragma unroll 1
                        for (int g = 0; g < (w.u.rows > half ? 2 : 1); g++)
                            smem[S::kOffScales + (units & 1) * 256 + g * 128 + thread] = (unsigned char)scale_row<DK>(base + g * S::kQ, thread);
                        fence_async_smem();
                        warp_arrive(smem_addr(&aux.q_ready[units++ & 1]));
                    }
                }
            } while (ok && w.next(b));
        }
    }
    }
    // common exit
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (aux.gave_up) {  // let copies in flight land before the shared memory is given back
        const unsigned long long t0 = now_ns();
        while (now_ns() - t0 < 10000000ull) {}
    }
    if (warp == 3) tmem_free(tmem, 512);
}

}  // namespace

}  // namespace pkv
