// kv_attention: softmax attention of a ragged batch of new tokens over paged keys and values.
//
// out = softmax(scale q K^T) V, one pass over the keys: a row keeps the running maximum m and the
// running sum l of 2^(c (s - m)) (c = scale log2 e), and the accumulator O is multiplied by
// 2^(c (m_old - m_new)) when m moves.  Partial results of disjoint key ranges join the same way.
//
// One persistent CTA per SM walks its piece of the batch's line of key tiles (kv_plan.cuh).  A unit
// is up to 256 query rows (tokens x heads of one key head's group) and its key tiles of 128 keys:
//   warps 0, 2    load K and V: one tiled TMA per (64-element panel, run of slots inside a page) into a
//                 ring of tiles each, the page ids looked up before the wait for a slot; warp 3 loads Q
//   warp 1        issues every tcgen05.mma: S = Q K^T and O += P V, accumulators in TMEM
//   warps 4-7, 8-11   two softmax groups, a thread per row: S from TMEM, maximum, exponentials, P back to
//                 TMEM (over S) as the A operand of the second product, O rescaled only when the
//                 maximum has grown by more than 2^8 (P stays below 2^8, in fp16 2^7 times that, inside
//                 16-bit range, so most tiles touch O not at all)
// TMEM: S0, S1 (128 columns each) and O0, O1 (128 columns each).  With more than 128 rows the two groups
// own 128 rows each and share every K and V tile; with fewer (decoding) they take the even and the odd
// key tiles of the same rows and are joined through TMEM, so both ways keep two tiles in flight between
// the tensor core and the exponentials.
//
// Decoding is bound by memory: 64 requests of 4096 to 12288 tokens, 32 heads over 8 of 128, take 322 to
// 331 us, 97% of the copy rate or more.  Chunks (four of 2048 to 4096 tokens over 4096 to 8192: 670 to 705 us, 1.3
// PFLOP/s, two thirds of the tensor cores' measured rate) fill no unit of the SM.  A step of 256 rows by 128 keys takes
// about 3600 cycles, and needs 2048 of the tensor core, 1536 of shared memory for its operands and 512 of the
// exponentials.  What bounds it is the order within a group: scores, their maximum, all 128 weights of every row, the value
// product, and only then the next scores; two groups do not hide each other's waits.  With keys of 192 a step takes
// about 5900 cycles, 2560 of them tensor work: there one stage of values and two of keys is all that fits.
#include <cmath>

#include "kv_attention.cuh"

namespace pkv {

namespace {

constexpr int kLeast = 4;  // tiles of a piece of a unit, at least (a join costs as much as three or four more tiles: 3 to 5 us)
constexpr int kThreads = 384;
constexpr int kRows = 256;  // rows of a unit, at most: 2 * floor(128 / group) tokens of a group
constexpr int kTileShift = 7, kTile = 1 << kTileShift;  // keys of a tile
constexpr uint32_t kPanel = 128 * 128;  // bytes of a 64-element panel of 128 rows

template <int DK, int DV>
struct Shape {
    static constexpr uint32_t kQ = 128 * DK * 2, kK = 128 * DK * 2, kV = 128 * DV * 2;
    static constexpr int kNK = DK == 64 ? 5 : DK == 128 ? 3 : 2;  // ring depths: what 227 KB holds
    static constexpr int kNV = DK == 64 ? 5 : DK == 128 ? 2 : 1;  // (192: four single panels of K and two tiles of V ran 7% slower)
    static constexpr uint32_t kOffK = 2 * kQ, kOffV = kOffK + kNK * kK, kOffAux = kOffV + kNV * kV;
    static constexpr uint32_t kBytes = kOffAux + 2048;
};

struct Params {
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

// Bookkeeping at the end of shared memory.
struct Aux {
    uint64_t k_full[5], k_empty[5], v_full[5], v_empty[5];
    uint64_t s_full[2], p_ready[2], o_done[2], q_full, q_empty, merge_ready, merge_free, join[2];
    int scan[48];
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
__device__ __forceinline__ bool load_tile(const Params &p, const CUtensorMap *map, const int32_t *row, int kb, int lo, int hi, int head,
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

template <int DK, int DV, bool Bf16>
__global__ void __launch_bounds__(kThreads, 1)
attention_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                 const __grid_constant__ CUtensorMap v_map, const Params p)
{
    using S = Shape<DK, DV>;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t base = smem_addr(smem);
    Aux &aux = *reinterpret_cast<Aux *>(smem + S::kOffAux);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const Batch &b = p.b;
    const Waiter wait{&aux.gave_up, b.err};

    if (tid == 0) {
        aux.gave_up = 0;
        for (int i = 0; i < S::kNK; i++) mbar_init(smem_addr(&aux.k_full[i]), 1), mbar_init(smem_addr(&aux.k_empty[i]), 1);
        for (int i = 0; i < S::kNV; i++) mbar_init(smem_addr(&aux.v_full[i]), 1), mbar_init(smem_addr(&aux.v_empty[i]), 1);
        for (int i = 0; i < 2; i++) {
            mbar_init(smem_addr(&aux.s_full[i]), 1);
            mbar_init(smem_addr(&aux.p_ready[i]), 4);
            mbar_init(smem_addr(&aux.o_done[i]), 1);
            mbar_init(smem_addr(&aux.join[i]), 4);
        }
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
    const Line line = find_place<kThreads>(b, blockIdx.x, gridDim.x, kLeast, aux.scan, &aux.place, blockIdx.x == 0);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, aux.tmem, 0);
    const int half = b.unit_rows / 2;  // rows of a softmax group
    Walk w;
    const bool any = w.start(b, aux.place, line);
    if (!any) {
        // nothing to do: on to the common exit
    } else if (warp == 0) {
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
    } else if (warp == 2) {
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
            const int group = (int)b.group.d, tok0 = (int)fdiv((uint32_t)w.u.row0, b.group), toks = w.u.rows / group, per_half = half / group;
            // boxes of q_box tokens; a box that begins in the first half ends there
            const int n0 = (min(toks, per_half) + p.q_box - 1) / p.q_box, n1 = toks > per_half ? (toks - per_half + p.q_box - 1) / p.q_box : 0;
            if (lane == 0) mbar_arrive_expect_tx(smem_addr(&aux.q_full), (uint32_t)((n0 + n1) * p.q_box * group) * DK * 2);
            __syncwarp();
            for (int i = lane; i < n0 + n1; i += 32) {
                const int g = i >= n0, t = (i - (g ? n0 : 0)) * p.q_box;
#pragma unroll
                for (int h = 0; h < DK / 64; h++)
                    tma_load_3d(base + g * S::kQ + h * kPanel + t * group * 128, &q_map, smem_addr(&aux.q_full), h * 64, w.at.head * group,
                                w.q.q0 + tok0 + g * per_half + t);
            }
            __syncwarp();
        } while (ok && w.next(b));
    } else if (warp == 1) {
        // ---- matrix products ----
        constexpr uint32_t qk_desc = mma_desc(Bf16, 128, 128, false), pv_desc = mma_desc(Bf16, 128, DV, true);
        const uint32_t elected = elect_one();
        const uint64_t qd = smem_desc(base, 16, 1024), kd = smem_desc(base + S::kOffK, 16, 1024), vd = smem_desc(base + S::kOffV, kPanel, 1024);
        int it = 0, steps[2] = {0, 0}, units = 0;
        bool ok = true;
        do {
            if (w.u.tiles == 0) continue;
            const bool both = w.u.rows > half;
            const int n = both ? 2 * w.n : w.n;
            ok = wait.warp(smem_addr(&aux.q_full), units++ & 1);
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
                // product: they may hold anything
                const int kb = (w.u.tile0 + w.at.off + vt - it) * kTile, q0 = seen_from(w.u, kb), q1 = seen_to(w.u, kb);
                if (!(both && s) && (kb < w.u.lo || kb + kTile > w.u.hi)) {
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
    } else {
        // ---- softmax: group g, a thread per row ----
        const int g = (warp - 4) >> 2, t = tid & 127;
        const uint32_t mine = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_at = tmem + g * 128 + mine, o_at = tmem + 256 + g * 128 + mine;
        const float slack = 8.0f / p.o.c;  // how far the maximum may grow before O is rescaled
        int steps = 0, joins = 0, cuts = 0;
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
            float m = -INFINITY, l = 0.0f;
            const int first = both ? 0 : g, step = both ? 1 : 2, kt0 = w.u.tile0 + w.at.off;
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
                    const bool grow = top > (Bf16 ? m + slack : __fadd_rd(m, slack));  // -inf + slack: the first finite score
                    if (__any_sync(0xffffffffu, grow)) {
                        const float to_m = grow ? top : m;
                        const float alpha = grow ? exp2_fast((m - to_m) * p.o.c) : 1.0f;
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
                    const float mc = weight_offset<Bf16>(m, p.o.c);
                    float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                    uint32_t pk[16];
                    // P takes the columns of the upper 64 scores: 32 keys' weights stand in 16 columns from 64 on, so
                    // going down no score is overwritten before it has been read
                    if (hide) {
#pragma unroll 1
                        for (int q = seen_to(w.u, kb) - 1; q >= seen_from(w.u, kb); q--) {
                            tmem_ld32(s_at + q * 32, x0);
                            tc_wait_ld();
                            hide32(x0, from - q * 32, to_key - q * 32);
                            weights32<Bf16>(x0, p.o.c, mc, sum, pk);
                            tmem_st16(s_at + 64 + q * 16, pk);
                        }
                    } else {
                        tmem_ld32(s_at + 64, x0);  // the last 32 are still in x1
                        weights32<Bf16>(x1, p.o.c, mc, sum, pk);
                        tmem_st16(s_at + 112, pk);
                        tc_wait_ld();
                        tmem_ld32(s_at + 32, x1);
                        weights32<Bf16>(x0, p.o.c, mc, sum, pk);
                        tmem_st16(s_at + 96, pk);
                        tc_wait_ld();
                        tmem_ld32(s_at, x0);
                        weights32<Bf16>(x1, p.o.c, mc, sum, pk);
                        tmem_st16(s_at + 80, pk);
                        tc_wait_ld();
                        weights32<Bf16>(x0, p.o.c, mc, sum, pk);
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
            const float inv = l > 0.0f ? 1.0f / l : 0.0f;
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
                        if (lse) *lse = l > 0.0f ? fmaf(m, p.o.scale, weight_log<Bf16>(l)) : -INFINITY;
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
                join_unit<DV, Bf16>(p.o, p.ws, cut, p.counters + 2 * cut.c0 + g, 2, 1, 0, 1, kRows * (DV + 2), row0, min(half, w.u.rows - row0), kRows,
                                    w.u.row0, w.q.q0, w.at.head * (int)b.group.d, b.group, smem_addr(&aux.join[g]), cuts, &aux.answer[g], wait, ok);
                if (!ok) break;
            }
        } while (w.next(b));
        (void)ok;
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

template <int DK, int DV, bool Bf16>
int launch_attention(const CUtensorMap &qm, const CUtensorMap &km, const CUtensorMap &vm, const Params &p, int parts, cudaStream_t s, bool prepare)
{
    const auto kernel = attention_kernel<DK, DV, Bf16>;
    if (prepare)
        return cuda_status(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Shape<DK, DV>::kBytes));
    return cuda_status(launch(kernel, dim3(parts), dim3(kThreads), Shape<DK, DV>::kBytes, s, qm, km, vm, p));
}

template <bool Bf16>
int pick_attention(int dk, int dv, const CUtensorMap &qm, const CUtensorMap &km, const CUtensorMap &vm, const Params &p, int parts, cudaStream_t s, bool prepare)
{
    if (dk <= 64 && dv <= 64) return launch_attention<64, 64, Bf16>(qm, km, vm, p, parts, s, prepare);
    if (dk <= 128) return launch_attention<128, 128, Bf16>(qm, km, vm, p, parts, s, prepare);
    return launch_attention<192, 128, Bf16>(qm, km, vm, p, parts, s, prepare);
}

}  // namespace

int check_batch(const kv_attn_batch *t)
{
    if (t == nullptr || t->n_reqs < 0 || t->n_tokens < 0 || t->max_blocks_per_req < 0 || t->bt_row_stride < 0) return KV_ERR_INVALID_ARG;
    if (t->n_reqs > 0 && (t->q_offsets == nullptr || t->kv_lens == nullptr || (t->block_table == nullptr && t->max_blocks_per_req > 0)))
        return KV_ERR_INVALID_ARG;
    if (t->n_reqs > 1 && t->bt_row_stride < t->max_blocks_per_req) return KV_ERR_INVALID_ARG;
    return KV_OK;
}

// Fills the batch a kernel works on; lengths are held in 32 bits.
int fill_batch(Batch *b, const kv_attn_batch *t, int heads, int kv_heads, int block_size, int unit_rows, int tile_shift, int causal, int window)
{
    const int64_t max_tokens = (int64_t)t->max_blocks_per_req * block_size;
    if (max_tokens > (1ll << 30) || t->n_tokens > (1ll << 30) / heads) return KV_ERR_UNSUPPORTED;
    b->q_offsets = t->q_offsets;
    b->kv_lens = t->kv_lens;
    b->n_reqs = t->n_reqs;
    b->n_tokens = (int32_t)t->n_tokens;
    b->max_tokens = (int32_t)max_tokens;
    b->kv_heads = kv_heads;
    b->unit_rows = unit_rows;
    b->tile_shift = tile_shift;
    b->causal = causal ? 1 : 0;
    b->window = window < max_tokens ? window : 0;  // a longer one hides nothing, and would overflow beside a position
    b->group = make_fastdiv((uint32_t)(heads / kv_heads));
    b->unit = make_fastdiv((uint32_t)unit_rows);
    // the line's steps are counted in 32 bits
    const int64_t units = t->n_tokens * heads / unit_rows + (int64_t)t->n_reqs * kv_heads;
    if (units > ((1ll << 31) - 1) / ((max_tokens >> tile_shift) + 1)) return KV_ERR_UNSUPPORTED;
    b->err = nullptr;
    return KV_OK;
}

// One plane of one tensor as rows of `heads` heads of `dim` 16-bit elements.
int check_plane(const kv_cache_desc *c, int tensor, int plane, int heads, int dim)
{
    const int st = check_cache(c);
    if (st != KV_OK) return st;
    if (tensor < 0 || tensor >= c->n_tensors || plane < 0 || plane >= c->n_planes) return KV_ERR_INVALID_ARG;
    if ((int64_t)heads * dim * 2 != c->row_bytes) return KV_ERR_INVALID_ARG;
    if (c->num_blocks >= (1ll << 31) || c->token_stride >= (1ll << 40) || c->block_stride >= (1ll << 40)) return KV_ERR_UNSUPPORTED;
    if (c->num_blocks == 0) return KV_ERR_INVALID_ARG;
    return KV_OK;
}

int box_tokens(int most, const kv_attn_batch *t)
{
    int n = 1;
    while (n < most && (most % n || (int64_t)n * t->n_reqs < t->n_tokens)) n++;
    return n;
}

int make_q_map(CUtensorMap *map, const void *q, int64_t token_stride, int64_t head_stride, int head_dim, int heads, int64_t tokens, int group,
               int box_tokens)
{
    if (token_stride >= (1ll << 40) || head_stride >= (1ll << 40)) return KV_ERR_UNSUPPORTED;
    const uint64_t dims[3] = {(uint64_t)head_dim, (uint64_t)heads, (uint64_t)tokens};
    const uint64_t strides[2] = {(uint64_t)head_stride, (uint64_t)token_stride};
    const uint32_t box[3] = {64, (uint32_t)group, (uint32_t)box_tokens};
    return make_map(map, (uint64_t)q, 3, dims, strides, box);
}

int piece_rows(int block_size, int tile)
{
    int n = 1;
    while (n < tile && block_size % (2 * n) == 0) n *= 2;
    return n;
}

int check_rows(const void *p, int64_t token_stride, int64_t head_stride)
{
    if (p == nullptr || token_stride < 0 || head_stride < 0) return KV_ERR_INVALID_ARG;
    if (!aligned16(p) || !aligned16(token_stride) || !aligned16(head_stride)) return KV_ERR_ALIGN;
    return KV_OK;
}

int preload_attention_kernels()
{
    Params p = {};
    CUtensorMap m;
    for (int dk : {64, 128, 192})
        for (bool bf : {false, true}) {
            const int st = bf ? pick_attention<true>(dk, dk == 64 ? 64 : 128, m, m, m, p, 0, nullptr, true)
                              : pick_attention<false>(dk, dk == 64 ? 64 : 128, m, m, m, p, 0, nullptr, true);
            if (st != KV_OK) return st;
        }
    return load_kernels(attention_kernel<64, 64, false>, attention_kernel<64, 64, true>, attention_kernel<128, 128, false>,
                        attention_kernel<128, 128, true>, attention_kernel<192, 128, false>, attention_kernel<192, 128, true>);
}

}  // namespace pkv

using namespace pkv;

extern "C" {

int kv_attention_workspace_bytes(int64_t *bytes_out)
{
    if (bytes_out == nullptr) return KV_ERR_INVALID_ARG;
    const DeviceInfo *d = current_device();
    if (d == nullptr) return KV_ERR_CUDA;
    *bytes_out = attention_workspace(d->num_sms);
    return KV_OK;
}

int kv_attention(const kv_attn_desc *d, const kv_attn_batch *batch, const kv_cache_desc *k, int32_t k_tensor, int32_t k_plane,
                 const kv_cache_desc *v, int32_t v_tensor, int32_t v_plane, const void *q, int64_t q_token_stride,
                 int64_t q_head_stride, void *out, int64_t out_token_stride, int64_t out_head_stride, float *lse, void *workspace,
                 int64_t workspace_bytes, kv_stream_t stream)
{
    if (d == nullptr || d->n_heads <= 0 || d->n_kv_heads <= 0 || d->n_heads % d->n_kv_heads != 0 || d->head_dim <= 0 ||
        d->head_dim_v <= 0 || d->window < 0 || !good_scale(d->scale) ||
        (d->dtype != KV_BF16 && d->dtype != KV_F16))
        return KV_ERR_INVALID_ARG;
    int st = check_batch(batch);
    if (st != KV_OK) return st;
    if (d->head_dim % 8 || d->head_dim_v % 8) return KV_ERR_ALIGN;
    const int group = d->n_heads / d->n_kv_heads;
    if (d->head_dim > 192 || d->head_dim_v > 128 || group > 128 || (d->window && !d->causal)) return KV_ERR_UNSUPPORTED;
    if ((st = check_plane(k, k_tensor, k_plane, d->n_kv_heads, d->head_dim)) != KV_OK) return st;
    if ((st = check_plane(v, v_tensor, v_plane, d->n_kv_heads, d->head_dim_v)) != KV_OK) return st;
    if (k->block_size != v->block_size) return KV_ERR_INVALID_ARG;
    if (batch->n_reqs == 0 || batch->n_tokens == 0) return KV_OK;
    if ((st = check_rows(q, q_token_stride, q_head_stride)) != KV_OK) return st;
    if ((st = check_rows(out, out_token_stride, out_head_stride)) != KV_OK) return st;
    if (workspace == nullptr) return KV_ERR_INVALID_ARG;
    if (!aligned16(workspace) || ((uintptr_t)lse & 3u)) return KV_ERR_ALIGN;
    Params p = {};
    if ((st = fill_batch(&p.b, batch, d->n_heads, d->n_kv_heads, k->block_size, 2 * (128 / group) * group, kTileShift, d->causal, d->window)) != KV_OK) return st;
    const DeviceInfo *dev = current_device();
    if (dev == nullptr) return KV_ERR_CUDA;
    if (workspace_bytes < attention_workspace(dev->num_sms)) return KV_ERR_RANGE;
    if ((st = prepare_attention(*dev)) != KV_OK) return st;
    p.b.err = dev->err_word;
    p.table = batch->block_table;
    p.table_stride = batch->bt_row_stride;
    p.num_blocks = (int32_t)(k->num_blocks < v->num_blocks ? k->num_blocks : v->num_blocks);
    p.no_page = (int32_t)(k->num_blocks < v->num_blocks ? v->num_blocks : k->num_blocks);
    p.block = make_fastdiv((uint32_t)k->block_size);
    p.piece_rows = piece_rows(k->block_size, kTile);
    p.o = Output{(char *)out, out_token_stride, out_head_stride, lse, d->n_heads, d->head_dim_v, d->scale, d->scale * kLog2e};
    p.counters = (int *)workspace;
    p.ws = (float *)((char *)workspace + kCounterBytes);
    p.q_box = box_tokens(128 / group, batch);
    CUtensorMap qm, km, vm;
    if ((st = make_q_map(&qm, q, q_token_stride, q_head_stride, d->head_dim, d->n_heads, batch->n_tokens, group, p.q_box)) != KV_OK) return st;
    if ((st = make_cache_map(&km, k, k_tensor, k_plane, d->n_kv_heads, d->head_dim, p.piece_rows)) != KV_OK) return st;
    if ((st = make_cache_map(&vm, v, v_tensor, v_plane, d->n_kv_heads, d->head_dim_v, p.piece_rows)) != KV_OK) return st;
    cudaStream_t s = (cudaStream_t)stream;
    return d->dtype == KV_BF16 ? pick_attention<true>(d->head_dim, p.o.dv, qm, km, vm, p, dev->num_sms, s, false)
                               : pick_attention<false>(d->head_dim, p.o.dv, qm, km, vm, p, dev->num_sms, s, false);
}

}  // extern "C"
