// kv_latent_attention for many requests of few rows: decoding with up to 64 heads on this GPU.
//
// Keys are whole rows of 576 elements, values their first 512, as in kv_latent.cu; with at most 64 query rows a
// unit one CTA holds everything and computes every score once.  What bounds it is memory, so the tiles are small
// (32 keys, 36 KB) and four deep: two tiles of 64 keys, the same bytes, left the loads idle while a tile was
// worked on (64 requests of 6000 to 10000 tokens, 16 heads: 158 us, against 111, 77% of the copy rate).
// An accumulator of 64 rows takes 16 of every 32 lanes of tensor memory, so the two halves of the values lie in
// the same 256 columns, one in the lower and one in the upper 16 lanes: row r in lane 32 (r / 16) + r % 16, and
// 16 above.  Shared memory: Q 72 KB, keys 144 KB, and the weights P, from where they are the second product's A
// operand.  Of a tile's 1600 cycles (this SM's share of the memory's rate) its products take about 1200 of the
// tensor core's operand reads, its weights about 400 in four warps.
//   warps 0, 2   load the panels of a tile, five and four (a warp issues a TMA in about 140 cycles)
//   warp 3       loads Q; warp 1 issues the products: S = Q K^T of the next tile before O += P V of this one
//   warps 4-7    16 rows each: a thread a row for the scores (the upper lanes idle), two threads a row for O
#include "kv_latent.cuh"

namespace pkv {

namespace {

constexpr int kLeast = 4;  // tiles of a piece of a unit, at least (as many keys as in kv_latent.cu)
constexpr int kThreads = 256;
constexpr int kRows = kLatentFewRows, kKeys = 1 << kLatentFewKeyShift, kHalf = kLatentRank / 2;
constexpr int kStages = 4;
constexpr uint32_t kQPanel = kRows * 128, kPanel = kKeys * 128, kTile = 9 * kPanel;  // bytes; a panel: 64 elements of each row
constexpr uint32_t kOffK = 9 * kQPanel, kOffP = kOffK + kStages * kTile, kOffAux = kOffP + kQPanel, kBytes = kOffAux + 1024;
constexpr uint32_t kTmO = 0, kTmS = 256;
constexpr uint32_t kUpper = 16u << 16;  // the upper 16 lanes

struct Aux {
    uint64_t k_full[kStages], k_empty[kStages], s_full[2], p_ready, o_done, q_full, q_empty, join;
    int scan[32];
    Place place;
    uint32_t tmem;
    int answer;
    int gave_up;
};
static_assert(sizeof(Aux) <= 1024, "bookkeeping");

template <bool Bf16>
__global__ void __launch_bounds__(kThreads, 1)
latent_few_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ CUtensorMap q_map, const LatentParams p)
{
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t base = smem_addr(smem);
    Aux &aux = *reinterpret_cast<Aux *>(smem + kOffAux);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const Batch &b = p.b;
    const Waiter wait{&aux.gave_up, b.err};

    if (tid == 0) {
        aux.gave_up = 0;
        for (int i = 0; i < kStages; i++) {
            mbar_init(smem_addr(&aux.k_full[i]), 2);
            mbar_init(smem_addr(&aux.k_empty[i]), 1);
        }
        for (int i = 0; i < 2; i++) mbar_init(smem_addr(&aux.s_full[i]), 1);
        mbar_init(smem_addr(&aux.p_ready), 4);
        mbar_init(smem_addr(&aux.o_done), 1);
        mbar_init(smem_addr(&aux.q_full), 1);
        mbar_init(smem_addr(&aux.q_empty), 1);
        mbar_init(smem_addr(&aux.join), 4);
        mbar_init_fence();
        tma_prefetch_map(&map);
        tma_prefetch_map(&q_map);
    }
    if (warp == 2) tmem_alloc(smem_addr(&aux.tmem), 512);
    grid_dep_entry();
    const Line line = find_place<kThreads>(b, blockIdx.x, gridDim.x, kLeast, aux.scan, &aux.place, blockIdx.x == 0);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, aux.tmem, 0);
    Walk w;
    if (!w.start(b, aux.place, line)) {
        // nothing to do: on to the common exit
    } else if (warp == 0 || warp == 2) {
        // ---- keys: panels 0-4 and 5-8 ----
        int it = 0;
        bool ok = true;
        do {
            for (int t = 0; ok && t < w.n && w.u.tiles; t++, it++) {
                const int s = it % kStages, kb = (w.u.tile0 + w.at.off + t) * kKeys;
                const uint32_t to = base + kOffK + s * kTile, bar = smem_addr(&aux.k_full[s]);
                const auto ready = [&] { return it < kStages || wait.warp(smem_addr(&aux.k_empty[s]), (it / kStages - 1) & 1); };
                ok = warp == 0 ? load_latent_tile<kKeys, 5>(p, w, kb, to, bar, &map, [](int h) { return h * 64; }, ready)
                               : load_latent_tile<kKeys, 4>(p, w, kb, to + 5 * kPanel, bar, &map, [](int h) { return (h + 5) * 64; }, ready);
            }
        } while (ok && w.next(b));
    } else if (warp == 3) {
        // ---- queries: as soon as the last scores of the unit before are out ----
        int units = 0;
        do {
            if (w.u.tiles == 0) continue;
            if (units && !wait.warp(smem_addr(&aux.q_empty), (units - 1) & 1)) break;
            units++;
            const int boxes = (w.u.rows + p.q_rows - 1) / p.q_rows;
            if (lane == 0) mbar_arrive_expect_tx(smem_addr(&aux.q_full), (uint32_t)(boxes * p.q_rows) * 9 * 128);
            __syncwarp();
            for (int i = lane; i < boxes; i += 32) {
                const int row = w.u.row0 + i * p.q_rows, tok = (int)fdiv((uint32_t)row, b.group), head = row - tok * (int)b.group.d;
#pragma unroll
                for (int h = 0; h < 9; h++)
                    tma_load_3d(base + h * kQPanel + i * p.q_rows * 128, &q_map, smem_addr(&aux.q_full), h * 64, head, w.q.q0 + tok);
            }
            __syncwarp();
        } while (w.next(b));
    } else if (warp == 1) {
        // ---- matrix products ----
        constexpr uint32_t qk_desc = mma_desc(Bf16, kRows, kKeys, false), pv_desc = mma_desc(Bf16, kRows, kHalf, true);
        const uint32_t elected = elect_one();
        const uint64_t qd = smem_desc(base, 16, 1024), kd = smem_desc(base + kOffK, 16, 1024), vd = smem_desc(base + kOffK, kPanel, 1024),
                       pd = smem_desc(base + kOffP, 16, 1024);
        int it = 0, units = 0;
        bool ok = true;
        do {
            if (w.u.tiles == 0) continue;
            ok = wait.warp(smem_addr(&aux.q_full), units++ & 1);
            if (!ok) break;
            const auto qk = [&](int i) {
                const int n = it + i, s = n % kStages;
                if (!wait.warp(smem_addr(&aux.k_full[s]), (n / kStages) & 1)) return false;
                tc_fence_after();
                const uint64_t ks = kd + s * (kTile >> 4);
#pragma unroll
                for (int kk = 0; kk < 36; kk++) {
                    const uint32_t p16 = kk / 4, o = (kk % 4) * 2;
                    mma_ss(tmem + kTmS + (n & 1) * kKeys, qd + p16 * (kQPanel >> 4) + o, ks + p16 * (kPanel >> 4) + o, qk_desc, kk > 0, elected);
                }
                if (i + 1 == w.n) tc_commit(smem_addr(&aux.q_empty), elected);
                tc_commit(smem_addr(&aux.s_full[n & 1]), elected);
                return true;
            };
            ok = qk(0);
            for (int i = 0; ok && i < w.n; i++) {
                if (i + 1 < w.n && !(ok = qk(i + 1))) break;
                const int n = it + i, s = n % kStages;
                ok = wait.warp(smem_addr(&aux.p_ready), n & 1);
                if (!ok) break;
                tc_fence_after();
                const uint64_t vs = vd + s * (kTile >> 4);
#pragma unroll
                for (int kk = 0; kk < kKeys / 16; kk++) {
                    mma_ss(tmem + kTmO, pd + kk * 2, vs + kk * (2048 >> 4), pv_desc, i > 0 || kk > 0, elected);
                    mma_ss(tmem + kTmO + kUpper, pd + kk * 2, vs + (4 * kPanel >> 4) + kk * (2048 >> 4), pv_desc, i > 0 || kk > 0, elected);
                }
                tc_commit(smem_addr(&aux.k_empty[s]), elected);
                tc_commit(smem_addr(&aux.o_done), elected);  // last: the softmax warps wait for it before the CTA ends
            }
            it += w.n;
        } while (ok && w.next(b));
    } else if (warp >= 4) {
        // ---- softmax: rows 16 x .. 16 x + 15 of the unit in this warp's lanes, twice ----
        const int x = warp & 3, row = 16 * x + (lane & 15), half = lane >> 4;
        const uint32_t mine = (uint32_t)(x * 32) << 16;
        const uint32_t o_at = tmem + kTmO + mine;
        const float slack = 8.0f / p.o.c;
        int it = 0, cuts = 0;
        bool ok = true;
        do {
            const bool live = row < w.u.rows;
            const int r = w.u.row0 + min(row, w.u.rows - 1);
            const int tok = (int)fdiv((uint32_t)r, b.group), head = r - tok * (int)b.group.d;
            const int64_t out_row = (int64_t)(w.q.q0 + tok);
            char *to = p.o.out + out_row * p.o.out_token + (int64_t)head * p.o.out_head + half * kHalf * 2;
            if (w.u.tiles == 0) {
                if (live) {
                    for (int col = 0; col < kHalf; col += 8) *reinterpret_cast<uint4 *>(to + col * 2) = make_uint4(0, 0, 0, 0);
                    if (p.o.lse && half == 0) p.o.lse[out_row * p.o.heads + head] = -INFINITY;
                }
                continue;
            }
            const bool warp_live = __any_sync(0xffffffffu, live);
            int lo, hi;
            sees(b, w.q, tok, lo, hi);
            float m = -INFINITY, l = 0.0f;
            const int kt0 = w.u.tile0 + w.at.off;
            for (int k = 0; k < w.n; k++) {
                const int kb = (kt0 + k) * kKeys, n = it + k;
                if (!wait.warp(smem_addr(&aux.s_full[n & 1]), (n >> 1) & 1)) { ok = false; break; }
                tc_fence_after();
                uint32_t pk[16];
                float alpha = 1.0f;
                bool any = false;
                if (warp_live) {
                    uint32_t v[32];
                    tmem_ld32(tmem + kTmS + (n & 1) * kKeys + mine, v);
                    tc_wait_ld();
                    if (__any_sync(0xffffffffu, kb < lo || kb + kKeys > hi)) hide32(v, lo - kb, hi - kb);
                    // the upper lanes hold no scores; they follow the row's maximum for their half of O
                    const float top = __shfl_sync(0xffffffffu, max32(v, -INFINITY), lane & 15);
                    const bool grow = top > (Bf16 ? m + slack : __fadd_rd(m, slack));
                    any = __any_sync(0xffffffffu, grow);
                    if (any) {
                        const float to_m = grow ? top : m;
                        alpha = grow ? exp2_fast((m - to_m) * p.o.c) : 1.0f;
                        l *= alpha;
                        m = to_m;
                    }
                    const float mc = weight_offset<Bf16>(m, p.o.c);
                    float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                    weights32<Bf16>(v, p.o.c, mc, sum, pk);
                    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                }
                // the product before this tile's: it reads P, and O is rescaled behind it
                if (n > 0 && !wait.warp(smem_addr(&aux.o_done), (n - 1) & 1)) { ok = false; break; }
                if (warp_live) {
                    if (any && k > 0) {
                        tc_fence_after();
#pragma unroll 1
                        for (int q = 0; q < kHalf / 32; q++) {
                            uint32_t o[32];
                            tmem_ld32(o_at + q * 32, o);
                            tc_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                            tmem_st32(o_at + q * 32, o);
                        }
                        tc_wait_st();
                    }
                    if (half == 0)
#pragma unroll
                        for (int c = 0; c < 4; c++)
                            st_smem16(base + kOffP + panel_off(row, c), make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]));
                }
                // rows that no query sees must not reach the second product (the scores of this tile are out)
                if (kb < w.u.lo || kb + kKeys > w.u.hi) {
                    const int key = kb + lane;
                    if (key < w.u.lo || key >= w.u.hi) {
                        const uint32_t va = base + kOffK + (n % kStages) * kTile + lane * 128 + x * 2 * kPanel;
#pragma unroll
                        for (int i = 0; i < 16; i++) st_smem16(va + (i >> 3) * kPanel + (i & 7) * 16, make_uint4(0, 0, 0, 0));
                    }
                }
                fence_async_smem();
                tc_fence_before();
                warp_arrive(smem_addr(&aux.p_ready));
            }
            if (!ok) break;
            it += w.n;
            if (!wait.warp(smem_addr(&aux.o_done), (it - 1) & 1)) { ok = false; break; }
            tc_fence_after();
            l = __shfl_sync(0xffffffffu, l, lane & 15);
            const bool whole = w.whole();
            const float inv = l > 0.0f ? 1.0f / l : 0.0f;
            // a CTA's two halves are the fragments of the join
            float *frag = p.ws + (int64_t)(2 * (2 * blockIdx.x + half) + (w.at.off == 0 ? 1 : 0)) * (kRows * (kHalf + 2));
            if (warp_live) {
#pragma unroll 1
                for (int q = 0; q < kHalf / 32; q++) {
                    uint32_t o[32];
                    tmem_ld32(o_at + q * 32, o);
                    tc_wait_ld();
                    float f[32];
#pragma unroll
                    for (int i = 0; i < 32; i++) f[i] = l == 0.0f ? 0.0f : __uint_as_float(o[i]);
                    if (whole)
                        store_rows32<Bf16>(live ? to : nullptr, f, inv, q * 32, kHalf);
                    else if (live)
                        store_fragment32(frag, kRows, row, q, f);
                }
                if (live) {
                    if (whole) {
                        if (p.o.lse && half == 0) p.o.lse[out_row * p.o.heads + head] = l > 0.0f ? fmaf(m, p.o.scale, weight_log<Bf16>(l)) : -INFINITY;
                    } else {
                        frag[kRows * kHalf + row] = m;
                        frag[kRows * (kHalf + 1) + row] = l;
                    }
                }
            }
            if (!whole) {
                const Cut cut(line, w.pos - w.at.off, unit_cost(w.u));
                join_unit<kHalf, Bf16>(p.o, p.ws, cut, p.counters + cut.c0, 1, 2, 0, 2, kRows * (kHalf + 2), 0, w.u.rows, kRows, w.u.row0, w.q.q0, 0,
                                       b.group, smem_addr(&aux.join), cuts, &aux.answer, wait, ok);
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
    if (warp == 2) tmem_free(tmem, 512);
}

}  // namespace

int run_latent_few(bool bf16, const CUtensorMap &map, const CUtensorMap &q_map, const LatentParams &p, int parts, cudaStream_t s)
{
    return cuda_status(launch(bf16 ? latent_few_kernel<true> : latent_few_kernel<false>, dim3(parts), dim3(kThreads), kBytes, s, map, q_map, p));
}

int preload_latent_few_kernels()
{
    int st = cuda_status(cudaFuncSetAttribute(latent_few_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kBytes));
    if (st == KV_OK) st = cuda_status(cudaFuncSetAttribute(latent_few_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kBytes));
    return st != KV_OK ? st : load_kernels(latent_few_kernel<false>, latent_few_kernel<true>);
}

}  // namespace pkv
