// kv_latent_attention: attention over one shared latent row a token (the absorbed form).
//
// This kernel takes units of up to 128 query rows (kv_latent_few.cu: 64).
//
// Keys are whole rows of 576 elements, values their first 512.  The accumulator of 128 query rows by 512
// values would fill tensor memory by itself, so two CTAs share a part of the batch's line
// (kv_plan.cuh): each forms the products S = Q K^T over all 576 elements and accumulates 256 of the 512
// values.  The scores are computed twice (576 + 256 multiply-adds a key, row and CTA instead of 544), but
// nothing has to be exchanged, and every operand stays on chip:
//   TMEM           O 256 columns, S twice 64, Q's first four panels 128 (A operand from TMEM)
//   shared memory  Q's other five panels 80 KB; two tiles of 64 keys, 72 KB each: the four panels that
//                  are this CTA's values, and the five that the scores alone use and free earlier
//   warps 0 and 2 load the two kinds of panels, warp 3 loads Q, warp 1 issues the products, warps 4-7 hold
//   a row a thread (maximum, exponentials, P over S, lazy rescaling as in kv_attention.cu).  S of the next
//   tile is formed before O += P V of this one, so the tensor core works while the exponentials run.
// 64 requests of 4096 to 12288 tokens, 128 heads, take 183 to 188 us, half of the rate at which memory could bring the rows
// (each is read once, by both CTAs of a pair, the second time from the L2).  A tile of 64 keys takes about 3300 cycles, and
// needs 1664 of the tensor core and about 2050 of shared memory for the products' operands and the loads.  What bounds it
// is a trip to memory a tile: two tiles stand at a time, and a tile's value panels are free only behind its value
// product, while the scores of the next but one wait for them.
#include "kv_latent.cuh"

namespace pkv {

namespace {

constexpr int kLeast = 2;  // steps of a piece of a unit, at least (of 64 keys)
constexpr int kThreads = 256;
constexpr int kRows = 128;
constexpr int kKeyShift = 6, kKeys = 1 << kKeyShift;  // keys of a tile
constexpr int kHalf = kLatentRank / 2;
constexpr int kQT = 4;         // panels of Q in tensor memory
constexpr uint32_t kQPanel = 128 * 128, kPanel = kKeys * 128;
constexpr uint32_t kOffV = 5 * kQPanel, kOffX = kOffV + 2 * 4 * kPanel, kOffAux = kOffX + 2 * 5 * kPanel;
constexpr uint32_t kBytes = kOffAux + 1024;
constexpr uint32_t kTmO = 0, kTmS = 256, kTmQ = 384;

struct Aux {
    uint64_t v_full[2], v_empty[2], x_full[2], x_empty[2], s_full[2], p_ready[2], o_done[2], q_staged, q_moved, q_full, q_empty, join;
    int scan[32];
    Place place;
    uint32_t tmem;
    int answer;
    int gave_up;
};
static_assert(sizeof(Aux) <= 1024, "bookkeeping");

template <bool Bf16>
__global__ void __launch_bounds__(kThreads, 1)
latent_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ CUtensorMap q_map, const LatentParams p)
{
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t base = smem_addr(smem);
    Aux &aux = *reinterpret_cast<Aux *>(smem + kOffAux);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int part = blockIdx.x >> 1, half = blockIdx.x & 1;
    const Batch &b = p.b;
    const Waiter wait{&aux.gave_up, b.err};

    if (tid == 0) {
        aux.gave_up = 0;
        for (int i = 0; i < 2; i++) {
            mbar_init(smem_addr(&aux.v_full[i]), 1);
            mbar_init(smem_addr(&aux.v_empty[i]), 1);
            mbar_init(smem_addr(&aux.x_full[i]), 1);
            mbar_init(smem_addr(&aux.x_empty[i]), 1);
            mbar_init(smem_addr(&aux.s_full[i]), 1);
            mbar_init(smem_addr(&aux.p_ready[i]), 4);
            // by the tile's parity: the softmax warps look at it only now and then, and when they do the
            // product two tiles before has completed (its scores' successor is out) but the last may not have
            mbar_init(smem_addr(&aux.o_done[i]), 1);
        }
        mbar_init(smem_addr(&aux.q_full), 1);
        mbar_init(smem_addr(&aux.q_staged), 1);
        mbar_init(smem_addr(&aux.q_moved), 4);
        mbar_init(smem_addr(&aux.q_empty), 1);
        mbar_init(smem_addr(&aux.join), 4);
        mbar_init_fence();
        tma_prefetch_map(&map);
    }
    if (warp == 2) tmem_alloc(smem_addr(&aux.tmem), 512);
    grid_dep_entry();
    const Line line = find_place<kThreads>(b, part, gridDim.x >> 1, kLeast, aux.scan, &aux.place, blockIdx.x == 0);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, aux.tmem, 0);
    Walk w;
    if (!w.start(b, aux.place, line)) {
        // nothing to do: on to the common exit
    } else if (warp == 0) {
        // ---- the five panels that only the scores use ----
        int it = 0;
        bool ok = true;
        do {
            for (int t = 0; ok && t < w.n && w.u.tiles; t++, it++) {
                const int s = it & 1;
                ok = load_latent_tile<kKeys, 5>(p, w, (w.u.tile0 + w.at.off + t) * kKeys, base + kOffX + s * 5 * kPanel, smem_addr(&aux.x_full[s]), &map,
                                  [&](int h) { return (h == 4 ? 8 : h + 4 - 4 * half) * 64; },  // the other half's values, the rotary part
                                  [&] { return it < 2 || wait.warp(smem_addr(&aux.x_empty[s]), ((it >> 1) - 1) & 1); });
            }
        } while (ok && w.next(b));
    } else if (warp == 2) {
        // ---- the four panels that are this CTA's values too ----
        int it = 0;
        bool ok = true;
        do {
            for (int t = 0; ok && t < w.n && w.u.tiles; t++, it++) {
                const int s = it & 1;
                ok = load_latent_tile<kKeys, 4>(p, w, (w.u.tile0 + w.at.off + t) * kKeys, base + kOffV + s * 4 * kPanel, smem_addr(&aux.v_full[s]), &map,
                                  [&](int h) { return (h + 4 * half) * 64; },
                                  [&] { return it < 2 || wait.warp(smem_addr(&aux.v_empty[s]), ((it >> 1) - 1) & 1); });
            }
        } while (ok && w.next(b));
    } else if (warp == 3) {
        // ---- Q: its four panels for tensor memory by way of the place of the other five, then those ----
        int units = 0;
        const int group = (int)b.group.d;
        do {
            if (w.u.tiles == 0) continue;
            if (units && !wait.warp(smem_addr(&aux.q_empty), (units - 1) & 1)) break;
            units++;
            const auto load = [&](auto count, uint32_t bar, auto column) {
                const int boxes = (w.u.rows + p.q_rows - 1) / p.q_rows;
                if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(boxes * p.q_rows) * count() * 128);
                __syncwarp();
                for (int i = lane; i < boxes; i += 32) {
                    const int row = w.u.row0 + i * p.q_rows, tok = (int)fdiv((uint32_t)row, b.group), head = row - tok * group;
#pragma unroll
                    for (int h = 0; h < count(); h++)
                        tma_load_3d(base + h * kQPanel + i * p.q_rows * 128, &q_map, bar, column(h), head, w.q.q0 + tok);
                }
                __syncwarp();
            };
            load(std::integral_constant<int, kQT>(), smem_addr(&aux.q_staged), [&](int h) { return (h + 4 * half) * 64; });
            if (!wait.warp(smem_addr(&aux.q_moved), (units - 1) & 1)) break;
            load(std::integral_constant<int, 5>(), smem_addr(&aux.q_full), [&](int h) { return (h == 4 ? 8 : h + 4 - 4 * half) * 64; });
        } while (w.next(b));
    } else if (warp == 1) {
        // ---- matrix products ----
        constexpr uint32_t qk_desc = mma_desc(Bf16, 128, kKeys, false), pv_desc = mma_desc(Bf16, 128, kHalf, true);
        const uint32_t elected = elect_one();
        const uint64_t qd = smem_desc(base, 16, 1024), xd = smem_desc(base + kOffX, 16, 1024), kd = smem_desc(base + kOffV, 16, 1024),
                       vd = smem_desc(base + kOffV, kPanel, 1024);
        int it = 0, units = 0;
        bool ok = true;
        do {
            if (w.u.tiles == 0) continue;
            // the TMA for q_full was issued after q_moved, so this covers both; the wait for q_moved orders tensor memory
            ok = wait.warp(smem_addr(&aux.q_moved), units & 1) && wait.warp(smem_addr(&aux.q_full), units & 1);
            units++;
            if (!ok) break;
            tc_fence_after();
            // Q's panels stand in the order of the key panels as this CTA holds them: the five others
            // (shared memory), the four of its values (tensor memory)
            const auto qk = [&](int i) {
                const int n = it + i, s = n & 1;
                const uint32_t d = tmem + kTmS + s * kKeys;
                const bool v_here = Waiter::over(smem_addr(&aux.v_full[s]), (n >> 1) & 1);
                if (!wait.warp(smem_addr(&aux.x_full[s]), (n >> 1) & 1)) return false;
                const uint64_t xs = xd + s * (5 * kPanel >> 4), ks = kd + s * (4 * kPanel >> 4);
#pragma unroll
                for (int kk = 0; kk < 20; kk++)
                    mma_ss(d, qd + (((kk / 4) * kQPanel + (kk % 4) * 32) >> 4), xs + (((kk / 4) * kPanel + (kk % 4) * 32) >> 4), qk_desc, kk > 0, elected);
                tc_commit(smem_addr(&aux.x_empty[s]), elected);
                if (i + 1 == w.n) tc_commit(smem_addr(&aux.q_empty), elected);
                if (!__all_sync(0xffffffffu, v_here) && !wait.warp(smem_addr(&aux.v_full[s]), (n >> 1) & 1)) return false;
#pragma unroll
                for (int kk = 0; kk < 16; kk++)
                    mma_ts(d, tmem + kTmQ + kk * 8, ks + (((kk / 4) * kPanel + (kk % 4) * 32) >> 4), qk_desc, true, elected);
                tc_commit(smem_addr(&aux.s_full[s]), elected);
                return true;
            };
            ok = qk(0);
            for (int i = 0; ok && i < w.n; i++) {
                if (i + 1 < w.n && !(ok = qk(i + 1))) break;
                const int n = it + i, s = n & 1;
                ok = wait.warp(smem_addr(&aux.p_ready[s]), (n >> 1) & 1);
                if (!ok) break;
                tc_fence_after();
                const uint64_t vs = vd + s * (4 * kPanel >> 4);
#pragma unroll
                for (int kk = 0; kk < kKeys / 16; kk++)
                    mma_ts(tmem + kTmO, tmem + kTmS + s * kKeys + kk * 8, vs + kk * (2048 >> 4), pv_desc, i > 0 || kk > 0, elected);
                tc_commit(smem_addr(&aux.v_empty[s]), elected);
                tc_commit(smem_addr(&aux.o_done[s]), elected);  // last: the softmax warps wait for it before the CTA ends
            }
            it += w.n;
        } while (ok && w.next(b));
    } else if (warp >= 4) {
        // ---- softmax: a thread per row ----
        const int t = tid & 127;
        const uint32_t mine = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t o_at = tmem + kTmO + mine;
        const float slack = 8.0f / p.o.c;
        int it = 0, cuts = 0, units = 0;
        bool ok = true;
        // A unit's four panels of Q into tensor memory, once the scores of the unit before are out.
        const auto move_q = [&](const Unit &u) {
            if (!wait.warp(smem_addr(&aux.q_staged), units++ & 1)) return false;
            if (__any_sync(0xffffffffu, t < u.rows)) {
#pragma unroll 1
                for (int q = 0; q < kQT; q++) {
                    uint32_t x[32];
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        const uint4 v = ld_smem16(base + q * kQPanel + panel_off(t, i));
                        x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
                    }
                    tmem_st32(tmem + kTmQ + q * 32 + mine, x);
                }
                tc_wait_st();
            }
            tc_fence_before();
            fence_async_smem();  // the loads before the TMA that overwrites what they read
            warp_arrive(smem_addr(&aux.q_moved));
            return true;
        };
        bool moved = false;  // the unit's Q is on its way already
        do {
            const bool live = t < w.u.rows;
            const int r = w.u.row0 + min(t, w.u.rows - 1);
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
            if (!moved && !(ok = move_q(w.u))) break;
            int lo, hi;
            sees(b, w.q, tok, lo, hi);
            float m = -INFINITY, l = 0.0f;
            const int kt0 = w.u.tile0 + w.at.off;
            for (int k = 0; k < w.n; k++) {
                const int kb = (kt0 + k) * kKeys, n = it + k, s = n & 1;
                const uint32_t s_at = tmem + kTmS + s * kKeys + mine;
                if (!wait.warp(smem_addr(&aux.s_full[s]), (n >> 1) & 1)) { ok = false; break; }
                tc_fence_after();
                if (warp_live) {
                    uint32_t x[2][32];
                    tmem_ld32(s_at, x[0]);
                    tmem_ld32(s_at + 32, x[1]);
                    tc_wait_ld();
                    if (__any_sync(0xffffffffu, kb < lo || kb + kKeys > hi)) {
                        hide32(x[0], lo - kb, hi - kb);
                        hide32(x[1], lo - kb - 32, hi - kb - 32);
                    }
                    const float top = max32(x[1], max32(x[0], -INFINITY));
                    const bool grow = top > (Bf16 ? m + slack : __fadd_rd(m, slack));
                    if (__any_sync(0xffffffffu, grow)) {
                        const float to_m = grow ? top : m;
                        const float alpha = grow ? exp2_fast((m - to_m) * p.o.c) : 1.0f;
                        l *= alpha;
                        m = to_m;
                        if (k > 0) {
                            if (!wait.warp(smem_addr(&aux.o_done[s ^ 1]), ((n - 1) >> 1) & 1)) { ok = false; break; }
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
                        }
                    }
                    const float mc = weight_offset<Bf16>(m, p.o.c);
                    float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                    uint32_t pk[16];
                    weights32<Bf16>(x[0], p.o.c, mc, sum, pk);
                    tmem_st16(s_at, pk);
                    weights32<Bf16>(x[1], p.o.c, mc, sum, pk);
                    tmem_st16(s_at + 16, pk);
                    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                    tc_wait_st();
                }
                // rows that no query sees must not reach the second product (the scores of this tile are out)
                if (kb < w.u.lo || kb + kKeys > w.u.hi) {
                    const int key = kb + (t & 63);
                    if (key < w.u.lo || key >= w.u.hi) {
                        const uint32_t va = base + kOffV + s * 4 * kPanel + (t & 63) * 128 + (t >> 6) * 2 * kPanel;
#pragma unroll
                        for (int i = 0; i < 16; i++) st_smem16(va + (i >> 3) * kPanel + (i & 7) * 16, make_uint4(0, 0, 0, 0));
                    }
                    fence_async_smem();
                }
                tc_fence_before();
                warp_arrive(smem_addr(&aux.p_ready[s]));
            }
            if (!ok) break;
            it += w.n;
            // the next unit's Q now, so that its first scores are formed while this one's rows are written
            {
                Walk nx = w;
                moved = false;
                while (!moved && nx.next(b)) moved = nx.u.tiles > 0;
                if (moved && !(ok = move_q(nx.u))) break;
            }
            if (!wait.warp(smem_addr(&aux.o_done[(it - 1) & 1]), ((it - 1) >> 1) & 1)) { ok = false; break; }
            tc_fence_after();
            const bool whole = w.whole();
            const float inv = l > 0.0f ? 1.0f / l : 0.0f;
            float *frag = p.ws + (int64_t)(2 * blockIdx.x + (w.at.off == 0 ? 1 : 0)) * (kRows * (kHalf + 2));
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
                        store_fragment32(frag, kRows, t, q, f);
                }
                if (live) {
                    if (whole) {
                        if (p.o.lse && half == 0) p.o.lse[out_row * p.o.heads + head] = l > 0.0f ? fmaf(m, p.o.scale, weight_log<Bf16>(l)) : -INFINITY;
                    } else {
                        frag[kRows * kHalf + t] = m;
                        frag[kRows * (kHalf + 1) + t] = l;
                    }
                }
            }
            if (!whole) {
                const Cut cut(line, w.pos - w.at.off, unit_cost(w.u));
                join_unit<kHalf, Bf16>(p.o, p.ws, cut, p.counters + 2 * cut.c0 + half, 2, 2, half, half + 1, kRows * (kHalf + 2), 0, w.u.rows, kRows,
                                       w.u.row0, w.q.q0, 0, b.group, smem_addr(&aux.join), cuts, &aux.answer, wait, ok);
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

int preload_latent_kernels()
{
    int st = cuda_status(cudaFuncSetAttribute(latent_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kBytes));
    if (st == KV_OK) st = cuda_status(cudaFuncSetAttribute(latent_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kBytes));
    if (st == KV_OK) st = preload_latent_few_kernels();
    return st != KV_OK ? st : load_kernels(latent_kernel<false>, latent_kernel<true>);
}

}  // namespace pkv

using namespace pkv;

extern "C" int kv_latent_attention(const kv_attn_desc *d, const kv_attn_batch *batch, const kv_cache_desc *cache, int32_t tensor,
                                   const void *q, int64_t q_token_stride, int64_t q_head_stride, void *out, int64_t out_token_stride,
                                   int64_t out_head_stride, float *lse, void *workspace, int64_t workspace_bytes, kv_stream_t stream)
{
    if (d == nullptr || d->n_heads <= 0 || d->n_kv_heads != 1 || d->window < 0 || !good_scale(d->scale) ||
        (d->dtype != KV_BF16 && d->dtype != KV_F16))
        return KV_ERR_INVALID_ARG;
    int st = check_batch(batch);
    if (st != KV_OK) return st;
    if (d->head_dim != kLatentDim || d->head_dim_v != kLatentRank || (d->window && !d->causal)) return KV_ERR_UNSUPPORTED;
    if ((st = check_plane(cache, tensor, 0, 1, kLatentDim)) != KV_OK) return st;
    if (batch->n_reqs == 0 || batch->n_tokens == 0) return KV_OK;
    if ((st = check_rows(q, q_token_stride, q_head_stride)) != KV_OK) return st;
    if ((st = check_rows(out, out_token_stride, out_head_stride)) != KV_OK) return st;
    if (workspace == nullptr) return KV_ERR_INVALID_ARG;
    if (!aligned16(workspace) || ((uintptr_t)lse & 3u)) return KV_ERR_ALIGN;
    const DeviceInfo *dev = current_device();
    if (dev == nullptr) return KV_ERR_CUDA;
    // Many requests of few rows (tokens times heads, on average) take the kernel that holds 64 rows and all values
    // a CTA, others the one of 128 rows with a CTA for each half of the values.  In us, one token of 16 heads after at
    // most 375, 2500 and 10000 tokens: 14.8, 19.6, 34.2 here against 16.3, 25.2, 33.8 there with 8 requests; 16.0,
    // 26.1, 60.7 against 16.7, 26.7, 53.1 with 19; 27.8, 73.6, 234.9 against 23.6, 57.3, 165.4 with 100.  Of 64 heads
    // 19.6, 41.5, 95.0 against 25.8, 49.3, 90.1 with 32 requests; 29.6, 63.9, 189.4 against 39.8, 66.7, 146.2 with
    // 76; 31.9, 80.0, 242.6 against 33.6, 72.0, 180.8 with 100.  With few requests the join of a unit's pieces, by one
    // CTA there, decides.  The host knows neither the lengths nor which of them a captured graph will meet: with 64 heads the
    // rule costs short contexts up to 10 us and brings long ones up to 62.
    // (Its tiles are half as long: the last condition keeps a batch of any capacity that the other takes.)
    const int64_t reqs = batch->n_reqs, few_rows = reqs < kLatentFewRows ? reqs : kLatentFewRows;
    const bool few = d->n_heads <= kLatentFewRows && batch->n_tokens <= few_rows * reqs / d->n_heads && reqs * 8 >= dev->num_sms &&
                     reqs * ((int64_t)batch->max_blocks_per_req * cache->block_size >> kLatentFewKeyShift) < (1ll << 29);
    // A unit is whole tokens of up to that many heads each, or a divisor of a token's heads; a TMA of q brings all
    // heads of as many tokens as a request has on average (a divisor of a unit's), or a unit.
    const int rows = few ? kLatentFewRows : kRows, key_shift = few ? kLatentFewKeyShift : kKeyShift;
    int box_heads = d->n_heads, box_tokens = 1;
    if (d->n_heads > rows) {
        for (box_heads = rows; d->n_heads % box_heads; box_heads--) {}
    } else {
        box_tokens = pkv::box_tokens(rows / d->n_heads, batch);
    }
    const int unit_rows = d->n_heads > rows ? box_heads : rows / d->n_heads * d->n_heads;
    LatentParams p = {};
    if ((st = fill_batch(&p.b, batch, d->n_heads, 1, cache->block_size, unit_rows, key_shift, d->causal, d->window)) != KV_OK) return st;
    if (workspace_bytes < attention_workspace(dev->num_sms)) return KV_ERR_RANGE;
    if ((st = prepare_attention(*dev)) != KV_OK) return st;
    p.b.err = dev->err_word;
    p.table = batch->block_table;
    p.table_stride = batch->bt_row_stride;
    p.num_blocks = (int32_t)cache->num_blocks;
    p.block = make_fastdiv((uint32_t)cache->block_size);
    p.piece_rows = piece_rows(cache->block_size, 1 << key_shift);
    p.o = Output{(char *)out, out_token_stride, out_head_stride, lse, d->n_heads, kLatentRank, d->scale, d->scale * kLog2e};
    p.counters = (int *)workspace;
    p.ws = (float *)((char *)workspace + kCounterBytes);
    CUtensorMap map, q_map;
    p.q_rows = box_heads * box_tokens;
    if ((st = make_q_map(&q_map, q, q_token_stride, q_head_stride, kLatentDim, d->n_heads, batch->n_tokens, box_heads, box_tokens)) != KV_OK) return st;
    if ((st = make_cache_map(&map, cache, tensor, 0, 1, kLatentDim, p.piece_rows)) != KV_OK) return st;
    if (few) return run_latent_few(d->dtype == KV_BF16, map, q_map, p, dev->num_sms, (cudaStream_t)stream);
    return cuda_status(launch(d->dtype == KV_BF16 ? latent_kernel<true> : latent_kernel<false>, dim3(dev->num_sms / 2 * 2), dim3(kThreads), kBytes,
                              (cudaStream_t)stream, map, q_map, p));
}
