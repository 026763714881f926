// kv_latent_expand: the latent rows of a paged cache multiplied out to per-head keys and values.
//
//   K[j, h] = [ W[h, 0:128] c_j ; rope_j ]     V[j, h] = W[h, 128:256] c_j       (c_j: 512 values, rope_j: 64)
//
// One product of 128 tokens by 128 columns (a head's keys, or its values) over 512.  A CTA keeps its token
// tile's latents in tensor memory (256 columns; they come by TMA, page by page, through 64 KB of shared memory) and
// streams the heads' weights past them in panels of 64 by 128: shared memory then moves 64 bytes a cycle in and
// 64 out, its rate, where both operands from there were a quarter over it.  Two accumulators of 128 columns,
// one for keys and one for values, each rounded and written by a warp group while the other is formed.  The line (kv_plan.cuh) runs over requests, token
// tiles and heads, in equal pieces a CTA, so few tokens spread their heads over the GPU.  The rotary part
// is copied beside the product.
// Four prompts of 4096 to 8192 tokens, 32 heads, take 142 us: 73% of the rate at which memory takes the rows, bound
// by the weights' way through the L2 and shared memory (half a tile's latents staged at a time, so that ten
// weight panels are in flight: 159 us with all of them staged and fewer panels).
#include "kv_attention.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 384;
constexpr int kTile = 128;
constexpr int kRank = 512, kRope = 64, kNope = 128, kV = 128, kN = kNope + kV;
constexpr uint32_t kAPanel = kTile * 128, kBPanel = kNope * 128;
constexpr int kStages = 10, kAPart = 4;  // panels of latents that stand in shared memory at a time
constexpr uint32_t kTmA = 256;  // accumulators: columns 0 and 128
constexpr uint32_t kOffB = kAPart * kAPanel, kOffAux = kOffB + kStages * kBPanel, kBytes = kOffAux + 1024;

struct Params {
    const int32_t *kv_lens;
    const int32_t *table, *out_table;
    int64_t table_stride, out_stride;
    int32_t n_reqs, max_tokens, out_tokens;  // capacities of a row of either table in tokens
    int32_t num_blocks, out_blocks;
    FastDiv block, out_block;
    int32_t piece_rows, heads;
    const char *rows;  // the latent tensor, for its rotary parts
    int64_t block_stride, token_stride;
    char *k, *v;
    int64_t k_block, k_token, v_block, v_token;
    int *err;
};

struct Aux {
    uint64_t a_full, a_moved[2], b_full[kStages], b_empty[kStages], d_full[2], d_empty[2];
    int scan[48];
    Place place;
    uint32_t tmem;
    int gave_up;
};
static_assert(sizeof(Aux) <= 1024, "bookkeeping");

__device__ __forceinline__ int request_len(const Params &p, int r, bool report)
{
    const int n = __ldg(p.kv_lens + r), most = min(p.max_tokens, p.out_tokens), len = min(max(n, 0), most);
    if (report && n != len) set_error(p.err, KV_DERR_TABLE);
    return len;
}

// The line: a unit is a token tile, its steps are the heads.
struct ExpandWork {
    static constexpr int kSnap = 0;
    const Params &p;
    bool report;
    __device__ __forceinline__ int units(int r) const { return (request_len(p, r, false) + kTile - 1) / kTile; }
    __device__ __forceinline__ void measure(int r, int &steps, int &n) const
    {
        const int tiles = (request_len(p, r, report) + kTile - 1) / kTile;
        n += tiles;
        steps = add_steps(steps, tiles * p.heads);
    }
    __device__ __forceinline__ int pieces(int r, int each) const { return units(r) * ceil_div(p.heads, each); }
    __device__ __forceinline__ Place own(int r, int k, int each) const
    {
        const int n = ceil_div(p.heads, each);
        Place pl;
        pl.req = r, pl.head = 0;
        pl.unit = (int)((uint32_t)k / (uint32_t)n);
        pl.nth = k - pl.unit * n;
        pl.off = pl.nth * each;
        pl.steps = min(each, p.heads - pl.off);
        return pl;
    }
};

// Fragments of a piece: heads [head, head + n) of one token tile.
struct Walk {
    int req, tile, head, left, len, n;
    __device__ __forceinline__ bool start(const Params &p, const Aux &a, int steps)
    {
        req = a.place.req, tile = a.place.unit, head = a.place.off, left = steps;
        if (left <= 0) return false;
        len = request_len(p, req, false);
        n = min(left, p.heads - head);
        return true;
    }
    __device__ __forceinline__ bool next(const Params &p)
    {
        left -= n;
        if (left <= 0) return false;
        head = 0;
        tile++;
        while (tile * kTile >= len) {
            tile = 0;
            len = request_len(p, ++req, false);
        }
        n = min(left, p.heads);
        return true;
    }
};

template <bool Bf16>
__global__ void __launch_bounds__(kThreads, 1)
expand_kernel(const __grid_constant__ CUtensorMap a_map, const __grid_constant__ CUtensorMap w_map, const Params p)
{
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t base = smem_addr(smem);
    Aux &aux = *reinterpret_cast<Aux *>(smem + kOffAux);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const Waiter wait{&aux.gave_up, p.err};

    if (tid == 0) {
        aux.gave_up = 0;
        mbar_init(smem_addr(&aux.a_full), 1);
        for (int i = 0; i < 2; i++) mbar_init(smem_addr(&aux.a_moved[i]), 8);  // the halves of a tile
        for (int i = 0; i < kStages; i++) mbar_init(smem_addr(&aux.b_full[i]), 1), mbar_init(smem_addr(&aux.b_empty[i]), 1);
        for (int i = 0; i < 2; i++) mbar_init(smem_addr(&aux.d_full[i]), 1), mbar_init(smem_addr(&aux.d_empty[i]), 4);
        mbar_init_fence();
        tma_prefetch_map(&a_map);
        tma_prefetch_map(&w_map);
    }
    if (warp == 2) tmem_alloc(smem_addr(&aux.tmem), 512);
    grid_dep_entry();
    const Line line = find_piece<kThreads>(p.n_reqs, blockIdx.x, gridDim.x, 1, aux.scan, &aux.place, ExpandWork{p, blockIdx.x == 0});
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, aux.tmem, 0);

    Walk w;
    if (!w.start(p, aux, line.steps)) {
        // nothing to do: on to the common exit
    } else if (warp == 2) {
        // ---- latents: half of a token tile's panels at a time, each as soon as the one before has been moved on ----
        const int pr = p.piece_rows;
        int round = 0;
        bool ok = true;
        do {
            const int kb = w.tile * kTile, p1 = (min(w.len - kb, kTile) + pr - 1) / pr;
            const int32_t *row = p.table + (int64_t)w.req * p.table_stride;
            const uint32_t abar = smem_addr(&aux.a_full);
            for (int part = 0; part < 8; part += kAPart, round++) {
                if (round && !(ok = wait.warp(smem_addr(&aux.a_moved[(round - 1) & 1]), ((round - 1) >> 1) & 1))) break;
                if (lane == 0) mbar_arrive_expect_tx(abar, (uint32_t)(p1 * pr) * kAPart * 128);
                __syncwarp();
                for (int j = lane; j < p1; j += 32) {
                    const uint32_t key = (uint32_t)(kb + j * pr), col = fdiv(key, p.block);
                    int page = __ldg(row + col);
                    if (page < 0 || page >= p.num_blocks) {
                        set_error(p.err, KV_DERR_TABLE);
                        page = p.num_blocks;  // outside the map: reads zeros
                    }
#pragma unroll
                    for (int h = 0; h < kAPart; h++)
                        tma_load_4d(base + h * kAPanel + j * pr * 128, &a_map, abar, (part + h) * 64, 0, (int)(key - col * p.block.d), page);
                }
                __syncwarp();
            }
        } while (ok && w.next(p));
    } else if (warp == 0) {
        // ---- weights ----
        int it = 0;
        bool ok = true;
        do {
            for (int h = 0; ok && h < 2 * w.n; h++)
                for (int kk = 0; kk < 8; kk++, it++) {
                    const int s = it % kStages;
                    if (it >= kStages && !(ok = wait.warp(smem_addr(&aux.b_empty[s]), ((it / kStages) - 1) & 1))) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(smem_addr(&aux.b_full[s]), kBPanel);
                        tma_load_3d(base + kOffB + s * kBPanel, &w_map, smem_addr(&aux.b_full[s]), kk * 64, (h & 1) * kNope, w.head + (h >> 1));
                    }
                    __syncwarp();
                }
        } while (ok && w.next(p));
    } else if (warp == 1) {
        constexpr uint32_t desc = mma_desc(Bf16, 128, kNope, false);
        const uint32_t elected = elect_one();
        const uint64_t bd = smem_desc(base + kOffB, 16, 1024);
        int it = 0, heads = 0, frag = 0;
        bool ok = true;
        do {
            ok = wait.warp(smem_addr(&aux.a_moved[0]), frag & 1) && wait.warp(smem_addr(&aux.a_moved[1]), frag & 1);
            frag++;
            tc_fence_after();
            for (int h = 0; ok && h < w.n; h++, heads++)
                for (int d = 0; ok && d < 2; d++) {
                    ok = heads < 1 || wait.warp(smem_addr(&aux.d_empty[d]), (heads - 1) & 1);
                    for (int kk = 0; ok && kk < 8; kk++, it++) {
                        const int s = it % kStages;
                        ok = wait.warp(smem_addr(&aux.b_full[s]), (it / kStages) & 1);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t bb = bd + s * (kBPanel >> 4);
#pragma unroll
                        for (int j = 0; j < 4; j++) mma_ts(tmem + d * kNope, tmem + kTmA + kk * 32 + j * 8, bb + j * 2, desc, kk > 0 || j > 0, elected);
                        tc_commit(smem_addr(&aux.b_empty[s]), elected);
                    }
                    if (ok) tc_commit(smem_addr(&aux.d_full[d]), elected);  // last: the writing warps wait for it before the CTA ends
                }
        } while (ok && w.next(p));
    } else if (warp >= 4) {
        const int g = (warp - 4) >> 2, t = tid & 127;  // group 0 writes the keys, group 1 the values
        const uint32_t mine = (uint32_t)((warp & 3) * 32) << 16;
        const int row_bytes = (g ? kV : kNope + kRope) * 2;
        int heads = 0;
        bool frag = false;  // a tile before this one
        bool ok = true;
        do {
            const int tok = w.tile * kTile + t;
            bool live = tok < w.len;
            char *to = nullptr;
            uint4 rope[kRope / 16];
            if (live) {
                const uint32_t col = fdiv((uint32_t)tok, p.out_block);
                const int page = __ldg(p.out_table + (int64_t)w.req * p.out_stride + col), slot = tok - (int)(col * p.out_block.d);
                if (page < 0 || page >= p.out_blocks) {
                    set_error(p.err, KV_DERR_TABLE);
                    live = false;  // nowhere to write
                } else {
                    to = g ? p.v + page * p.v_block + slot * p.v_token : p.k + page * p.k_block + slot * p.k_token;
                }
            }
            // the rotary parts: eight lanes a row (16 bytes each), four rows at a time, half of the rows a group
            char *rope_to[kRope / 16];
#pragma unroll
            for (int i = 0; i < kRope / 16; i++) {
                const int row = (warp & 3) * 32 + g * 16 + i * 4 + (lane >> 3), rt = w.tile * kTile + row;
                rope_to[i] = nullptr;
                if (rt < w.len) {
                    const uint32_t col = fdiv((uint32_t)rt, p.out_block), scol = fdiv((uint32_t)rt, p.block);
                    const int page = __ldg(p.out_table + (int64_t)w.req * p.out_stride + col), slot = rt - (int)(col * p.out_block.d);
                    const int spage = __ldg(p.table + (int64_t)w.req * p.table_stride + scol), sslot = rt - (int)(scol * p.block.d);
                    if (page >= 0 && page < p.out_blocks) rope_to[i] = p.k + page * p.k_block + slot * p.k_token + kNope * 2 + (lane & 7) * 16;
                    rope[i] = spage >= 0 && spage < p.num_blocks
                                  ? *reinterpret_cast<const uint4 *>(p.rows + spage * p.block_stride + sslot * p.token_stride + kRank * 2 + (lane & 7) * 16)
                                  : make_uint4(0, 0, 0, 0);
                }
            }
            // the tile's latents into tensor memory, half of the panels a group, once the last product of the tile before,
            // which reads the ones that they replace, has ended (both groups have seen the last but one end, so the
            // barrier is in this phase or past it)
            if (frag && !wait.warp(smem_addr(&aux.d_full[1]), (heads - 1) & 1)) break;
            tc_fence_after();
            frag = true;
            for (int part = 0; part < 8; part += kAPart) {
                if (!(ok = wait.warp(smem_addr(&aux.a_full), (part / kAPart) & 1))) break;
#pragma unroll 1
                for (int i = g; i < kAPart; i += 2) {
                    uint32_t x[32];
#pragma unroll
                    for (int j = 0; j < 8; j++) {
                        const uint4 v = ld_smem16(base + i * kAPanel + panel_off(t, j));
                        x[4 * j] = v.x, x[4 * j + 1] = v.y, x[4 * j + 2] = v.z, x[4 * j + 3] = v.w;
                    }
                    tmem_st32(tmem + kTmA + (part + i) * 32 + mine, x);
                }
                tc_wait_st();
                tc_fence_before();
                fence_async_smem();  // the loads before the TMA that overwrites what they read
                warp_arrive(smem_addr(&aux.a_moved[part / kAPart]));
            }
            if (!ok) break;
            for (int h = 0; h < w.n; h++, heads++) {
                const int head = w.head + h;
                if (!wait.warp(smem_addr(&aux.d_full[g]), heads & 1)) { ok = false; break; }
                tc_fence_after();
#pragma unroll 1
                for (int q = 0; q < kNope / 32; q++) {
                    uint32_t x[32];
                    tmem_ld32(tmem + g * kNope + q * 32 + mine, x);
                    tc_wait_ld();
                    float f[32];
#pragma unroll
                    for (int i = 0; i < 32; i++) f[i] = __uint_as_float(x[i]);
                    // a warp group takes the keys, the other the values
                    store_rows32<Bf16>(live ? to + head * row_bytes : nullptr, f, 1.0f, q * 32, kNope);
                }
                tc_fence_before();
                warp_arrive(smem_addr(&aux.d_empty[g]));
#pragma unroll
                for (int i = 0; i < kRope / 16; i++)
                    if (rope_to[i] != nullptr) *reinterpret_cast<uint4 *>(rope_to[i] + head * (kNope + kRope) * 2) = rope[i];
            }
        } while (ok && w.next(p));
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

int preload_expand_kernels()
{
    int st = cuda_status(cudaFuncSetAttribute(expand_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kBytes));
    if (st == KV_OK) st = cuda_status(cudaFuncSetAttribute(expand_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kBytes));
    return st != KV_OK ? st : load_kernels(expand_kernel<false>, expand_kernel<true>);
}

}  // namespace pkv

using namespace pkv;

extern "C" int kv_latent_expand(int32_t dtype, int32_t n_heads, const kv_cache_desc *cache, int32_t tensor, const int32_t *block_table,
                                int32_t n_reqs, int32_t max_blocks_per_req, int64_t bt_row_stride, const int32_t *kv_lens, const void *weight,
                                const kv_cache_desc *k_out, int32_t k_tensor, const kv_cache_desc *v_out, int32_t v_tensor,
                                const int32_t *out_table, int32_t out_blocks_per_req, int64_t out_row_stride, kv_stream_t stream)
{
    if ((dtype != KV_BF16 && dtype != KV_F16) || n_heads <= 0 || n_reqs < 0 || max_blocks_per_req < 0 || out_blocks_per_req < 0 ||
        bt_row_stride < 0 || out_row_stride < 0)
        return KV_ERR_INVALID_ARG;
    int st = check_plane(cache, tensor, 0, 1, kRank + kRope);
    if (st != KV_OK) return st;
    if ((st = check_plane(k_out, k_tensor, 0, n_heads, kNope + kRope)) != KV_OK) return st;
    if ((st = check_plane(v_out, v_tensor, 0, n_heads, kV)) != KV_OK) return st;
    if (k_out->block_size != v_out->block_size) return KV_ERR_INVALID_ARG;
    if (n_reqs == 0 || max_blocks_per_req == 0 || out_blocks_per_req == 0) return KV_OK;
    if (block_table == nullptr || out_table == nullptr || kv_lens == nullptr || weight == nullptr) return KV_ERR_INVALID_ARG;
    if (n_reqs > 1 && (bt_row_stride < max_blocks_per_req || out_row_stride < out_blocks_per_req)) return KV_ERR_INVALID_ARG;
    if (!aligned16(weight)) return KV_ERR_ALIGN;
    const int64_t max_tokens = (int64_t)max_blocks_per_req * cache->block_size, out_tokens = (int64_t)out_blocks_per_req * k_out->block_size;
    if (max_tokens > (1ll << 30) || out_tokens > (1ll << 30) || (int64_t)n_reqs * n_heads > ((1ll << 31) - 1) / (max_tokens / kTile + 1))
        return KV_ERR_UNSUPPORTED;
    const DeviceInfo *dev = current_device();
    if (dev == nullptr) return KV_ERR_CUDA;
    if ((st = prepare_attention(*dev)) != KV_OK) return st;
    Params p = {};
    p.kv_lens = kv_lens;
    p.table = block_table;
    p.out_table = out_table;
    p.table_stride = bt_row_stride;
    p.out_stride = out_row_stride;
    p.n_reqs = n_reqs;
    p.max_tokens = (int32_t)max_tokens;
    p.out_tokens = (int32_t)out_tokens;
    p.num_blocks = (int32_t)cache->num_blocks;
    p.out_blocks = (int32_t)(k_out->num_blocks < v_out->num_blocks ? k_out->num_blocks : v_out->num_blocks);
    p.block = make_fastdiv((uint32_t)cache->block_size);
    p.out_block = make_fastdiv((uint32_t)k_out->block_size);
    p.piece_rows = piece_rows(cache->block_size, kTile);
    p.heads = n_heads;
    p.rows = (const char *)cache->base[tensor];
    p.block_stride = cache->block_stride;
    p.token_stride = cache->token_stride;
    p.k = (char *)k_out->base[k_tensor];
    p.v = (char *)v_out->base[v_tensor];
    p.k_block = k_out->block_stride;
    p.k_token = k_out->token_stride;
    p.v_block = v_out->block_stride;
    p.v_token = v_out->token_stride;
    p.err = dev->err_word;
    CUtensorMap am, wm;
    if ((st = make_cache_map(&am, cache, tensor, 0, 1, kRank + kRope, p.piece_rows)) != KV_OK) return st;
    const uint64_t dims[3] = {kRank, kN, (uint64_t)n_heads}, strides[2] = {kRank * 2, kRank * 2 * kN};
    const uint32_t box[3] = {64, kNope, 1};
    if ((st = make_map(&wm, (uint64_t)weight, 3, dims, strides, box)) != KV_OK) return st;
    return cuda_status(launch(dtype == KV_BF16 ? expand_kernel<true> : expand_kernel<false>, dim3(dev->num_sms), dim3(kThreads), kBytes,
                              (cudaStream_t)stream, am, wm, p));
}
